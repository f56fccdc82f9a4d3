"""Plain fp64 definitions of the row-wise operators around the products: root-mean-square norm with
the residual's addition, routing of tokens to experts, gated SiLU, and their gradients.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never imports this file.

Inputs are float64 arrays holding the exact values of the inputs; outputs are unrounded. The
gradients are the formulas; ``tests/test_oracle_rows.py`` checks them against differences of the
forward definitions.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def rmsnorm(x, residual, weight, eps):
    """(h, rstd, y): h = x + residual, rstd = 1 / sqrt(mean(h^2) + eps), y = h * rstd * weight."""
    h = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, rstd, h * rstd[:, None] * weight


def e4m3_row_scale(y):
    """One scale per row: the largest magnitude over 448, 1 for a row of zeros."""
    m = np.abs(y).max(axis=1)
    return np.where(m > 0, m / E4M3_MAX, 1.0)


def rmsnorm_bwd(dy, h, weight, rstd, dres=None):
    """(dx, dweight) for given rstd."""
    n = h * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - n * (g * n).mean(axis=1, keepdims=True))
    return (dx if dres is None else dx + dres), (dy * n).sum(axis=0)


def scores(logits, score):
    """softmax over a row (0 for a row of -inf, NaN where a logit is +inf) or sigmoid."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-logits))
    m = logits.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.exp(logits - np.where(np.isneginf(m), 0.0, m))
    s = e.sum(axis=1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def _descending(key):
    """Indices by descending key, NaN last, equal keys in index order."""
    k = np.where(np.isnan(key), -np.inf, key)
    return np.lexsort((np.broadcast_to(np.arange(key.shape[1]), key.shape), np.isnan(key), -k), axis=1)


def route(logits, k, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """(ids, gates, margin): the chosen experts in descending order of their keys, their gates, and how
    far the nearest decision of a row (between groups, or between successive keys of the choice and
    the best one left out) was from being a different one, ties excluded."""
    T, E = logits.shape
    s = scores(logits, score)
    key = s if bias is None else s + bias
    if score == "softmax" and bias is None:
        key = logits
    margin = np.full(T, np.inf)

    def note(sorted_keys, n):
        with np.errstate(invalid="ignore"):
            gap = sorted_keys[:, :-1] - sorted_keys[:, 1:]
        gap = np.where((gap > 0) & np.isfinite(gap), gap, np.inf)[:, :n]
        if gap.shape[1]:
            np.minimum(margin, gap.min(axis=1), out=margin)

    out = np.zeros((T, E), dtype=bool)
    if n_group > 1:
        per = E // n_group
        in_group = (np.exp(logits - logits.max(axis=1, keepdims=True)) if key is logits and group_top == 2 else key)
        best = -np.sort(-in_group.reshape(T, n_group, per), axis=2)[:, :, :group_top].sum(axis=2)
        order = _descending(best)
        note(np.take_along_axis(best, order, 1)[:, :topk_group + 1][:, -2:], 1)
        keep = np.zeros((T, n_group), dtype=bool)
        np.put_along_axis(keep, order[:, :topk_group], True, 1)
        out = ~np.repeat(keep, per, axis=1)
    rank = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), np.isnan(key),
                       -np.where(np.isnan(key), -np.inf, key), out), axis=1)
    note(np.take_along_axis(np.where(out, -np.inf, key), rank, 1), k)
    ids = rank[:, :k]
    g = np.take_along_axis(s, ids, 1)
    if renorm:
        if score == "softmax":   # the softmax of the chosen logits, where the row's is a number
            g = np.where(np.isnan(g), g, scores(np.take_along_axis(logits, ids, 1), "softmax"))
        else:
            S = g.sum(axis=1, keepdims=True)
            g = g / np.where(S == 0, 1.0, S)
    return ids, g * scale, margin


def route_bwd(logits, ids, dgates, score="softmax", renorm=True, scale=1.0):
    """The gradient of sum(gates * dgates) by the logits, the choice held fixed; places that name one expert add up."""
    s = scores(logits, score)
    sel = np.take_along_axis(s, ids, 1)
    dg = dgates * scale
    d = np.zeros_like(logits)
    at = (np.arange(len(ids))[:, None], ids)
    if renorm:
        if score == "softmax":
            p = scores(np.take_along_axis(logits, ids, 1), "softmax")
            np.add.at(d, at, p * (dg - (dg * p).sum(axis=1, keepdims=True)))
            return d
        S = sel.sum(axis=1, keepdims=True)
        S = np.where(S > 0, S, 1.0)
        dg = (dg - (dg * sel).sum(axis=1, keepdims=True) / S) / S
    np.add.at(d, at, dg)
    if score == "softmax":
        return s * (d - (d * s).sum(axis=1, keepdims=True))
    return d * s * scores(-logits, "sigmoid")


def swiglu(y, row_scale=None):
    I = y.shape[1] // 2
    c = 1.0 if row_scale is None else row_scale[:, None]
    g, u = y[:, :I] * c, y[:, I:] * c
    return g * scores(g, "sigmoid") * u


def swiglu_bwd(y, dout):
    I = y.shape[1] // 2
    g, u = y[:, :I], y[:, I:]
    s = scores(g, "sigmoid")
    return np.concatenate([dout * u * s * (1.0 + g * (1.0 - s)), dout * g * s], axis=1)
