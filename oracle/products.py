"""64-bit reference of the products without communication (linear layer, products grouped by expert, the sum
of a token's expert rows) and their gradients, in numpy on the CPU. Shares nothing with the kernels.

Every product also has its magnitude, the same sum over absolute values, by which rounding errors of the
accumulation are bounded."""
from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "swiglu")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])
_C, _D = math.sqrt(2.0 / math.pi), 0.044715


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def act(name, v):
    """act(v); for swiglu of the two halves of v's columns."""
    if name == "none":
        return v
    if name == "relu":
        return np.where(v < 0, 0.0, v)
    if name == "gelu":
        return 0.5 * v * _erfc(-v * math.sqrt(0.5))
    if name == "gelu_tanh":
        return v * sigmoid(2.0 * _C * (v + _D * v ** 3))
    if name == "silu":
        return v * sigmoid(v)
    half = v.shape[-1] // 2
    return act("silu", v[..., :half]) * v[..., half:]


def act_grad(name, v, dy):
    """Gradient of sum(act(v) * dy) by v."""
    if name == "none":
        return dy
    if name == "relu":
        return np.where(v > 0, dy, 0.0)
    if name == "gelu":
        return dy * (0.5 * _erfc(-v * math.sqrt(0.5)) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        s = sigmoid(2.0 * _C * (v + _D * v ** 3))
        return dy * (s + v * s * (1.0 - s) * 2.0 * _C * (1.0 + 3.0 * _D * v * v))
    if name == "silu":
        s = sigmoid(v)
        return dy * (s + v * s * (1.0 - s))
    half = v.shape[-1] // 2
    g, u = v[..., :half], v[..., half:]
    return np.concatenate([act_grad("silu", g, dy * u), dy * act("silu", g)], -1)


def product(A, B):
    """A @ B and its magnitude."""
    return A @ B, np.abs(A) @ np.abs(B)


def grouped(X, offsets, B):
    """Rows offsets[e] .. offsets[e+1]-1 of X times B[e], and their magnitudes; rows of no expert are NaN."""
    out = np.full((X.shape[0], B.shape[2]), np.nan)
    mag = out.copy()
    for e in range(B.shape[0]):
        at = slice(offsets[e], offsets[e + 1])
        out[at], mag[at] = product(X[at], B[e])
    return out, mag


def grouped_bwd(dY, X, offsets, B):
    """dX, dB and their magnitudes."""
    dX, mX = grouped(dY, offsets, np.swapaxes(B, 1, 2))
    dB = np.zeros(B.shape)
    mB = np.zeros(B.shape)
    for e in range(B.shape[0]):
        at = slice(offsets[e], offsets[e + 1])
        dB[e], mB[e] = product(X[at].T, dY[at])
    return (dX, mX), (dB, mB)


def combine(Z, dest, gates, T):
    """out[t] = sum_j gates[t][j] Z[dest[t][j]], entries outside Z's rows adding nothing, and its magnitude."""
    dest = np.asarray(dest).reshape(T, -1)
    ok = (dest >= 0) & (dest < Z.shape[0])
    g = np.where(ok, 1.0 if gates is None else gates, 0.0)
    rows = Z[np.where(ok, dest, 0)] if Z.shape[0] else np.zeros(dest.shape + (Z.shape[1],))
    rows = np.where(ok[:, :, None], rows, 0.0)
    return np.einsum("tk,tkh->th", g, rows), np.einsum("tk,tkh->th", np.abs(g), np.abs(rows))


def combine_bwd(dout, Z, dest, gates):
    """dZ (rows that dest does not name: NaN), dgates and the latter's magnitude."""
    T = dout.shape[0]
    dest = np.asarray(dest).reshape(T, -1)
    dZ = np.full(Z.shape, np.nan)
    dg, mag = np.zeros(dest.shape), np.zeros(dest.shape)
    for t in range(T):
        for j, r in enumerate(dest[t]):
            if 0 <= r < Z.shape[0]:
                dZ[r] = (1.0 if gates is None else gates[t, j]) * dout[t]
                dg[t, j] = dout[t] @ Z[r]
                mag[t, j] = np.abs(dout[t]) @ np.abs(Z[r])
    return dZ, dg, mag
