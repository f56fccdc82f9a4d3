"""Pins of the oracle of the row-wise operators: hand-worked values, central differences of the
forward definitions for the gradients, brute force for the routing; planted mistakes must fail."""
import itertools

import numpy as np
import pytest

from oracle import rows as RO


def differences(f, x, at, h=1e-5):
    """Central differences of the scalar f at x for the elements `at`."""
    out = []
    for i in at:
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out.append((f(a) - f(b)) / (2 * h))
    return np.array(out)


def some(rng, shape, n=12):
    flat = rng.choice(int(np.prod(shape)), size=min(n, int(np.prod(shape))), replace=False)
    return [tuple(int(v) for v in np.unravel_index(i, shape)) for i in flat]


def test_rmsnorm_by_hand():
    h, rstd, y = RO.rmsnorm(np.array([[2.0, -1.0]]), np.array([[1.0, 5.0]]), np.array([1.0, 0.5]), 0.0)
    # h = (3, 4): mean square 12.5
    assert np.array_equal(h, [[3.0, 4.0]])
    assert np.allclose(rstd, 12.5 ** -0.5, rtol=1e-15)
    assert np.allclose(y, [[3.0 / 12.5 ** 0.5, 2.0 / 12.5 ** 0.5]], rtol=1e-15)
    assert np.array_equal(RO.e4m3_row_scale(np.array([[0.0, 0.0], [-896.0, 2.0]])), [1.0, 2.0])


@pytest.mark.parametrize("T,H", [(1, 8), (5, 16), (3, 40)])
def test_rmsnorm_bwd_against_differences(T, H):
    rng = np.random.default_rng(T * 100 + H)
    x, r, w, c, d = (rng.standard_normal(s) for s in ((T, H), (T, H), (H,), (T, H), (T, H)))
    f = lambda x, w: (RO.rmsnorm(x, r, w, 1e-3)[2] * c).sum() + (RO.rmsnorm(x, r, w, 1e-3)[0] * d).sum()  # noqa: E731
    h, rstd, _ = RO.rmsnorm(x, r, w, 1e-3)
    dx, dw = RO.rmsnorm_bwd(c, h, w, rstd, d)
    at = some(rng, (T, H))
    assert np.allclose(differences(lambda v: f(v, w), x, at), [dx[i] for i in at], rtol=1e-6, atol=1e-8)
    at = some(rng, (H,))
    assert np.allclose(differences(lambda v: f(x, v), w, at), [dw[i] for i in at], rtol=1e-6, atol=1e-8)
    wrong = dx + 1e-3
    assert not np.allclose(differences(lambda v: f(v, w), x, some(rng, (T, H))), wrong.flat[0], rtol=1e-6, atol=1e-8)


def brute_route(x, k, score, bias, n_group, topk_group, group_top):
    """The choice of one row by repeated search for the largest, in the words of the definition."""
    E = len(x)
    s = RO.scores(x[None], score)[0]
    key = [s[e] + (0.0 if bias is None else bias[e]) for e in range(E)]
    per = E // n_group
    gscore = [sum(sorted(key[g * per:(g + 1) * per], reverse=True)[:group_top]) for g in range(n_group)]
    groups = []
    for _ in range(topk_group):
        groups.append(max((g for g in range(n_group) if g not in groups), key=lambda g: (gscore[g], -g)))
    ids = []
    for _ in range(k):
        ids.append(max((e for e in range(E) if e // per in groups and e not in ids), key=lambda e: (key[e], -e)))
    return ids


@pytest.mark.parametrize("score,bias", list(itertools.product(["softmax", "sigmoid"], [False, True])))
@pytest.mark.parametrize("E,k,n_group,topk_group,group_top", [(6, 2, 1, 1, 1), (12, 3, 4, 2, 1), (12, 4, 3, 2, 2),
                                                             (8, 8, 2, 2, 2), (5, 5, 1, 1, 1), (4, 1, 4, 1, 2)])
def test_route_against_brute_force(score, bias, E, k, n_group, topk_group, group_top):
    rng = np.random.default_rng(E * k)
    x = rng.integers(-3, 4, (40, E)).astype(np.float64) / 2   # many ties
    b = rng.integers(-2, 3, E) / 4.0 if bias else None
    ids, gates, _ = RO.route(x, k, score, b, n_group, topk_group, group_top, True, 2.5)
    if score == "softmax" and not bias:
        want = [brute_route(r, k, score, b, n_group, topk_group, group_top) for r in x]
        # the order of equal logits is exact; sums of softmax scores of equal logits may round apart
        ok = [i == w for i, w in zip(ids.tolist(), want)]
        assert np.mean(ok) > 0.9
    else:
        assert ids.tolist() == [brute_route(r, k, score, b, n_group, topk_group, group_top) for r in x]
    assert np.allclose(gates.sum(1), 2.5, rtol=1e-12)


def test_route_order_of_nan_and_masked():
    x = np.array([[np.nan, -np.inf, 0.0, -np.inf], [-np.inf] * 4])
    ids, gates, _ = RO.route(x, 4, "sigmoid", None, renorm=False)
    assert ids.tolist() == [[2, 1, 3, 0], [0, 1, 2, 3]]
    assert gates[0, 1] == 0 and np.isnan(gates[0, 3]) and np.array_equal(gates[1], np.zeros(4))
    ids, gates, _ = RO.route(x[1:], 2, "softmax")
    assert ids.tolist() == [[0, 1]] and np.array_equal(gates, np.zeros((1, 2)))
    # a group that is not chosen gives nothing, whatever the chosen ones hold
    x = np.array([[5.0, -np.inf, 1.0, 0.0], [0.0, 0.0, 1.0, 0.5]])
    assert RO.route(x, 2, "softmax", None, 2, 1, 1)[0].tolist() == [[0, 1], [2, 3]]


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_route_bwd_against_differences(score, renorm):
    rng = np.random.default_rng(7)
    x, dg = rng.standard_normal((4, 9)), rng.standard_normal((4, 3))
    ids = RO.route(x, 3, score)[0]

    def f(x):
        s = np.take_along_axis(RO.scores(x, score), ids, 1)
        return (2.5 * (s / s.sum(1, keepdims=True) if renorm else s) * dg).sum()

    d = RO.route_bwd(x, ids, dg, score, renorm, 2.5)
    at = [(i, j) for i in range(4) for j in range(9)]
    assert np.allclose(differences(f, x, at), d.ravel(), rtol=1e-6, atol=1e-9)
    assert not np.allclose(differences(f, x, at), RO.route_bwd(x, ids, dg, score, not renorm, 2.5).ravel(), rtol=1e-6,
                           atol=1e-9)


def test_swiglu_against_differences():
    rng = np.random.default_rng(8)
    y, do = rng.standard_normal((3, 10)), rng.standard_normal((3, 5))
    assert np.allclose(RO.swiglu(np.array([[0.0, 2.0, 3.0, 4.0]])), [[0.0, 2 / (1 + np.exp(-2.0)) * 4]], rtol=1e-15)
    assert np.allclose(RO.swiglu(np.array([[1.0, 3.0]]), np.array([2.0])), RO.swiglu(np.array([[2.0, 6.0]])), rtol=1e-15)
    at = [(i, j) for i in range(3) for j in range(10)]
    got = differences(lambda v: (RO.swiglu(v) * do).sum(), y, at)
    assert np.allclose(got, RO.swiglu_bwd(y, do).ravel(), rtol=1e-6, atol=1e-9)
    assert not np.allclose(got, RO.swiglu_bwd(y[:, ::-1], do).ravel(), rtol=1e-6, atol=1e-9)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_softmax_of_an_infinite_logit_is_no_number(renorm):
    """exp(inf - inf) is NaN and stands in the sum under every score of the row."""
    x = np.array([[0.0, np.inf, 1.0], [0.0, 1.0, 2.0]])
    ids, gates, _ = RO.route(x, 2, "softmax", None, renorm=renorm)
    assert ids.tolist() == [[1, 2], [2, 1]]
    assert np.isnan(gates[0]).all() and np.isfinite(gates[1]).all()
    assert np.isnan(RO.scores(x[:1], "softmax")).all()
    # also where a bias keeps that expert out of the choice
    assert np.isnan(RO.route(x[:1], 1, "softmax", np.array([0.0, -np.inf, 0.0]), renorm=renorm)[1]).all()


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [False, True])))
def test_route_bwd_of_ids_that_come_twice_against_differences(score, renorm):
    rng = np.random.default_rng(9)
    x, dg = rng.standard_normal((3, 7)), rng.standard_normal((3, 4))
    ids = np.array([[1, 1, 4, 2], [5, 0, 3, 5], [6, 6, 6, 0]])

    def f(x):
        s = np.take_along_axis(RO.scores(x, score), ids, 1)
        return (2.5 * (s / s.sum(1, keepdims=True) if renorm else s) * dg).sum()

    at = [(i, j) for i in range(3) for j in range(7)]
    d = RO.route_bwd(x, ids, dg, score, renorm, 2.5)
    assert np.allclose(differences(f, x, at), d.ravel(), rtol=1e-6, atol=1e-9)
