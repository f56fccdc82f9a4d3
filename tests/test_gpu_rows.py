"""The row-wise operators on the GPU through the C ABI against the fp64 oracle: sizes from one row
to several per block, odd sizes, strides, every type, masked and non-finite rows, gradients against
the formula and against differences of the forward call.

Tolerances. U[type] is half a step of the output type relative to the value (8, 24 and 4 bits of
significand), e4m3 also half its smallest step, 2^-10. fp32 arithmetic adds F = 2^-24 per rounding:
a sum of n values in at most n/32 serial steps and a tree is off by at most F * (n/32 + 32) of the sum
of the magnitudes, which every tolerance below takes from the oracle's terms."""
import numpy as np
import pytest
import torch

import comm_overlapped_gemm_gb300 as tdx
from oracle import rows as RO

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24, "e4m3": 2.0 ** -4}
SMALLEST = {"bf16": 0.0, "fp32": 0.0, "e4m3": 2.0 ** -10}
F = 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
CODE = {"bf16": tdx.TDX_BF16, "fp32": tdx.TDX_FP32, "e4m3": tdx.TDX_FP8_E4M3}
PAD = -77.0


def dev(a, name):
    """fp64 values -> device tensor of the type, and the exact fp64 values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(TORCH[name])
    return t.cuda(), t.double().numpy()


def strided(rows, cols, name, ld=0, fill=PAD):
    """A device tensor of the shape inside rows of ld elements filled with a mark."""
    buf = torch.full((rows, ld or cols), fill, dtype=torch.float32, device="cuda").to(TORCH[name])
    return buf, buf[:, :cols]


def host(t):
    torch.cuda.synchronize()
    return t.float().cpu().numpy().astype(np.float64)


def near(got, want, tol, what=""):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), [(tuple(i), got[tuple(i)], want[tuple(i)]) for i in np.argwhere(bad)[:3]])


# ---------------------------------------------------------------------------------------- norm
def run_norm(x, r, w, dtype, out, rows_scaled=False, eps=1e-6, out_scale=1.0, pad=0, stream=None):
    T, H = x.shape
    ld = H + pad if pad else 0
    xs = strided(T, H, dtype, ld)[1]
    xs.copy_(x)
    rs = None
    if r is not None:
        rs = strided(T, H, dtype, ld)[1]
        rs.copy_(r)
    hb, h = strided(T, H, dtype, ld) if r is not None else (None, None)
    yb, y = strided(T, H, out, H + 2 * pad if pad else 0)
    scale = torch.full((T,), PAD, device="cuda") if rows_scaled else None
    rstd = torch.full((T,), PAD, device="cuda")
    o = tdx.make_norm_opts(out_dtype=CODE[out], eps=eps, out_scale=out_scale, ld_x=ld, ld_residual=ld, ld_h=ld,
                           ld_y=H + 2 * pad if pad else 0)
    tdx.check(tdx.tdx_rmsnorm(xs, rs, w, h, y, scale, rstd, T, H, CODE[dtype], o, stream))
    for buf in (hb, yb):
        if buf is not None and pad:
            assert bool((buf[:, H:].float() == torch.tensor(PAD).to(buf.dtype).float().item()).all())
    return h, y, scale, rstd


NORM_SIZES = [(1, 16), (1, 8192), (3, 48), (2, 1024), (17, 208), (5, 7168), (129, 2064), (2, 5136), (700, 144),
              (2, 16384), (1, 32768), (3, 33024)]


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dtype,out,mode", [("bf16", "bf16", ""), ("bf16", "e4m3", "rows"), ("bf16", "e4m3", "tensor"),
                                            ("bf16", "fp32", ""), ("fp32", "bf16", ""), ("fp32", "fp32", ""),
                                            ("fp32", "e4m3", "rows")])
@pytest.mark.parametrize("res,pad", [(True, 0), (False, 16), (True, 48)])
def test_rmsnorm(T, H, dtype, out, mode, res, pad):
    rng = np.random.default_rng(T * 7 + H)
    x, xv = dev(rng.standard_normal((T, H)), dtype)
    r, rv = dev(3 * rng.standard_normal((T, H)), dtype) if res else (None, None)
    w, wv = dev(1 + 0.2 * rng.standard_normal(H), dtype)
    scale = 0.0625
    h, y, rs, rstd = run_norm(x, r, w, dtype, out, mode == "rows", out_scale=scale, pad=pad)
    wh, wrstd, wy = RO.rmsnorm(xv, rv, wv, 1e-6)
    calc = F * (H / 32 + 64)
    near(host(rstd), wrstd, calc * wrstd, "rstd")
    if res:
        near(host(h), wh, U[dtype] * np.abs(wh) + F * np.abs(wh), "h")
    if out == "e4m3":
        ws = RO.e4m3_row_scale(wy) if mode == "rows" else np.full(T, scale)
        if mode == "rows":
            near(host(rs), ws, 2 * calc * ws, "row_scale")
        wy = np.clip(wy / ws[:, None], -448, 448)
    near(host(y), wy, (U[out] + 3 * calc) * np.abs(wy) * (1 + 2.0 ** -6) + SMALLEST[out], "y")


@pytest.mark.parametrize("H", [64, 4096, 33024])
def test_rmsnorm_rows_that_hold_nothing_or_too_much(H):
    x = torch.randn(6, H, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    ordinary = x.clone()
    x[1] = 0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 0
    x[4, 3] = -2.0 ** 60
    w = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    plain = run_norm(ordinary, None, w, "bf16", "bf16", eps=0.5)[1]
    _, y, _, rstd = run_norm(x, None, w, "bf16", "bf16", eps=0.5)
    assert torch.equal(y[[0, 5]], plain[[0, 5]])              # the others do not feel them
    assert int(torch.count_nonzero(y[1])) == 0 and rstd[1].item() == pytest.approx(0.5 ** -0.5, rel=1e-6)
    assert bool(torch.isnan(y[2]).all())
    # 1 / sqrt(inf) = 0: the row becomes 0, and 0 * inf = NaN where the infinity stood
    assert bool(torch.isnan(y[3, 7])) and int(torch.count_nonzero(torch.nan_to_num(y[3].float()))) == 0
    assert y[4, 3].item() == pytest.approx(-(H ** 0.5), rel=2 ** -8) and int(torch.count_nonzero(y[4])) == 1
    _, q, scale, _ = run_norm(x, None, w, "bf16", "e4m3", True, eps=0.5)
    q = q.float()
    assert scale[1].item() == 1.0 and int(torch.count_nonzero(q[1])) == 0
    assert bool(torch.isnan(q[2]).all()) and q[4, 3].item() == -448.0
    # a tensor scale that is too small saturates
    _, q, _, _ = run_norm(x[:1], None, w, "bf16", "e4m3", eps=0.5, out_scale=1e-4)
    big = x[0].float().abs() > 0.1
    assert bool((q[0].float()[big].abs() == 448.0).all())


@pytest.mark.parametrize("H", [128, 2048, 33024])
def test_rmsnorm_row_scales_of_tiny_rows(H):
    """Rows near the smallest float have a scale near it and ordinary codes."""
    rng = np.random.default_rng(H)
    x, xv = dev(rng.standard_normal((5, H)) * np.array([1e-20, 1e-33, 3e-37, 1e-38, 1.0])[:, None], "fp32")
    w, wv = dev(1 + 0.2 * rng.standard_normal(H), "fp32")
    _, q, scale, _ = run_norm(x, None, w, "fp32", "e4m3", True, eps=1.0)
    _, _, wy = RO.rmsnorm(xv, None, wv, 1.0)
    ws = RO.e4m3_row_scale(wy)
    calc = F * (H / 32 + 64)
    near(host(scale)[:4], ws[:4], 2 * calc * ws[:4] + 2.0 ** -149, "scale")
    # a scale that is itself subnormal has fewer bits: its relative rounding goes into the codes' bound
    coarse = (2.0 ** -149 / ws)[:, None]
    want = wy / ws[:, None]
    near(host(q), want, (U["e4m3"] + 3 * calc + coarse) * np.abs(want) * (1 + 2.0 ** -6) + SMALLEST["e4m3"], "codes")


def test_rmsnorm_in_place_on_another_stream_and_repeatable():
    g = torch.Generator().manual_seed(5)
    x, r = (torch.randn(33, 2048, generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.randn(2048, generator=g).bfloat16().cuda()
    h, y, _, rstd = run_norm(x, r, w, "bf16", "bf16")
    for target in ("x", "residual"):
        s = torch.cuda.Stream()
        a, b = x.clone(), r.clone()
        y2, rstd2 = torch.empty_like(y), torch.empty_like(rstd)
        torch.cuda.synchronize()
        tdx.check(tdx.tdx_rmsnorm(a, b, w, a if target == "x" else b, y2, None, rstd2, 33, 2048, 0, None, s))
        s.synchronize()
        assert torch.equal(a if target == "x" else b, h) and torch.equal(y2, y) and torch.equal(rstd2, rstd)
        assert torch.equal(b if target == "x" else a, r if target == "x" else x)


BWD_SIZES = [(1, 16), (1, 8192), (3, 48), (305, 208), (17, 7168), (700, 144), (1400, 1024), (2, 16384), (2, 32768)]


@pytest.mark.parametrize("T,H", BWD_SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("res,pad", [(True, 0), (False, 8), (True, 24)])
def test_rmsnorm_bwd(T, H, dtype, res, pad):
    rng = np.random.default_rng(T * 11 + H)
    h, hv = dev(3 * rng.standard_normal((T, H)), dtype)
    dy, dyv = dev(0.1 * rng.standard_normal((T, H)), dtype)
    dr, drv = dev(0.1 * rng.standard_normal((T, H)), dtype) if res else (None, None)
    w, wv = dev(1 + 0.2 * rng.standard_normal(H), dtype)
    rstd, rv = dev(1 / np.sqrt((hv * hv).mean(1) + 1e-6), "fp32")
    lds = [H + pad * i if pad else 0 for i in (1, 2, 3, 4)]
    bufs = [strided(T, H, dtype, ld) for ld in lds]
    for (_, v), src in zip(bufs, (dy, dr, h)):
        if src is not None:
            v.copy_(src)
    dxb, dx = bufs[3]
    dw = torch.full((H,), PAD, device="cuda")
    ws = torch.full((tdx.tdx_rmsnorm_bwd_workspace_size(T, H, CODE[dtype]),), 255, dtype=torch.uint8, device="cuda")
    o = tdx.make_norm_opts(ld_x=lds[0], ld_residual=lds[1], ld_h=lds[2], ld_y=lds[3])

    def call():
        tdx.check(tdx.tdx_rmsnorm_bwd(bufs[0][1], bufs[2][1], w, rstd, bufs[1][1] if res else None, dx, dw, ws, T, H,
                                      CODE[dtype], o))
    call()
    wdx, wdw = RO.rmsnorm_bwd(dyv, hv, wv, rv, drv)
    n, g = hv * rv[:, None], dyv * wv
    calc = F * (H / 32 + 64)
    mag = rv[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True)) + (np.abs(drv) if res else 0)
    near(host(dx), wdx, U[dtype] * np.abs(wdx) + calc * mag, "dx")
    near(host(dw), wdw, F * (T + 32) * np.abs(dyv * n).sum(0), "dw")
    if pad:
        assert bool((dxb[:, H:].float() == torch.tensor(PAD).to(dxb.dtype).float().item()).all())
    first = dw.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(dw, first)                     # the order of the sums is fixed


def test_rmsnorm_bwd_of_no_rows_and_in_place():
    dw = torch.full((64,), PAD, device="cuda")
    ws = torch.empty(tdx.tdx_rmsnorm_bwd_workspace_size(0, 64, 0), dtype=torch.uint8, device="cuda")
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    e = torch.empty(64, device="cuda", dtype=torch.bfloat16)
    rstd = torch.empty(1, device="cuda")
    tdx.check(tdx.tdx_rmsnorm_bwd(e, e, w, rstd, None, e, dw, ws, 0, 64, 0))
    assert int(torch.count_nonzero(dw)) == 0
    g = torch.Generator().manual_seed(6)
    h, dy, dr = (torch.randn(40, 1024, generator=g).cuda() for _ in range(3))
    w, rstd = torch.randn(1024, generator=g).cuda(), 1 / h.square().mean(-1).sqrt()
    ws = torch.empty(tdx.tdx_rmsnorm_bwd_workspace_size(40, 1024, 2), dtype=torch.uint8, device="cuda")
    outs = []
    for alias in (None, "dy", "dr"):
        a, b = dy.clone(), dr.clone()
        dx = {None: torch.empty_like(h), "dy": a, "dr": b}[alias]
        dw = torch.empty(1024, device="cuda")
        tdx.check(tdx.tdx_rmsnorm_bwd(a, h, w, rstd, b, dx, dw, ws, 40, 1024, 2))
        outs.append((dx, dw))
    assert all(torch.equal(outs[0][i], o[i]) for o in outs[1:] for i in (0, 1))


def test_rmsnorm_bwd_against_differences_of_the_forward_call():
    """A directional difference of the fp32 forward kernel: its rounding (F per value) over a step of
    2^-7 in a sum of 4096 products of size one leaves 4096 * F * 2^7 * 8 = 2.5e-1 at worst and its root
    in practice; the step's own error is of third order, 2^-14."""
    g = torch.Generator().manual_seed(9)
    T, H, eps = 4, 1024, 1e-3
    x, c, d = (torch.randn(T, H, generator=g).cuda() for _ in range(3))
    w = torch.randn(H, generator=g).cuda()

    def f(x, w):
        _, y, _, rstd = run_norm(x, None, w, "fp32", "fp32", eps=eps)
        return float((y.double() * c.double()).sum()), rstd

    step = 2.0 ** -7
    _, rstd = f(x, w)
    dx, dw = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = torch.empty(tdx.tdx_rmsnorm_bwd_workspace_size(T, H, 2), dtype=torch.uint8, device="cuda")
    tdx.check(tdx.tdx_rmsnorm_bwd(c, x, w, rstd, None, dx, dw, ws, T, H, 2))
    got = (f(x + step * d, w)[0] - f(x - step * d, w)[0]) / (2 * step)
    assert got == pytest.approx(float((dx.double() * d.double()).sum()), abs=2e-2)
    got = (f(x, w + step * d[0])[0] - f(x, w - step * d[0])[0]) / (2 * step)
    assert got == pytest.approx(float((dw.double() * d[0].double()).sum()), abs=2e-2)


# --------------------------------------------------------------------------------------- route
def run_route(logits, k, dtype="fp32", bias=None, counts=None, stream=None, pad=0, **kw):
    T, E = logits.shape
    x = strided(T, E, dtype, E + pad)[1]
    x.copy_(logits)
    idx = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    gates = torch.full((T, k), PAD, device="cuda")
    tdx.check(tdx.tdx_moe_route(x, bias, idx, gates, counts, T, E, k, CODE[dtype],
                                tdx.make_route_opts(ld_logits=E + pad if pad else 0, **kw), stream))
    torch.cuda.synchronize()
    return idx.cpu().numpy().astype(np.int64), gates.double().cpu().numpy()


def score_code(score):
    return tdx.TDX_SCORE_SIGMOID if score == "sigmoid" else tdx.TDX_SCORE_SOFTMAX


ROUTE_SIZES = [  # T, E, k, n_group, topk_group, group_top
    (1, 64, 8, 1, 1, 1), (700, 64, 8, 1, 1, 1), (33, 256, 8, 8, 4, 2), (1, 1, 1, 1, 1, 1), (50, 2, 2, 1, 1, 1),
    (65, 7, 3, 1, 1, 1), (300, 60, 4, 1, 1, 1), (100, 100, 6, 4, 2, 1), (64, 512, 16, 16, 4, 2), (40, 384, 12, 32, 5, 2),
    (9, 16, 16, 1, 1, 1), (31, 33, 5, 3, 2, 2), (20, 8, 2, 8, 3, 2), (2500, 128, 8, 1, 1, 1), (300, 160, 6, 8, 3, 1),
    (70, 32, 16, 2, 1, 2), (11, 500, 7, 1, 1, 1), (300, 48, 4, 2, 1, 1), (900, 96, 6, 4, 2, 2), (64, 240, 8, 2, 1, 2),
    (700, 240, 8, 10, 4, 2), (40, 480, 8, 2, 1, 2), (33, 500, 5, 5, 2, 2), (700, 120, 4, 5, 3, 1)]


@pytest.mark.parametrize("T,E,k,n_group,topk_group,group_top", ROUTE_SIZES)
@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype,renorm,pad", [("fp32", True, 0), ("fp32", False, 5), ("bf16", True, 3)])
def test_route(T, E, k, n_group, topk_group, group_top, score, bias, dtype, renorm, pad):
    rng = np.random.default_rng(E * 31 + k)
    x, xv = dev(1.5 * rng.standard_normal((T, E)), dtype)
    b, bv = dev(0.05 * rng.standard_normal(E), "fp32") if bias else (None, None)
    ids, gates = run_route(x, k, dtype, b, pad=pad, score=score_code(score), renorm=int(renorm), scale=2.5,
                           n_group=n_group, topk_group=topk_group, group_top=group_top)
    want, wg, margin = RO.route(xv, k, score, bv, n_group, topk_group, group_top, renorm, 2.5)
    # a key is off by some ten roundings of a number below 2; logits that are compared as such are exact
    clear = margin > 32 * F
    assert clear.mean() >= 0.9                         # how many rows the comparison covers
    assert np.array_equal(ids[clear], want[clear])
    assert ((ids >= 0) & (ids < E)).all() and all(len(set(r)) == k for r in ids.tolist())
    spread = np.abs(xv).max() * 2
    near(gates[clear], wg[clear], F * (E / 16 + 64 + spread) * wg[clear], "gates")


@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("T,E,k,n_group,topk_group,group_top", [s for s in ROUTE_SIZES if s[0] > 8])
def test_route_ties_go_to_the_lowest_index(T, E, k, n_group, topk_group, group_top, score, bias):
    """A few values only, so that most keys and groups tie: equal inputs give equal keys, and distinct
    ones lie apart by far more than the kernel's rounding."""
    rng = np.random.default_rng(E + k)
    # no two different pairs of these have scores of one sum (as 1/2 + 1/2 = s(x) + s(-x) would), and for
    # sums of two the bias is the same for all
    x, xv = dev(np.array([-1.0, -0.25, 0.0, 0.5, 1.25])[rng.integers(0, 5, (T, E))], "bf16")
    b, bv = dev((rng.integers(-1, 2, E) if group_top == 1 else np.ones(E)) / 64.0, "fp32") if bias else (None, None)
    ids, _ = run_route(x, k, "bf16", b, score=score_code(score), n_group=n_group, topk_group=topk_group,
                       group_top=group_top)
    # the oracle's keys rounded to 12 digits, so that sums of equal terms tie there as well
    s = RO.scores(xv, score)
    key = xv if score == "softmax" else np.round(s + (0 if bv is None else bv), 12)
    gkey = np.round(np.exp(xv - xv.max(1, keepdims=True)), 12) if score == "softmax" and group_top == 2 else key
    if n_group > 1:
        per = E // n_group
        best = np.round(-np.sort(-gkey.reshape(T, n_group, per), axis=2)[:, :, :group_top].sum(2), 11)
        keep = np.argsort(-best, axis=1, kind="stable")[:, :topk_group]
        on = np.zeros((T, n_group), bool)
        np.put_along_axis(on, keep, True, 1)
        key = np.where(np.repeat(on, per, 1), key, -np.inf)
    assert np.array_equal(ids, np.argsort(-key, axis=1, kind="stable")[:, :k])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,n_group", [(64, 8, 1), (12, 4, 3), (256, 8, 8), (33, 5, 3)])
def test_route_masked_and_non_finite_logits(score, E, k, n_group):
    kw = dict(n_group=n_group, topk_group=max(1, n_group - 1), group_top=1, score=score_code(score))
    rng = np.random.default_rng(E)
    x = rng.standard_normal((8, E)).astype(np.float32)
    x[1] = -np.inf                                     # a row whose mask leaves nothing
    x[2, 1:] = -np.inf                                 # one expert left
    x[3] = np.finfo(np.float32).min                    # masked with the type's lowest value
    x[4, 3] = np.nan
    x[5] = np.nan
    x[6, :E // 2] = -np.inf
    x[7] = 0.0
    x[7, 1::2] = -0.0                                  # the zeros are equal
    for renorm in (0, 1):
        ids, gates = run_route(torch.from_numpy(x), k, renorm=renorm, **kw)
        want, wg, _ = RO.route(x.astype(np.float64), k, score, None, n_group, kw["topk_group"], 1, bool(renorm), 1.0)
        assert np.array_equal(ids, want)
        rows = [0, 1, 2, 3, 6, 7]
        near(gates[rows], wg[rows], F * (E / 16 + 80) * np.abs(wg[rows]), "gates")
        if score == "softmax":
            assert np.isnan(gates[[4, 5]]).all()
        else:
            assert np.isnan(gates[5]).all()


@pytest.mark.parametrize("E,k,n_group,topk_group,group_top,score", [(64, 8, 1, 1, 1, "softmax"), (256, 8, 8, 4, 2, "sigmoid"),
                                                                  (500, 16, 4, 2, 2, "sigmoid"), (30, 2, 3, 2, 1, "softmax")])
def test_route_of_more_tokens_than_the_warps_take_at_once(E, k, n_group, topk_group, group_top, score):
    T = 40003 if E <= 64 else 20011
    rng = np.random.default_rng(E)
    x, xv = dev(1.5 * rng.standard_normal((T, E)), "fp32")
    b, bv = dev(0.05 * rng.standard_normal(E), "fp32") if score == "sigmoid" else (None, None)
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    ids, gates = run_route(x, k, "fp32", b, counts, score=score_code(score), n_group=n_group, topk_group=topk_group,
                           group_top=group_top)
    want, wg, margin = RO.route(xv, k, score, bv, n_group, topk_group, group_top)
    clear = margin > 32 * F
    assert clear.mean() >= 0.9
    assert np.array_equal(ids[clear], want[clear])
    near(gates[clear], wg[clear], F * (E / 16 + 64 + np.abs(xv).max() * 2) * wg[clear], "gates")
    assert np.array_equal(counts.cpu().numpy(), np.bincount(ids.ravel(), minlength=E))
    dg, dgv = dev(rng.standard_normal((T, k)), "fp32")
    out = torch.full((T, E), PAD, device="cuda")
    tdx.check(tdx.tdx_moe_route_bwd(x, torch.from_numpy(ids.astype(np.int32)).cuda(), dg, out, T, E, k, 2,
                                    tdx.make_route_opts(score=score_code(score), renorm=0)))
    wd = RO.route_bwd(xv, ids, dgv, score, False, 1.0)
    mag = 2 * RO.scores(xv, score) * np.abs(dgv).sum(1, keepdims=True)
    near(host(out), wd, U["fp32"] * np.abs(wd) + F * (E / 16 + 64 + 4 * np.abs(xv).max()) * mag, "dlogits")


@pytest.mark.parametrize("E,n_group", [(64, 1), (256, 8), (512, 16), (100, 1), (24, 1)])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
def test_route_keys_that_differ_in_their_last_bits(E, n_group, score, bias):
    """Keys a few steps of fp32 apart, which the leading bits do not tell from one another: the order is
    that of the definition's fp32 keys, computed here with the device's own exp and quotient."""
    T, k = 700, 8
    g = torch.Generator().manual_seed(E)
    base = torch.randn(T, 1, generator=g)
    x = (base + 2.0 ** -22 * torch.randint(-6, 7, (T, E), generator=g)).cuda()
    x[::3] += (torch.rand(x[::3].shape, generator=g) < 0.5).cuda() * 1.0       # two clusters of keys
    b = (2.0 ** -20 * torch.randint(-2, 3, (E,), generator=g)).cuda() if bias else None
    ids, _ = run_route(x, k, "fp32", b, score=score_code(score), n_group=n_group, topk_group=max(1, n_group // 2),
                       group_top=1)
    key = x + 0.0
    if score == "sigmoid":
        key = 1.0 / (1.0 + torch.exp(-x))
        if bias:
            key = key + b
    key = key.cpu().numpy().astype(np.float64)
    if n_group > 1:
        per = E // n_group
        best = key.reshape(T, n_group, per).max(2)
        keep = np.argsort(-best, axis=1, kind="stable")[:, :n_group // 2]
        on = np.zeros((T, n_group), bool)
        np.put_along_axis(on, keep, True, 1)
        key = np.where(np.repeat(on, per, 1), key, -np.inf)
    assert np.array_equal(ids, np.argsort(-key, axis=1, kind="stable")[:, :k])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,n_group,topk_group", [(64, 8, 1, 1), (40, 4, 1, 1), (256, 8, 8, 4), (48, 6, 2, 1), (500, 16, 5, 3)])
def test_route_bias_of_infinity(score, E, k, n_group, topk_group):
    """A bias of -inf leaves an expert out while others are there, one of +inf puts it in front; neither
    is seen in the gates."""
    T = 300
    rng = np.random.default_rng(E)
    x, xv = dev(rng.standard_normal((T, E)), "fp32")
    for value, some_of in (([-np.inf], 3), ([np.inf], 1), ([np.inf, -np.inf], 2)):
        b = 0.05 * rng.standard_normal(E)
        at = rng.choice(E, size=some_of * len(value), replace=False)
        b[at] = np.repeat(value, some_of)
        b, bv = dev(b, "fp32")
        ids, gates = run_route(x, k, "fp32", b, score=score_code(score), n_group=n_group, topk_group=topk_group)
        want, wg, margin = RO.route(xv, k, score, bv, n_group, topk_group)
        clear = margin > 32 * F
        assert clear.mean() >= 0.9 and np.array_equal(ids[clear], want[clear])
        assert np.isfinite(gates).all()
        near(gates[clear], wg[clear], F * (E / 16 + 64 + np.abs(xv).max() * 2) * wg[clear], "gates")


def test_route_counts_are_added_and_streams_hold():
    x = torch.randn(1000, 48, generator=torch.Generator().manual_seed(2)).cuda()
    counts = torch.arange(48, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ids, _ = run_route(x, 4, counts=counts, stream=s)
    s.synchronize()
    assert np.array_equal(counts.cpu().numpy(), np.bincount(ids.ravel(), minlength=48) + np.arange(48))
    again, _ = run_route(x, 4)
    assert np.array_equal(ids, again)


@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (700, 64, 8), (33, 256, 8), (1, 1, 1), (50, 2, 2), (65, 7, 3), (64, 512, 16),
                                   (9, 16, 16), (40, 33, 5), (2500, 128, 8), (11, 500, 7)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype,renorm,pad", [("fp32", True, 0), ("fp32", False, 5), ("bf16", False, 0), ("bf16", True, 3)])
def test_route_bwd(T, E, k, score, dtype, renorm, pad):
    rng = np.random.default_rng(E * 13 + k)
    x, xv = dev(1.5 * rng.standard_normal((T, E)), dtype)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    dg, dgv = dev(rng.standard_normal((T, k)), "fp32")
    xs = strided(T, E, dtype, E + pad)[1]
    xs.copy_(x)
    ob, out = strided(T, E, dtype, E + pad)
    o = tdx.make_route_opts(score=score_code(score), renorm=int(renorm), scale=2.5, ld_logits=E + pad if pad else 0)
    tdx.check(tdx.tdx_moe_route_bwd(xs, torch.from_numpy(ids.astype(np.int32)).cuda(), dg, out, T, E, k, CODE[dtype], o))
    want = RO.route_bwd(xv, ids, dgv, score, renorm, 2.5)
    # every term is a score times what the row's gates receive; renormalised scores divide by their sum
    s = RO.scores(xv, score)
    sel = np.take_along_axis(s, ids, 1).sum(1, keepdims=True)
    mag = 2.5 * s * np.abs(dgv).sum(1, keepdims=True) * (2 / np.minimum(sel, 1) if renorm else 2)
    tol = F * (E / 16 + 64 + 4 * np.abs(xv).max()) * mag
    if renorm or score == "sigmoid":                   # nothing but the choice receives anything
        on = np.zeros((T, E), bool)
        np.put_along_axis(on, ids, True, 1)
        tol = np.where(on, tol, 0)
    near(host(out), want, U[dtype] * np.abs(want) + tol, "dlogits")
    if pad:
        assert bool((ob[:, E:].float() == torch.tensor(PAD).to(ob.dtype).float().item()).all())


def test_route_bwd_of_masked_rows_and_bad_ids():
    x = torch.zeros(3, 40, device="cuda")
    x[0] = float("-inf")
    x[1, 2:] = float("-inf")
    ids = torch.tensor([[0, 1], [0, 1], [7, 99]], dtype=torch.int32, device="cuda")
    ids[2, 1] = 1 << 30
    dg = torch.ones(3, 2, device="cuda")
    for score in (0, 1):
        for renorm in (0, 1):
            out = torch.full((3, 40), PAD, device="cuda")
            tdx.check(tdx.tdx_moe_route_bwd(x, ids, dg, out, 3, 40, 2, 2, tdx.make_route_opts(score=score, renorm=renorm)))
            torch.cuda.synchronize()
            assert bool(torch.isfinite(out).all())
            assert int(torch.count_nonzero(out[0])) == 0
    ids[2, 1] = -3
    tdx.check(tdx.tdx_moe_route_bwd(x, ids, dg, out, 3, 40, 2, 2, tdx.make_route_opts(score=1, renorm=0)))
    assert out[2].nonzero().tolist() == [[7]] and out[2, 7].item() == pytest.approx(0.25, rel=1e-6)


def test_route_bwd_against_differences_of_the_forward_call():
    """fp32 gates of size one and a step of 2^-6: rounding leaves a few F * 2^6, the step's third-order
    error 2^-12 times derivatives below one, over 6 x 4 gates weighted by about one."""
    g = torch.Generator().manual_seed(4)
    x = 3 * torch.randn(6, 40, generator=g)
    d, dg = torch.randn(6, 40, generator=g), torch.randn(6, 4, generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (0, 1):
            kw = dict(score=score_code(score), renorm=renorm)
            ids, _ = run_route(x, 4, **kw)

            def f(v):
                i, gates = run_route(v, 4, **kw)
                table = np.zeros((6, 40))
                np.put_along_axis(table, i, gates, 1)
                assert np.array_equal(np.sort(i), np.sort(ids))
                return (np.take_along_axis(table, ids, 1) * dg.double().numpy()).sum()

            out = torch.empty(6, 40, device="cuda")
            tdx.check(tdx.tdx_moe_route_bwd(x.cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(), dg.cuda(), out, 6,
                                            40, 4, 2, tdx.make_route_opts(**kw)))
            h = 2.0 ** -10
            got = (f(x + h * d) - f(x - h * d)) / (2 * h)
            assert got == pytest.approx(float((out.double().cpu() * d.double()).sum()), abs=5e-3)


# -------------------------------------------------------------------------------------- swiglu
SWIGLU_SIZES = [(1, 16), (8, 2048), (3, 48), (40, 208), (300, 1024), (7, 3584), (1000, 16), (2, 40000), (5000, 64)]


@pytest.mark.parametrize("R,I", SWIGLU_SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "e4m3"), ("bf16", "fp32"), ("fp32", "bf16"),
                                       ("fp32", "fp32"), ("fp32", "e4m3")])
@pytest.mark.parametrize("scaled,pad", [("", 0), ("rows", 16), ("dest", 0), ("dest", 32)])
def test_swiglu(R, I, dtype, out, scaled, pad):
    rng = np.random.default_rng(R + I)
    y, yv = dev(2 * rng.standard_normal((R, 2 * I)), dtype)
    ys = strided(R, 2 * I, dtype, 2 * I + pad)[1]
    ys.copy_(y)
    ob, o = strided(R, I, out, I + 2 * pad)
    rs, dest, c, topk = None, None, None, 0
    if scaled == "rows":
        rs, c = dev(0.5 + rng.random(R), "fp32")
    elif scaled == "dest":
        topk = next(k for k in (8, 5, 4, 3, 2, 1) if R % k == 0)
        rs, rv = dev(0.5 + rng.random(R // topk), "fp32")
        perm = rng.permutation(R)
        dest = torch.from_numpy(perm.astype(np.int32)).cuda()
        c = np.empty(R)
        c[perm] = np.repeat(rv, topk)
    opts = tdx.make_act_opts(out_dtype=CODE[out], out_scale=0.125, topk=topk, ld_y=2 * I + pad if pad else 0,
                             ld_out=I + 2 * pad if pad else 0)
    tdx.check(tdx.tdx_swiglu(ys, o, rs, dest, R, I, CODE[dtype], opts))
    want = RO.swiglu(yv, c)
    if out == "e4m3":
        want = np.clip(want / 0.125, -448, 448)
    g = np.abs(yv[:, :I] * (1 if c is None else c[:, None]))
    near(host(o), want, (U[out] + F * (24 + 4 * g)) * np.abs(want) * (1 + 2.0 ** -6) + SMALLEST[out], "out")
    if pad:
        assert bool((ob[:, I:].float() == torch.tensor(PAD).to(ob.dtype).float().item()).all())


@pytest.mark.parametrize("topk", [0, 3])
def test_swiglu_of_more_rows_than_the_blocks_take_at_once(topk):
    R, I = 4101, 2080
    rng = np.random.default_rng(topk)
    y, yv = dev(2 * rng.standard_normal((R, 2 * I)), "bf16")
    rs = dest = c = None
    if topk:
        rs, rv = dev(0.5 + rng.random(R // topk), "fp32")
        perm = rng.permutation(R)
        dest = torch.from_numpy(perm.astype(np.int32)).cuda()
        c = np.empty(R)
        c[perm] = np.repeat(rv, topk)
    out = torch.full((R, I), PAD, dtype=torch.bfloat16, device="cuda")
    tdx.check(tdx.tdx_swiglu(y, out, rs, dest, R, I, 0, tdx.make_act_opts(topk=topk)))
    want = RO.swiglu(yv, c)
    g = np.abs(yv[:, :I] * (1 if c is None else c[:, None]))
    near(host(out), want, (U["bf16"] + F * (24 + 4 * g)) * np.abs(want) * (1 + 2.0 ** -6), "out")
    if not topk:
        do, dov = dev(0.1 * rng.standard_normal((R, I)), "bf16")
        dy = torch.full_like(y, PAD)
        tdx.check(tdx.tdx_swiglu_bwd(y, do, dy, R, I, 0))
        want = RO.swiglu_bwd(yv, dov)
        s, u = RO.scores(yv[:, :I], "sigmoid"), np.abs(yv[:, I:])
        mag = np.concatenate([np.abs(dov) * u * s * (1 + g), np.abs(want[:, I:])], 1)
        near(host(dy), want, U["bf16"] * np.abs(want) + F * (24 + 4 * np.concatenate([g, g], 1)) * mag * (1 + 2.0 ** -6))


def test_swiglu_extremes_and_rows_that_dest_skips():
    y = torch.zeros(4, 32, device="cuda")
    y[:, 16:] = 2.0
    y[0, :6] = torch.tensor([-1000.0, 1000.0, -87.0, float("inf"), float("nan"), -2e38])
    out = torch.full((4, 16), PAD, device="cuda")
    o = tdx.make_act_opts(out_dtype=tdx.TDX_FP32)
    tdx.check(tdx.tdx_swiglu(y, out, None, None, 4, 16, 2, o))
    v = out[0].tolist()
    assert v[0] == 0.0 and v[1] == 2000.0 and abs(v[2]) < 1e-34 and v[3] == float("inf") and np.isnan(v[4]) and v[5] == 0.0
    assert int(torch.count_nonzero(out[1:])) == 0
    out.fill_(PAD)
    dest = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    o = tdx.make_act_opts(out_dtype=tdx.TDX_FP32, topk=2)
    tdx.check(tdx.tdx_swiglu(y, out, torch.tensor([1.0, 3.0], device="cuda"), dest, 4, 16, 2, o))
    assert bool((out[[1, 3]] == PAD).all()) and int(torch.count_nonzero(out[2])) == 0
    assert out[0, 1].item() == 18000.0
    # a row whose halves are masked to the lowest value
    y[1] = torch.finfo(torch.bfloat16).min
    yb, ob = y.bfloat16(), torch.empty(4, 16, device="cuda", dtype=torch.bfloat16)
    tdx.check(tdx.tdx_swiglu(yb, ob, None, None, 4, 16, 0))
    assert int(torch.count_nonzero(ob[1])) == 0


@pytest.mark.parametrize("R,I", SWIGLU_SIZES)
@pytest.mark.parametrize("dtype,pad,alias", [("bf16", 0, False), ("bf16", 24, True), ("fp32", 0, True), ("fp32", 4, False)])
def test_swiglu_bwd(R, I, dtype, pad, alias):
    rng = np.random.default_rng(R * 3 + I)
    y, yv = dev(2 * rng.standard_normal((R, 2 * I)), dtype)
    do, dov = dev(0.1 * rng.standard_normal((R, I)), dtype)
    ys = strided(R, 2 * I, dtype, 2 * I + pad)[1]
    ys.copy_(y)
    dos = strided(R, I, dtype, I + 3 * pad)[1]
    dos.copy_(do)
    ob, out = strided(R, 2 * I, dtype, 2 * I + pad)
    o = tdx.make_act_opts(ld_y=2 * I + pad if pad else 0, ld_out=I + 3 * pad if pad else 0)
    tdx.check(tdx.tdx_swiglu_bwd(ys, dos, ys if alias else out, R, I, CODE[dtype], o))
    want = RO.swiglu_bwd(yv, dov)
    g, u = np.abs(yv[:, :I]), np.abs(yv[:, I:])
    s = RO.scores(yv[:, :I], "sigmoid")
    mag = np.concatenate([np.abs(dov) * u * s * (1 + g), np.abs(want[:, I:])], 1)
    calc = F * (24 + 4 * np.concatenate([g, g], 1))
    near(host(ys if alias else out), want, U[dtype] * np.abs(want) + calc * mag * (1 + 2.0 ** -6), "dy")
    if pad and not alias:
        assert bool((ob[:, 2 * I:].float() == torch.tensor(PAD).to(ob.dtype).float().item()).all())


def test_swiglu_bwd_against_differences_of_the_forward_call():
    """fp32 outputs of size one over 8 x 64 elements, a step of 2^-7: the step's third-order error is
    below 2^-14 per element, rounding below F * 2^7."""
    g = torch.Generator().manual_seed(11)
    y, d, do = torch.randn(8, 128, generator=g), torch.randn(8, 128, generator=g), torch.randn(8, 64, generator=g)

    def f(v):
        out = torch.empty(8, 64, device="cuda")
        tdx.check(tdx.tdx_swiglu(v.cuda(), out, None, None, 8, 64, 2, tdx.make_act_opts(out_dtype=tdx.TDX_FP32)))
        return float((out.double().cpu() * do.double()).sum())

    dy = torch.empty(8, 128, device="cuda")
    tdx.check(tdx.tdx_swiglu_bwd(y.cuda(), do.cuda(), dy, 8, 64, 2))
    h = 2.0 ** -7
    got = (f(y + h * d) - f(y - h * d)) / (2 * h)
    assert got == pytest.approx(float((dy.double().cpu() * d.double()).sum()), abs=2e-2)


def test_tensors_beyond_2_to_the_31_elements():
    """Row offsets past 32 bits: the last rows of a tall tensor are those of a short one."""
    H, T = 8192, 270000                                # 2.2e9 elements
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, H, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    x[-5:] = tail
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y, ys = torch.empty_like(x), torch.empty_like(tail)
    tdx.check(tdx.tdx_rmsnorm(x, None, w, None, y, None, None, T, H, 0))
    tdx.check(tdx.tdx_rmsnorm(tail, None, w, None, ys, None, None, 5, H, 0))
    assert torch.allclose(y[-5:].float(), ys.float(), rtol=2.0 ** -7, atol=0)
    out, outs = (torch.empty(n, H // 2, dtype=torch.bfloat16, device="cuda") for n in (T, 5))
    tdx.check(tdx.tdx_swiglu(x, out, None, None, T, H // 2, 0))
    tdx.check(tdx.tdx_swiglu(tail, outs, None, None, 5, H // 2, 0))
    assert torch.allclose(out[-5:].float(), outs.float(), rtol=2.0 ** -7, atol=0)
