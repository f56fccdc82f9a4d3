"""The row-wise operators at the ends of fp32's range, and on the paths that need many rows: finite
rows whose products overflow, infinities, NaN weights, scores near the smallest float, several rows per
block, several choices per lane, offsets past 32 bits. Tolerances as in test_gpu_rows.py."""
import numpy as np
import pytest
import torch

import comm_overlapped_gemm_gb300 as tdx
from oracle import rows as RO
from test_gpu_rows import CODE, F, PAD, SMALLEST, TORCH, U, dev, host, near, run_norm, run_route, score_code, strided

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("T,H", [(6, 64), (200, 1040), (6, 4096), (200, 4096), (6, 33024)])
@pytest.mark.parametrize("out,mode", [("bf16", ""), ("e4m3", "tensor"), ("e4m3", "rows")])
@pytest.mark.parametrize("res", [False, True])
def test_rmsnorm_of_the_lowest_values_is_zero(T, H, out, mode, res):
    """A row masked to the type's lowest value: its sum of squares is infinite, 1 / root is 0, and
    so is every h * rstd * weight, whatever the weight."""
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(H)).bfloat16().cuda()
    x[1] = torch.finfo(torch.bfloat16).min
    x[4, 3:7] = torch.finfo(torch.bfloat16).max
    w = torch.full((H,), 1.5, device="cuda", dtype=torch.bfloat16)
    r = torch.zeros_like(x) if res else None
    _, y, scale, rstd = run_norm(x, r, w, "bf16", out, mode == "rows")
    for t in (1, 4):
        assert rstd[t].item() == 0.0
        assert int(torch.count_nonzero(y[t].float())) == 0
        if mode == "rows":
            assert scale[t].item() == 1.0
    assert bool(torch.isfinite(y.float()).all())


@pytest.mark.parametrize("T,H", [(4, 64), (200, 1040), (4, 4096), (4, 33024)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("out,mode", [("fp32", ""), ("bf16", ""), ("e4m3", "tensor"), ("e4m3", "rows")])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("size", [1e30, 2.5e37])
def test_rmsnorm_of_large_weights(T, H, dtype, out, mode, res, size):
    """h * weight is beyond fp32 (1e12 * 1e30), y = h * rstd * weight is not: up to 10 sizes."""
    rng = np.random.default_rng(H)
    x, xv = dev(1e12 * rng.standard_normal((T, H)), dtype)
    r, rv = dev(1e12 * rng.standard_normal((T, H)), dtype) if res else (None, None)
    w, wv = dev(size * (1 + 0.2 * rng.standard_normal(H)), dtype)
    scale = 2.0 ** 100
    _, y, rs, rstd = run_norm(x, r, w, dtype, out, mode == "rows", out_scale=scale)
    _, wrstd, wy = RO.rmsnorm(xv, rv, wv, 1e-6)
    calc = F * (H / 32 + 64)
    near(host(rstd), wrstd, calc * wrstd, "rstd")
    if out == "e4m3":
        ws = RO.e4m3_row_scale(wy) if mode == "rows" else np.full(T, scale)
        if mode == "rows":
            near(host(rs), ws, 2 * calc * ws, "row_scale")
        wy = np.clip(wy / ws[:, None], -448, 448)
    near(host(y), wy, (U[out] + 3 * calc) * np.abs(wy) * (1 + 2.0 ** -6) + SMALLEST[out], "y")


@pytest.mark.parametrize("H", [64, 4096, 33024])
def test_rmsnorm_tensor_scale_near_the_smallest(H):
    """1 / (root * scale) is beyond fp32 and zeros stay zeros; what is not zero saturates."""
    x = torch.zeros(2, H, device="cuda")
    x[1, 5] = -1e-10
    w = torch.ones(H, device="cuda")
    _, y, _, _ = run_norm(x, None, w, "fp32", "e4m3", eps=1e-12, out_scale=1e-36)
    assert int(torch.count_nonzero(y.float()[0])) == 0
    assert y[1, 5].float().item() == -448.0 and int(torch.count_nonzero(y.float()[1])) == 1


@pytest.mark.parametrize("T,H", [(3, 128), (3, 2048), (200, 2048), (3, 33024)])
@pytest.mark.parametrize("dtype,res", [("bf16", False), ("bf16", True), ("fp32", False)])
def test_rmsnorm_row_scale_of_a_weight_that_is_no_number(T, H, dtype, res):
    """max|y| of every row is NaN: the scale is 1, and the other columns are y itself."""
    g = torch.Generator().manual_seed(H)
    x, r = (torch.randn(T, H, generator=g).to(TORCH[dtype]).cuda() for _ in range(2))
    w = torch.ones(H, dtype=TORCH[dtype], device="cuda")
    w[H - 3] = float("nan")
    _, q, scale, _ = run_norm(x, r if res else None, w, dtype, "e4m3", True)
    assert bool((scale == 1.0).all())
    assert bool(torch.isnan(q[:, H - 3].float()).all())
    _, one, _, _ = run_norm(x, r if res else None, torch.ones_like(w), dtype, "e4m3", out_scale=1.0)
    keep = torch.arange(H, device="cuda") != H - 3
    assert torch.equal(q.float()[:, keep], one.float()[:, keep])


# --------------------------------------------------------------------------------------- route
@pytest.mark.parametrize("T,E,k,n_group", [(5, 64, 8, 1), (900, 64, 8, 1), (900, 33, 12, 1), (5, 256, 8, 8), (900, 256, 8, 8),
                                           (40, 500, 5, 5)])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("bias", [False, True])
def test_route_softmax_of_an_infinite_logit_is_no_number(T, E, k, n_group, renorm, bias):
    """exp(inf - inf) is NaN and stands in every sum: all gates of the row are NaN, the other rows' are not."""
    g = torch.Generator().manual_seed(E)
    x = torch.randn(T, E, generator=g)
    x[1, 7] = float("inf")
    x[3, 7] = x[3, 2] = float("inf")
    x[4] = -float("inf")
    b = 0.01 * torch.randn(E, generator=g).cuda() if bias else None
    ids, gates = run_route(x, k, bias=b, renorm=renorm, n_group=n_group, topk_group=max(1, n_group - 1))
    assert np.isnan(gates[[1, 3]]).all()
    rest = np.delete(np.arange(T), [1, 3])
    assert np.isfinite(gates[rest]).all() and (gates[4] == 0).all()
    if not bias:
        assert (ids[1, 0], ids[3, 0], ids[3, 1]) == (7, 2, 7)


@pytest.mark.parametrize("T,E,k", [(40, 24, 2), (9, 24, 4), (40, 64, 8), (40, 256, 8), (40, 500, 16), (9, 64, 1)])
@pytest.mark.parametrize("scale", [1.0, 40.0])
def test_route_bwd_of_scores_near_the_smallest_float(T, E, k, scale):
    """Renormalised sigmoid gates of logits between -88.5 and -86 (scores from 3.7e-39 up): the gates are of
    size one, and so are their gradients. A score is off by a rounding of exp and of the quotient, and
    below 2^-126 by half of 2^-149, 2^-22 of the smallest: 8 F in all, 16 F in a quotient of two."""
    rng = np.random.default_rng(E + k)
    x, xv = dev(rng.uniform(-88.5, -86.0, (T, E)), "fp32")
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    if k > 1:
        x[1::2], xv[1::2] = -88.0, -88.0
        x[1::2, 1::2], xv[1::2, 1::2] = -88.0 - 2.0 ** -3, -88.0 - 2.0 ** -3
    dg, dgv = dev(rng.standard_normal((T, k)), "fp32")
    out = torch.full((T, E), PAD, device="cuda")
    o = tdx.make_route_opts(score=tdx.TDX_SCORE_SIGMOID, renorm=1, scale=scale)
    tdx.check(tdx.tdx_moe_route_bwd(x, torch.from_numpy(ids.astype(np.int32)).cuda(), dg, out, T, E, k, 2, o))
    want = RO.route_bwd(xv, ids, dgv, "sigmoid", True, scale)
    sel = np.take_along_axis(RO.scores(xv, "sigmoid"), ids, 1)
    mag = scale * (sel / sel.sum(1, keepdims=True)) * (np.abs(dgv) + np.abs(dgv).sum(1, keepdims=True))
    tol = np.zeros((T, E))
    np.put_along_axis(tol, ids, F * (64 + 4 * k) * mag, 1)
    near(host(out), want, U["fp32"] * np.abs(want) + tol, "dlogits")


# -------------------------------------------------------------------------------------- swiglu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scaled", ["", "rows", "dest"])
def test_swiglu_to_e4m3_of_lowest_values_is_zero(dtype, scaled):
    """g * sigmoid(g) is 0, and so is its product with any finite u, whatever the scale it is stored with."""
    R, I = 6, 32
    t = torch.finfo(TORCH[dtype])
    y = torch.zeros(R, 2 * I, dtype=TORCH[dtype], device="cuda")
    y[0] = t.min
    y[1, I:] = t.max                          # g = 0
    y[2, :I], y[2, I:] = -100.0, t.min
    y[3, :I], y[3, I:] = 1.0, t.max           # infinite over the scale: saturates
    y[4, :I], y[4, I:] = -1.0, 3e37
    y[5, :I], y[5, I:] = 2.0, 0.25
    ones = torch.ones(R, device="cuda")
    dest = torch.arange(R, dtype=torch.int32, device="cuda") if scaled == "dest" else None
    out = torch.full((R, I), PAD, device="cuda").to(torch.float8_e4m3fn)
    o = tdx.make_act_opts(out_dtype=tdx.TDX_FP8_E4M3, out_scale=0.0625, topk=1 if scaled == "dest" else 0)
    tdx.check(tdx.tdx_swiglu(y, out, ones if scaled else None, dest, R, I, CODE[dtype], o))
    v = out.float().cpu()
    assert int(torch.count_nonzero(v[:3])) == 0
    assert bool((v[3] == 448).all()) and bool((v[4] == -448).all())
    want = 2.0 / (1.0 + np.exp(-2.0)) * 0.25 / 0.0625
    assert bool(((v[5] - want).abs() <= 2.0 ** -4 * want).all())


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_swiglu_where_the_sigmoid_is_near_the_smallest_float(dtype, out):
    """exp(-g) between 2^126 and fp32's largest: the value is small, not zero. exp of an argument of 89 is
    off by at most 106 steps of 2^-23 in the approximate form."""
    g = np.linspace(-88.5, -86.0, 64)
    y, yv = dev(np.concatenate([g, np.full(64, 2.0 ** 100)])[None].repeat(3, 0), dtype)
    o = torch.full((3, 64), PAD, dtype=TORCH[out], device="cuda")
    tdx.check(tdx.tdx_swiglu(y, o, None, None, 3, 64, CODE[dtype], tdx.make_act_opts(out_dtype=CODE[out])))
    want = RO.swiglu(yv)
    near(host(o), want, (U[out] + F * (24 + 4 * np.abs(yv[:, :64]))) * np.abs(want), "out")
    do, dov = dev(np.full((3, 64), 2.0 ** 20), dtype)
    dy = torch.full_like(y, PAD)
    tdx.check(tdx.tdx_swiglu_bwd(y, do, dy, 3, 64, CODE[dtype]))
    want = RO.swiglu_bwd(yv, dov)
    a = np.abs(yv[:, :64])
    calc = F * (24 + 4 * np.concatenate([a, a], 1)) + 2.0 ** -21   # the sigmoid's own subnormal steps
    near(host(dy), want, (U[dtype] + calc) * np.abs(want), "dy")


def test_swiglu_to_fp32_within_a_few_roundings():
    """exp (2 F), the sum, the quotient (F each) and two products (F each), and the same for the gradient's
    five factors: 16 F, for any g whose result is no subnormal."""
    g = np.linspace(-86.0, 86.0, 4096)
    y, yv = dev(np.concatenate([g, np.linspace(0.5, 1.5, 4096)])[None].repeat(2, 0), "fp32")
    o, dy = torch.full((2, 4096), PAD, device="cuda"), torch.full_like(y, PAD)
    tdx.check(tdx.tdx_swiglu(y, o, None, None, 2, 4096, 2, tdx.make_act_opts(out_dtype=2)))
    near(host(o), RO.swiglu(yv), 16 * F * np.abs(RO.swiglu(yv)), "out")
    do, dov = dev(np.ones((2, 4096)), "fp32")
    tdx.check(tdx.tdx_swiglu_bwd(y, do, dy, 2, 4096, 2))
    s, a = RO.scores(yv[:, :4096], "sigmoid"), np.abs(yv[:, :4096])
    mag = np.concatenate([s * (1 + a * (1 - s)) * yv[:, 4096:], s * a], 1)
    near(host(dy), RO.swiglu_bwd(yv, dov), 16 * F * mag, "dy")
    half = y.bfloat16()
    o.fill_(PAD)
    tdx.check(tdx.tdx_swiglu(half, o, None, None, 2, 4096, 0, tdx.make_act_opts(out_dtype=2)))
    want = RO.swiglu(half.double().cpu().numpy())
    near(host(o), want, 16 * F * np.abs(want), "out of bf16")
