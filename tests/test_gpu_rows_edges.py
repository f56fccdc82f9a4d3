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


@pytest.mark.parametrize("T,H", [(200, 1040), (333, 2064), (200, 7168), (160, 16384)])
@pytest.mark.parametrize("dtype,out,mode", [("bf16", "bf16", ""), ("bf16", "e4m3", "rows"), ("bf16", "e4m3", "tensor"),
                                            ("bf16", "fp32", ""), ("fp32", "fp32", ""), ("fp32", "e4m3", "rows")])
@pytest.mark.parametrize("res,pad", [(True, 0), (False, 16), (True, 48)])
def test_rmsnorm_of_more_rows_than_multiprocessors(T, H, dtype, out, mode, res, pad):
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
    again = run_norm(x, r, w, dtype, out, mode == "rows", out_scale=scale, pad=pad)
    for a, b in zip((h, y, rs, rstd), again):
        if a is not None:
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("T,H", [(200, 2048), (333, 7168)])
@pytest.mark.parametrize("target", ["x", "residual"])
def test_rmsnorm_in_place_of_more_rows_than_multiprocessors(T, H, target):
    g = torch.Generator().manual_seed(5)
    x, r = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.randn(H, generator=g).bfloat16().cuda()
    h, y, _, rstd = run_norm(x, r, w, "bf16", "bf16")
    a, b = x.clone(), r.clone()
    y2, rstd2 = torch.empty_like(y), torch.empty_like(rstd)
    tdx.check(tdx.tdx_rmsnorm(a, b, w, a if target == "x" else b, y2, None, rstd2, T, H, 0))
    assert torch.equal(a if target == "x" else b, h) and torch.equal(y2, y) and torch.equal(rstd2, rstd)
    assert torch.equal(b if target == "x" else a, r if target == "x" else x)


# Rows that 152 multiprocessors have in hand at once, by the row's length, and sizes of more than 2 * stages + 1
# rounds of them, the last one uneven, in every layout of the kernel
BWD_IN_HAND = [(64, 19456), (128, 9728), (256, 4864), (512, 2432), (1024, 1216), (2560, 456), (1 << 30, 152)]
BWD_ROUNDS = [(100003, 48), (50021, 112), (25013, 208), (12503, 400), (6211, 1024), (3301, 2064), (1093, 4112),
              (1200, 7168), (1093, 8192), (801, 8208), (801, 16384), (1000, 20000)]


@pytest.mark.parametrize("T,H", BWD_ROUNDS)
@pytest.mark.parametrize("dtype,res,pad", [("bf16", True, 0), ("bf16", False, 8), ("fp32", True, 8), ("fp32", False, 0)])
def test_rmsnorm_bwd_of_many_rows_per_block(T, H, dtype, res, pad):
    g = torch.Generator(device="cuda").manual_seed(T + H)

    def make(scale, *shape):
        return torch.randn(*shape, generator=g, device="cuda").mul_(scale).to(TORCH[dtype])

    def padded(src):
        v = strided(T, H, dtype, H + pad)[1]
        v.copy_(src)
        return v

    h, dy, w = make(3.0, T, H), make(0.1, T, H), make(0.2, H) + 1
    dr = make(0.1, T, H) if res else None
    rstd = 1 / (h.float().square().mean(-1) + 1e-6).sqrt()
    ld = H + pad if pad else 0
    o = tdx.make_norm_opts(ld_x=ld, ld_residual=ld, ld_h=ld, ld_y=ld)
    ws = torch.full((tdx.tdx_rmsnorm_bwd_workspace_size(T, H, CODE[dtype]),), 255, dtype=torch.uint8, device="cuda")
    dys, hs, drs = padded(dy), padded(h), padded(dr) if res else None
    got = []
    for _ in range(3):
        dxb, dx = strided(T, H, dtype, H + pad)
        dw = torch.full((H,), PAD, device="cuda")
        tdx.check(tdx.tdx_rmsnorm_bwd(dys, hs, w, rstd, drs, dx, dw, ws, T, H, CODE[dtype], o))
        got.append((dxb, dw))
    assert all(torch.equal(got[0][i], other[i]) for other in got[1:] for i in (0, 1))
    if pad:
        assert bool((got[0][0][:, H:].float() == PAD).all())
    # the formula in 64 bits, on the device
    hd, dyd, rd = h.double(), dy.double(), rstd.double()[:, None]
    n, gd = hd * rd, dyd * w.double()
    want = rd * (gd - n * (gd * n).mean(1, keepdim=True)) + (dr.double() if res else 0)
    mag = rd * (gd.abs() + n.abs() * (gd * n).abs().mean(1, keepdim=True)) + (dr.double().abs() if res else 0)
    off = (got[0][0][:, :H].double() - want).abs() - (U[dtype] * want.abs() + F * (H / 32 + 64) * mag)
    assert float(off.max()) <= 0, "dx"
    # a column's additions one after another: the rounds, up to 32 rows of a block, up to 19 blocks, 32 warps
    serial = T / next(rows for most, rows in BWD_IN_HAND if H <= most) + 96
    off = (got[0][1].double() - (dyd * n).sum(0)).abs() - F * serial * (dyd * n).abs().sum(0)
    assert float(off.max()) <= 0, "dw"
    # in place over the gradient that comes in
    tdx.check(tdx.tdx_rmsnorm_bwd(dys, hs, w, rstd, drs, dys, got[0][1], ws, T, H, CODE[dtype], o))
    assert torch.equal(dys, got[1][0][:, :H]) and torch.equal(got[0][1], got[1][1])


# --------------------------------------------------------------------------------------- route
@pytest.mark.parametrize("T,E,k,n_group", [(5, 64, 8, 1), (900, 64, 8, 1), (900, 33, 12, 1), (5, 256, 8, 8),
                                           (900, 256, 8, 8), (40, 500, 5, 5)])
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


@pytest.mark.parametrize("T,E,k", [(700, 64, 16), (700, 20, 12), (900, 128, 16), (700, 33, 9)])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_route_of_several_places_per_lane(T, E, k, score, bias, dtype):
    rng = np.random.default_rng(E * 31 + k)
    x, xv = dev(1.5 * rng.standard_normal((T, E)), dtype)
    b, bv = dev(0.05 * rng.standard_normal(E), "fp32") if bias else (None, None)
    ids, gates = run_route(x, k, dtype, b, score=score_code(score))
    want, wg, margin = RO.route(xv, k, score, bv)
    clear = margin > 32 * F
    assert clear.mean() >= 0.9
    assert np.array_equal(ids[clear], want[clear])
    near(gates[clear], wg[clear], F * (E / 16 + 64 + np.abs(xv).max() * 2) * wg[clear], "gates")
    # ties: a few values only, equal keys in the order of their experts
    x, xv = dev(np.array([-1.0, -0.25, 0.0, 0.5, 1.25])[rng.integers(0, 5, (T, E))], "bf16")
    b, bv = dev(rng.integers(-1, 2, E) / 64.0, "fp32") if bias else (None, None)
    ids, _ = run_route(x, k, "bf16", b, score=score_code(score))
    key = xv if score == "softmax" and not bias else np.round(RO.scores(xv, score) + (0 if bv is None else bv), 12)
    if not (score == "softmax" and bias):   # sums of a softmax score and a bias may round together
        assert np.array_equal(ids, np.argsort(-key, axis=1, kind="stable")[:, :k])


@pytest.mark.parametrize("T,E,k", [(700, 64, 16), (700, 24, 10), (900, 128, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_of_several_places_per_lane_whose_keys_differ_in_their_last_bits(T, E, k, score):
    g = torch.Generator().manual_seed(E)
    x = (torch.randn(T, 1, generator=g) + 2.0 ** -22 * torch.randint(-6, 7, (T, E), generator=g)).cuda()
    x[::3] += (torch.rand(x[::3].shape, generator=g) < 0.5).cuda() * 1.0
    ids, _ = run_route(x, k, score=score_code(score))
    key = (x if score == "softmax" else 1.0 / (1.0 + torch.exp(-x))).cpu().numpy().astype(np.float64)
    assert np.array_equal(ids, np.argsort(-key, axis=1, kind="stable")[:, :k])


@pytest.mark.parametrize("T,E,k", [(300, 24, 4), (300, 64, 8), (300, 64, 16), (300, 128, 16), (300, 256, 8),
                                   (300, 500, 16)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [0, 1])
def test_route_bwd_of_ids_that_come_twice(T, E, k, score, renorm):
    """Places that name one expert add up, in pairs and three of a kind, on one lane and on several."""
    rng = np.random.default_rng(E + k)
    x, xv = dev(1.5 * rng.standard_normal((T, E)), "fp32")
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    ids[::4, 1] = ids[::4, 0]
    ids[1::4, k - 1] = ids[1::4, 0]
    ids[2::4, [1, k - 1]] = ids[2::4, [k // 2]]
    if k > 8:
        ids[::4, 8] = ids[::4, 0]
        ids[1::4, 15 if k > 15 else 9] = ids[1::4, 7 if k > 15 else 1]
    dg, dgv = dev(rng.standard_normal((T, k)), "fp32")
    out = torch.full((T, E), PAD, device="cuda")
    tdx.check(tdx.tdx_moe_route_bwd(x, torch.from_numpy(ids.astype(np.int32)).cuda(), dg, out, T, E, k, 2,
                                    tdx.make_route_opts(score=score_code(score), renorm=renorm)))
    want = RO.route_bwd(xv, ids, dgv, score, bool(renorm), 1.0)
    s = RO.scores(xv, score)
    S = np.take_along_axis(s, ids, 1).sum(1, keepdims=True)
    mag = s * np.abs(dgv).sum(1, keepdims=True) * (2 / np.minimum(S, 1) if renorm else 2)
    near(host(out), want, U["fp32"] * np.abs(want) + F * (E / 16 + 64 + 4 * np.abs(xv).max()) * mag, "dlogits")


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


# ---------------------------------------------------------------------------------------- sizes
def test_gradients_and_routing_beyond_2_to_the_31_elements():
    """Row offsets past 32 bits: the last rows of a tall tensor are those of a short one."""
    H, T = 8192, 270000                                # 2.2e9 elements
    gen = torch.Generator().manual_seed(1)
    h, dy = (torch.ones(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tail_h, tail_dy = (torch.randn(5, H, generator=gen).bfloat16().cuda() for _ in range(2))
    h[-5:], dy[-5:] = tail_h, tail_dy
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    rstd = torch.ones(T, device="cuda")
    dx, few = torch.empty_like(h), torch.empty_like(tail_h)
    dw, dws = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(tdx.tdx_rmsnorm_bwd_workspace_size(T, H, 0), dtype=torch.uint8, device="cuda")
    tdx.check(tdx.tdx_rmsnorm_bwd(dy, h, w, rstd, None, dx, dw, ws, T, H, 0))
    tdx.check(tdx.tdx_rmsnorm_bwd(tail_dy, tail_h, w, rstd[-5:].clone(), None, few, dws, ws, 5, H, 0))
    assert torch.equal(dx[-5:], few)
    assert int(torch.count_nonzero(dx[:-5])) == 0      # g - n * mean(g n) = 1 - 1
    want = (tail_dy.double() * tail_h.double()).sum(0) + (T - 5)
    assert float((dw.double() - want).abs().max()) <= F * (T + 32) * (T + 100)
    del h, dy, dx
    T, E, k = 4300000, 512, 4                          # 2.2e9 logits
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(700, E, generator=gen).bfloat16().cuda()
    x[-700:] = tail
    idx, gates = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    few_idx, few_gates = torch.empty(700, k, dtype=torch.int32, device="cuda"), torch.empty(700, k, device="cuda")
    tdx.check(tdx.tdx_moe_route(x, None, idx, gates, None, T, E, k, 0))
    tdx.check(tdx.tdx_moe_route(tail, None, few_idx, few_gates, None, 700, E, k, 0))
    assert torch.equal(idx[-700:], few_idx) and torch.equal(gates[-700:], few_gates)
    assert bool((idx[:-700] == torch.arange(k, device="cuda")).all()) and bool((gates[:-700] == 0.25).all())
    dg = torch.randn(T, k, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    dl, few = torch.full_like(x, PAD), torch.empty_like(tail)
    o = tdx.make_route_opts(renorm=0)
    tdx.check(tdx.tdx_moe_route_bwd(x, idx, dg, dl, T, E, k, 0, o))
    tdx.check(tdx.tdx_moe_route_bwd(tail, few_idx, dg[-700:].clone(), few, 700, E, k, 0, o))
    assert torch.equal(dl[-700:], few)
    s = dg[:-700].sum(1)                               # p (dg_i - p sum dg), p = 2^-9
    at = torch.arange(0, T - 700, 99991, device="cuda")
    assert torch.allclose(dl[at, E - 1].float(), -s[at] * 2.0 ** -18, rtol=2.0 ** -7, atol=2.0 ** -38)
