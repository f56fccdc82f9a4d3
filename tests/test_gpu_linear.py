"""GPU tests of the linear layer, the products grouped by expert and their gradients against the 64-bit oracle.

Integer inputs: every partial sum is an integer below 2^24, so fp32 results are the oracle's exactly and
bf16 results its rounding. Random inputs: the tensor cores add K products 16 (bf16) or 32 (e4m3) at a time to an
fp32 accumulator and may truncate each addition, an error of at most 2^-22 of the magnitude per addition; with the
sum of partial accumulators and the epilogue's scales

    |v - exact| <= (K / 16 + 16) * 2^-22 * magnitude.

A result then takes the activation (slope at most 1.13; its approximate exponential within
2^-22 * (4 + |exponent|)) and one rounding, half a step relative: bf16 2^-8, e4m3 2^-4 (2^-10 below its normal
range), fp32 2^-24."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import comm_overlapped_gemm_gb300 as tdx
    from oracle import products as P

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24, E4: 2.0 ** -4}


def code(t):
    return {BF: tdx.TDX_BF16, F32: tdx.TDX_FP32, E4: tdx.TDX_FP8_E4M3}[t]


def act_code(name):
    return getattr(tdx, "TDX_ACT_" + name.upper())


def gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


def ints(g, *shape, most=4, dtype=None):
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype or BF).cuda()


def rand(g, *shape, scale=1.0, dtype=None):
    v = torch.randn(*shape, generator=g) * scale
    return v.to(dtype or BF).cuda()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def padded(t, pad):
    """The same matrix with `pad` more columns in memory, filled with NaN; returns (view, stride)."""
    if not pad:
        return t, 0
    big = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=F32, device="cuda").to(t.dtype)
    big[..., :t.shape[-1]] = t
    return big, t.shape[-1] + pad


def same(got, want, dtype):
    """got is want rounded to dtype, bit for bit (NaN equals NaN)."""
    w = torch.from_numpy(np.ascontiguousarray(want)).to(F32).to(dtype).float()
    g = got.float().cpu()
    assert torch.equal(torch.nan_to_num(g, nan=12345.0), torch.nan_to_num(w, nan=12345.0)), \
        float((g - w).abs().nan_to_num(0).max())


def close(got, want, slack, dtype):
    """|got - want| <= slack + the rounding to dtype."""
    g = f64(got)
    lim = slack + HALF[dtype] * (np.abs(want) + slack) + (2.0 ** -10 if dtype == E4 else 2.0 ** -126)
    bad = ~(np.abs(g - want) <= lim)
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(g - want) / lim)))


def acc_slack(K, mag):
    return (K / 16 + 16) * 2.0 ** -22 * mag


def run_linear(A, B, bias=None, res=None, rs=None, out=None, act="none", alpha=1.0, z=False, out_scale=1.0, pad=0,
               offsets=None, es=None, status=None):
    M, K = A.shape
    N = B.shape[-1]
    cols = N // 2 if act == "swiglu" else N
    out = out or BF
    C = torch.full((M, cols + pad), 777.0, dtype=F32, device="cuda").to(out)
    Z = torch.full((M, N + pad), 777.0, dtype=BF, device="cuda") if z else None
    Ap, la = padded(A, 16 * pad // 16)
    Bp, lb = padded(B, pad)
    Rp, lr = padded(res, pad) if res is not None else (None, 0)
    o = tdx.make_linear_opts(out_dtype=code(out), act=act_code(act), alpha=alpha, out_scale=out_scale, ld_a=la, ld_b=lb,
                             ld_c=cols + pad if pad else 0, ld_residual=lr, ld_z=N + pad if pad else 0,
                             device_status=status)
    if offsets is None:
        tdx.check(tdx.tdx_linear(Ap, Bp, bias, Rp, rs, C, Z, M, K, N, code(A.dtype), o))
    else:
        tdx.check(tdx.tdx_grouped_gemm(Ap, offsets, Bp, rs, es, C, Z, M, K, N, B.shape[0], code(A.dtype), o))
    torch.cuda.synchronize()
    if pad:
        assert (C[:, cols:].float() == torch.tensor(777.0).to(out).float()).all()   # behind the rows: as it was
    return C[:, :cols], None if Z is None else Z[:, :N]


SIZES = [(1, 8, 8), (1, 64, 128), (1, 4096, 1024), (2, 1000, 136), (16, 8192, 1024), (63, 72, 8), (127, 128, 120),
         (128, 512, 128), (129, 520, 264), (200, 64, 2048), (255, 1024, 1000), (300, 4096, 264), (1000, 264, 1000),
         (1999, 520, 2040), (2048, 1024, 4096), (4097, 256, 1288), (130, 8, 10000), (1, 72, 100000)]


# ---------------------------------------------------------------------------------- linear layer
@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("pad", [0, 16])
def test_linear_integers(M, K, N, pad):
    g = gen(M * 7 + K + N)
    A, B = ints(g, M, K), ints(g, K, N)
    bias, res = ints(g, N, most=60), ints(g, M, N, most=60)
    want = 0.5 * (f64(A) @ f64(B)) + f64(bias)
    C, z = run_linear(A, B, bias, res, out=F32, alpha=0.5, z=True, pad=pad)
    same(C, want + f64(res), F32)
    same(z, want, BF)
    C, _ = run_linear(A, B, pad=pad)
    same(C, f64(A) @ f64(B), BF)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("M,K,N", [(1, 512, 256), (77, 1000, 528), (2100, 264, 2064)])
@pytest.mark.parametrize("out", [BF, F32, E4])
def test_linear_activations(act, M, K, N, out):
    g = gen(11 * M + N)
    A, B, bias = rand(g, M, K), rand(g, K, N, scale=2.0 / K ** 0.5), rand(g, N)
    cols = N // 2 if act == "swiglu" else N
    if out == E4 and cols % 16:
        pytest.skip("e4m3 rows are multiples of 16 bytes")
    res = rand(g, M, cols)
    scale = 0.0625 if out == E4 else 1.0
    C, z = run_linear(A, B, bias, res, out=out, act=act, z=True, out_scale=scale)
    v, mag = P.product(f64(A), f64(B))
    v, mag = v + f64(bias), mag + np.abs(f64(bias))
    dv = acc_slack(K, mag)
    close(z, v, dv, BF)
    y = P.act(act, v)
    if act == "swiglu":
        gate, up, dg, du = v[:, :cols], v[:, cols:], dv[:, :cols], dv[:, cols:]
        slack = 1.1 * dg * (np.abs(up) + du) + np.abs(P.act("silu", gate)) * du
        expo = np.abs(gate)
    else:
        slack, expo = 1.13 * dv, 1.6 * np.abs(v + 0.045 * v ** 3) if act == "gelu_tanh" else np.abs(v)
    slack = slack + 2.0 ** -21 * (4 + expo) * np.abs(y)
    want = (y + f64(res)) / scale
    close(C, np.clip(want, -448, 448) if out == E4 else want, (slack + 2.0 ** -23 * np.abs(y + f64(res))) / scale, out)


@pytest.mark.parametrize("M,K,N", [(1, 8192, 512), (5, 144, 48), (130, 1040, 272), (257, 528, 2064), (2304, 1024, 2048)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_e4m3(M, K, N, act):
    if act == "swiglu" and N % 32:
        pytest.skip("halves of 16-byte steps")
    g = gen(M + K)
    A, B = rand(g, M, K, scale=30.0, dtype=E4), rand(g, K, N, scale=30.0, dtype=E4)
    rs = (torch.rand(M, generator=g) + 0.5).cuda()
    C, z = run_linear(A, B, rs=rs, alpha=2.0 ** -14, act=act, z=True)
    v, mag = P.product(f64(A), f64(B))
    f = f64(rs)[:, None] * 2.0 ** -14
    v, dv = v * f, acc_slack(K, mag * f)
    close(z, v, dv, BF)
    if act == "none":
        close(C, v, dv, BF)
    else:
        h = N // 2
        y = P.act("swiglu", v)
        close(C, y, 1.1 * dv[:, :h] * (np.abs(v[:, h:]) + dv[:, h:]) + np.abs(P.act("silu", v[:, :h])) * dv[:, h:] +
              2.0 ** -21 * (4 + np.abs(v[:, :h])) * np.abs(y), BF)


def test_linear_e4m3_integers():
    for M, K, N in [(1, 16, 16), (100, 4096, 1024), (1200, 272, 1040), (3000, 512, 2048)]:
        g = gen(N)
        A, B = ints(g, M, K, dtype=E4), ints(g, K, N, dtype=E4)
        C, _ = run_linear(A, B, out=F32, pad=16)
        same(C, f64(A) @ f64(B), F32)


@pytest.mark.parametrize("M,K,N", [(3, 64, 64), (200, 72, 528), (2304, 128, 2064)])
@pytest.mark.parametrize("out", [BF, F32])
def test_linear_rows_off_32_byte_boundaries(M, K, N, out):
    """Buffers and strides that are multiples of 16 bytes and no more; rows and columns around them untouched."""
    g = gen(M)
    e = 8 if out == BF else 4
    A, B, bias = ints(g, M, K), ints(g, K, N), ints(g, N)
    buf = torch.full((M * (N + e) + e,), 777.0, device="cuda").to(out)
    C = buf[e:].view(M, N + e)
    zbuf = torch.full((M * (N + 8) + 8,), 777.0, device="cuda").to(BF)
    Z = zbuf[8:].view(M, N + 8)
    for z in (None, Z):
        o = tdx.make_linear_opts(out_dtype=code(out), ld_c=N + e, ld_z=N + 8)
        tdx.check(tdx.tdx_linear(A, B, bias, None, None, C, z, M, K, N, tdx.TDX_BF16, o))
        want = f64(A) @ f64(B) + f64(bias)
        same(C[:, :N], want, out)
        assert (C[:, N:] == C.new_tensor(777.0)).all() and (buf[:e] == buf.new_tensor(777.0)).all()
    same(Z[:, :N], want, BF)
    assert (Z[:, N:] == Z.new_tensor(777.0)).all()
    # gate and up halves, 16-byte steps apart
    h = N // 2
    Y = buf[e:e + M * (h + e)].view(M, h + e)
    buf.fill_(777.0)
    o = tdx.make_linear_opts(out_dtype=code(out), act=tdx.TDX_ACT_SWIGLU, ld_c=h + e, ld_z=N + 8)
    tdx.check(tdx.tdx_linear(A, B, bias, None, None, Y, Z, M, K, N, tdx.TDX_BF16, o))
    same(Z[:, :N], want, BF)
    y = P.act("swiglu", want)
    # where exp(-g) passes fp32's range (2^128) the sigmoid, then below 2^-128, is taken as 0: off by |g| 2^-128 |u|
    tiny = 2.0 ** -127 * np.abs(want[:, :h] * want[:, h:])
    close(Y[:, :h], y, 2.0 ** -21 * (4 + np.abs(want[:, :h])) * np.abs(y) + tiny, out)
    assert (Y[:, h:] == Y.new_tensor(777.0)).all()


def test_linear_e4m3_to_e4m3():
    """The e4m3 product's gated result as the next product's e4m3 input. Codes lie up to half a step (2^-4) off."""
    for M, K, N in [(1, 512, 256), (300, 272, 1056), (1100, 512, 2048)]:
        g = gen(M)
        A, B = rand(g, M, K, scale=30.0, dtype=E4), rand(g, K, N, scale=30.0, dtype=E4)
        C, _ = run_linear(A, B, out=E4, act="swiglu", alpha=2.0 ** -14, out_scale=0.03125)
        v, mag = P.product(f64(A), f64(B))
        v, dv, h = v * 2.0 ** -14, acc_slack(K, mag * 2.0 ** -14), N // 2
        y = P.act("swiglu", v)
        slack = 1.1 * dv[:, :h] * (np.abs(v[:, h:]) + dv[:, h:]) + np.abs(P.act("silu", v[:, :h])) * dv[:, h:] + \
            2.0 ** -21 * (4 + np.abs(v[:, :h])) * np.abs(y)
        close(C, np.clip(y * 32, -448, 448), slack * 32, E4)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu", "swiglu"])
def test_activations_of_a_masks_lowest_value(act):
    """Values at the ends of the type: the gate is 0 or the value itself, its gradient 0 or dy."""
    low, high = float(torch.finfo(BF).min), float(torch.finfo(BF).max)
    x = [low, -1e30, -1e19, -200.0, -30.0, 0.0, 30.0, 200.0, 1e19, 1e30, high]
    n = 16
    gate = torch.tensor(x + [0.0] * (n - len(x)), device="cuda").to(BF)
    up = torch.ones(n, dtype=BF, device="cuda")
    bias = torch.cat([gate, up]) if act == "swiglu" else gate
    N = bias.numel()
    A, B = torch.zeros(3, 8, dtype=BF, device="cuda"), torch.zeros(8, N, dtype=BF, device="cuda")
    want = torch.where(gate > 0, gate, torch.zeros_like(gate)).double().cpu().numpy()
    for out in (BF, F32):
        C, _ = run_linear(A, B, bias, out=out, act=act)
        # from |x| = 30 on what is left of the gate is below 30 * exp(-30) = 3e-12
        assert (np.abs(f64(C) - want) <= 2.0 ** -8 * np.abs(want) + 3e-12).all()
    z, dy = bias.expand(3, N).contiguous(), torch.full((3, n), 2.0, dtype=BF, device="cuda")
    dz = torch.empty_like(z)
    tdx.check(tdx.tdx_linear_act_bwd(dy, z, dz, None, None, 3, N, 0, tdx.make_linear_opts(act=act_code(act))))
    got = f64(dz)[:, :n]
    slope = np.where(f64(gate) > 0, 2.0, 0.0)
    at0 = np.array([v == 0.0 for v in x] + [True] * (n - len(x)))
    slope[at0] = 0.0 if act == "relu" else 1.0
    assert (np.abs(got - slope) <= 1e-9).all()
    if act != "swiglu":   # the same gradient in place of dy
        tdx.check(tdx.tdx_linear_act_bwd(dy, z, dy, None, None, 3, N, 0, tdx.make_linear_opts(act=act_code(act))))
        assert torch.equal(dy, dz)


def test_linear_residual_in_place_and_inf():
    g = gen(5)
    for M, N in [(3, 64), (700, 2048)]:
        A, B, C = ints(g, M, 128), ints(g, 128, N), ints(g, M, N)
        want = f64(A) @ f64(B) + f64(C)
        tdx.check(tdx.tdx_linear(A, B, None, C, None, C, None, M, 128, N, tdx.TDX_BF16))
        same(C, want, BF)
        # an infinity and a NaN stay in their own row
        A[1, 5], A[2, 7] = float("inf"), float("nan")
        C2, _ = run_linear(A, B, out=F32)
        with np.errstate(invalid="ignore"):
            want = f64(A) @ f64(B)
            assert np.array_equal(np.isnan(f64(C2)), np.isnan(want))
        keep = [i for i in range(M) if i not in (1, 2)]
        same(C2[keep], want[keep], F32)


# ------------------------------------------------------------------------------------- gradients
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
@pytest.mark.parametrize("M,N", [(1, 16), (2, 64), (33, 208), (1000, 528), (5003, 32), (4097, 2064)])
def test_linear_act_bwd(act, M, N):
    g = gen(M + N)
    cols = N // 2 if act == "swiglu" else N
    z, dy = rand(g, M, N, scale=2.0), rand(g, M, cols)
    zp, lz = padded(z, 8)
    dyp, ld = padded(dy, 24)
    dz = torch.full_like(zp, 777.0)
    db = torch.full((N,), 777.0, device="cuda")
    o = tdx.make_linear_opts(act=act_code(act), ld_z=lz, ld_c=ld)
    ws = torch.empty(tdx.tdx_linear_act_bwd_workspace_size(M, N, tdx.TDX_BF16, o), dtype=torch.uint8, device="cuda")
    tdx.check(tdx.tdx_linear_act_bwd(dyp, zp, dz, db, ws, M, N, tdx.TDX_BF16, o))
    torch.cuda.synchronize()
    v = f64(z)
    want = P.act_grad(act, v, f64(dy))
    assert (dz[:, N:] == 777.0).all()
    # the derivative's terms are up to 1 + |x| in size, each within 2^-21 * (4 + |exponent|)
    x = v[:, :cols] if act == "swiglu" else v
    expo = 1.6 * np.abs(x + 0.045 * x ** 3) if act == "gelu_tanh" else x * x if act == "gelu" else np.abs(x)
    size = np.abs(f64(dy)) * (1 + 1.6 * np.abs(x) * (1 + 0.14 * x * x))
    slack = 2.0 ** -21 * (4 + expo) * size
    if act == "swiglu":
        slack = np.concatenate([slack * np.abs(v[:, cols:]), slack * (1 + np.abs(x))], 1)
    if act in ("none", "relu"):
        same(dz[:, :N], want, BF)
        slack = 0 * want
    else:
        close(dz[:, :N], want, slack, BF)
    # M additions in fp32 (few long partial sums): each within 2^-24 of the magnitude
    lim = slack.sum(0) + (M + 2) * 2.0 ** -24 * np.abs(want).sum(0)
    assert (np.abs(f64(db) - want.sum(0)) <= lim + 1e-30).all()
    # dz in place of z, and sums alone
    db2 = torch.empty_like(db)
    tdx.check(tdx.tdx_linear_act_bwd(dyp, zp, None, db2, ws, M, N, tdx.TDX_BF16, o))
    z2 = zp.clone()
    tdx.check(tdx.tdx_linear_act_bwd(dyp, z2, z2, None, None, M, N, tdx.TDX_BF16, o))
    assert torch.equal(db2, db) and torch.equal(z2[:, :N], dz[:, :N])


BWD_SIZES = [(1, 8, 8), (1, 512, 1024), (7, 64, 136), (64, 72, 128), (65, 128, 264), (200, 1000, 520), (1021, 1024, 1024),
             (3001, 264, 136), (2000, 2048, 2056), (8200, 128, 256), (4096, 512, 2048)]


@pytest.mark.parametrize("M,K,N", BWD_SIZES)
@pytest.mark.parametrize("pad", [0, 16])
def test_linear_bwd_integers(M, K, N, pad):
    g = gen(M + K + N)
    dz, A, B, dres = ints(g, M, N), ints(g, M, K), ints(g, K, N), ints(g, M, K, most=60)
    (dzp, lz), (Ap, la), (Bp, lb), (rp, lr) = (padded(t, pad) for t in (dz, A, B, dres))
    for out, dw, acc in [(F32, F32, 1), (BF, BF, 0), (BF, BF, 1)]:
        dA = torch.full((M, K + pad), 777.0, device="cuda", dtype=out)
        old = ints(g, K, N + pad, most=9).to(dw)
        dB = old.clone()
        o = tdx.make_linear_opts(out_dtype=code(out), dw_dtype=code(dw), accumulate=acc, alpha=0.5, ld_a=la, ld_b=lb,
                                 ld_z=lz, ld_residual=lr, ld_c=K + pad if pad else 0)
        tdx.check(tdx.tdx_linear_bwd(dzp, Ap, Bp, rp, dA, dB, M, K, N, tdx.TDX_BF16, o))
        torch.cuda.synchronize()
        same(dA[:, :K], 0.5 * f64(dz) @ f64(B).T + f64(dres), out)
        same(dB[:, :N], 0.5 * f64(A).T @ f64(dz) + (f64(old[:, :N]) if acc else 0), dw)
        assert (dA[:, K:] == 777.0).all() and torch.equal(dB[:, N:], old[:, N:])


def test_linear_bwd_no_rows():
    """The sum over no rows is 0, and adds nothing to an accumulated gradient."""
    B = torch.ones(64, 128, dtype=BF, device="cuda")
    some = torch.ones(8, 128, dtype=BF, device="cuda")
    for acc, want in [(0, 0.0), (1, 3.0)]:
        dB = torch.full((64, 128), 3.0, device="cuda")
        o = tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32, accumulate=acc)
        tdx.check(tdx.tdx_linear_bwd(some, some, B, None, some, dB, 0, 64, 128, tdx.TDX_BF16, o))
        assert (dB == want).all() and (some == 1.0).all()


# --------------------------------------------------------------------------------------- grouped
def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


GROUPS = [
    ([1], 0, 0, 64, 128), ([0, 0, 3], 0, 0, 72, 136), ([5, 0, 1, 0, 0, 2], 0, 3, 512, 264),
    ([1, 1, 1, 1, 1, 1, 1, 1], 0, 0, 1024, 256), ([64, 128, 0, 63, 65, 1], 2, 1, 264, 120),
    ([300, 0, 129, 1, 255, 257, 64], 0, 5, 136, 1032), ([2000, 100, 1900], 0, 0, 256, 512),
    ([700, 0, 513, 800, 127, 1, 1500, 256], 7, 9, 512, 2048), ([0, 0], 0, 4, 64, 64),
    ([3] * 100, 0, 0, 64, 72), ([1, 0] * 256, 0, 0, 64, 64), ([130, 1, 65, 0, 64, 63, 600] * 6, 0, 2, 512, 2048)]


@pytest.mark.parametrize("counts,first,behind,K,N", GROUPS)
@pytest.mark.parametrize("pad", [0, 16])
def test_grouped_integers(counts, first, behind, K, N, pad):
    g = gen(sum(counts) + N)
    R, E = first + sum(counts) + behind, len(counts)
    X, B = ints(g, R, K), ints(g, E, K, N)
    X[:first] = float("nan")
    X[R - behind:] = float("inf")
    off = offsets_of(counts, first)
    want, _ = P.grouped(f64(X), off.tolist(), f64(B))
    C, z = run_linear(X, B, out=F32, z=True, offsets=off, pad=pad)
    inside = slice(first, R - behind)
    same(C[inside], want[inside], F32)
    same(z[inside], want[inside], BF)
    for t in (C, z):   # rows of no expert: as they were (777 as the type holds it)
        assert (t[:first] == t.new_tensor(777.0)).all() and (t[R - behind:] == t.new_tensor(777.0)).all()


@pytest.mark.parametrize("counts,first,behind,K,N", GROUPS)
@pytest.mark.parametrize("pad", [0, 16])
def test_grouped_bwd_integers(counts, first, behind, K, N, pad):
    g = gen(sum(counts) + K)
    R, E = first + sum(counts) + behind, len(counts)
    dY, X, B = ints(g, R, N), ints(g, R, K), ints(g, E, K, N)
    for t, bad in ((X, float("nan")), (dY, float("inf"))):   # rows of no expert reach nothing
        t[:first] = bad
        t[R - behind:] = bad
    off = offsets_of(counts, first)
    (dX, _), (dB, _) = P.grouped_bwd(f64(dY), f64(X), off.tolist(), f64(B))
    inside = slice(first, R - behind)
    (dyp, lz), (Xp, la), (Bp, lb) = (padded(t, pad) for t in (dY, X, B))
    for out, dw, acc in [(F32, F32, 1), (BF, BF, 0)]:
        got = torch.full((R, K + pad), 777.0, device="cuda", dtype=out)
        old = ints(g, E, K, N + pad, most=9).to(dw)
        gw = old.clone()
        o = tdx.make_linear_opts(out_dtype=code(out), dw_dtype=code(dw), accumulate=acc, ld_a=la, ld_b=lb, ld_z=lz,
                                 ld_c=K + pad if pad else 0)
        tdx.check(tdx.tdx_grouped_gemm_bwd(dyp, Xp, off, Bp, got, gw, R, K, N, E, tdx.TDX_BF16, o))
        torch.cuda.synchronize()
        same(got[inside, :K], dX[inside], out)
        assert (got[:first] == got.new_tensor(777.0)).all() and (got[R - behind:] == got.new_tensor(777.0)).all()
        same(gw[..., :N], dB + (f64(old[..., :N]) if acc else 0), dw)
        assert torch.equal(gw[..., N:], old[..., N:])


def test_grouped_bwd_foreign_infinities():
    """An expert's last rows share K slices with the next one's first: an infinity or a NaN there must not
    enter its sums."""
    g = gen(3)
    for counts, K, N in [([5, 3, 70, 1, 130], 128, 128), ([300, 1000, 257, 900], 512, 1024)]:
        R, E = sum(counts), len(counts)
        dY, X = ints(g, R, N), ints(g, R, K)
        off = offsets_of(counts)
        at = off.tolist()
        X[at[1]:at[2]] = float("nan")
        dY[at[3]:at[4]] = float("inf")
        dB = torch.empty(E, K, N, device="cuda")
        o = tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32)
        tdx.check(tdx.tdx_grouped_gemm_bwd(dY, X, off, None, None, dB, R, K, N, E, tdx.TDX_BF16, o))
        for e in range(E):
            if e == 1:
                assert torch.isnan(dB[e]).all()
            elif e != 3:
                same(dB[e], f64(X[at[e]:at[e + 1]]).T @ f64(dY[at[e]:at[e + 1]]), F32)


@pytest.mark.parametrize("act", ["none", "silu", "swiglu"])
def test_grouped_e4m3(act):
    for counts, K, N in [([1, 0, 2], 528, 288), ([300, 17, 0, 500], 1040, 1056), ([1500, 600, 2000, 900], 512, 2048)]:
        g = gen(K)
        R, E = sum(counts), len(counts)
        X, B = rand(g, R, K, scale=30.0, dtype=E4), rand(g, E, K, N, scale=30.0, dtype=E4)
        rs, es = (torch.rand(R, generator=g) + 0.5).cuda(), (torch.rand(E, generator=g) + 0.5).cuda()
        off = offsets_of(counts)
        C, z = run_linear(X, B, rs=rs, es=es, act=act, alpha=2.0 ** -14, z=True, offsets=off)
        v, mag = P.grouped(f64(X), off.tolist(), f64(B))
        f = 2.0 ** -14 * f64(rs)[:, None] * np.repeat(f64(es), counts)[:, None]
        v, dv = v * f, acc_slack(K, mag * f)
        close(z, v, dv, BF)
        h = N // 2
        y = P.act(act, v)
        if act == "swiglu":
            slack = 1.1 * dv[:, :h] * (np.abs(v[:, h:]) + dv[:, h:]) + np.abs(P.act("silu", v[:, :h])) * dv[:, h:]
            slack = slack + 2.0 ** -21 * (4 + np.abs(v[:, :h])) * np.abs(y)
        else:
            slack = 1.1 * dv + 2.0 ** -21 * (4 + np.abs(v)) * np.abs(y)
        close(C, y, slack, BF)


def test_grouped_bwd_no_rows():
    """Experts without any row: their gradients are 0, and dX, of no rows, is left alone."""
    one = torch.ones(8, 128, dtype=BF, device="cuda")
    B = torch.ones(3, 64, 128, dtype=BF, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    for rows in (0, 8):   # no rows at all, and 8 rows of no expert
        dB = torch.full((3, 64, 128), 3.0, device="cuda")
        dX = torch.full((8, 64), 3.0, dtype=BF, device="cuda")
        X = torch.full((8, 64), float("nan"), dtype=BF, device="cuda")
        tdx.check(tdx.tdx_grouped_gemm_bwd(one, X, off, B, dX, dB, rows, 64, 128, 3, tdx.TDX_BF16,
                                           tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32)))
        assert (dB == 0).all() and (dX == 3.0).all()
        Y = torch.full((8, 128), 3.0, dtype=BF, device="cuda")
        tdx.check(tdx.tdx_grouped_gemm(X, off, B, None, None, Y, None, rows, 64, 128, 3, tdx.TDX_BF16))
        assert (Y == 3.0).all()


def test_grouped_offsets_out_of_order():
    """Entries outside [0, R] are taken into it, one below its predecessor is raised to it."""
    g = gen(9)
    R, K, N = 200, 64, 128
    X, B = ints(g, R, K), ints(g, 5, K, N)
    off = torch.tensor([-7, 60, 20, 90, 1000, 150], dtype=torch.int32, device="cuda")
    sane = [0, 60, 60, 90, 200, 200]
    C, _ = run_linear(X, B, out=F32, offsets=off)
    same(C, P.grouped(f64(X), sane, f64(B))[0], F32)
    dY = ints(g, R, N)
    dB = torch.empty(5, K, N, device="cuda")
    o = tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32)
    tdx.check(tdx.tdx_grouped_gemm_bwd(dY, X, off, None, None, dB, R, K, N, 5, tdx.TDX_BF16, o))
    same(dB, P.grouped_bwd(f64(dY), f64(X), sane, f64(B))[1][0], F32)


# -------------------------------------------------------------------------------- long fp32 sums
@pytest.mark.parametrize("M,N", [(8, 128), (100, 272), (2048, 2304)])
def test_fp32_results_of_long_sums(M, N):
    """The tensor cores truncate each of a sum's additions, which for terms of one sign drifts with K. fp32 results
    add segments of 14 slices (896 of K in bf16: 56 additions within 2^-22 each, 80 with a margin as above) in
    fp32, K / 896 additions within 2^-24 each: whatever K, the error stays below that of the segments' own."""
    g = gen(M)
    K = 32768
    A = (torch.rand(M, K, generator=g) + 0.5).to(BF).cuda()
    B = (torch.rand(K, N, generator=g) + 0.5).to(BF).cuda()
    lim = 80 * 2.0 ** -22 + (K / 896 + 8) * 2.0 ** -24
    want = A.double() @ B.double()
    C, _ = run_linear(A, B, out=F32)
    assert float(((C.double() - want) / want).abs().max()) <= lim
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    C, _ = run_linear(A, B[None], out=F32, offsets=off)
    assert float(((C.double() - want) / want).abs().max()) <= lim
    # the weight gradient over K rows, plain and grouped, and the input gradient over K columns
    X, off = A.t().contiguous(), torch.tensor([0, K - 5, K], dtype=torch.int32, device="cuda")
    o = tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32, out_dtype=tdx.TDX_FP32)
    if M % 8 == 0:
        dB, dBg = torch.empty(M, N, device="cuda"), torch.empty(2, M, N, device="cuda")
        tdx.check(tdx.tdx_linear_bwd(B, X, None, None, None, dB, K, M, N, tdx.TDX_BF16, o))
        tdx.check(tdx.tdx_grouped_gemm_bwd(B, X, off, None, None, dBg, K, M, N, 2, tdx.TDX_BF16, o))
        assert float(((dB.double() - want) / want).abs().max()) <= lim
        assert float(((dBg.double().sum(0) - want) / want).abs().max()) <= lim
    dA = torch.empty(M, N, device="cuda")
    tdx.check(tdx.tdx_linear_bwd(A, None, B.t().contiguous(), None, dA, None, M, N, K, tdx.TDX_BF16, o))
    assert float(((dA.double() - want) / want).abs().max()) <= lim
    # act and gate over summed segments
    C, z = run_linear(A, B * 2.0 ** -15, out=F32, act="swiglu", z=True)
    w = (want * 2.0 ** -15).cpu().numpy()
    close(z, w, lim * np.abs(w), BF)
    y = P.act("swiglu", w)
    close(C, y, (2.2 * lim + 2.0 ** -21 * (4 + np.abs(w[:, :N // 2]))) * np.abs(y), F32)
