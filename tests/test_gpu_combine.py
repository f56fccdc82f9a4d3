"""GPU tests of the sum of a token's expert rows and its gradient against the 64-bit oracle.

Sums of up to 16 fp32 products: each of the 16 fused additions rounds within 2^-24 of the running sum, which stays
below the magnitude: 17 * 2^-24 * magnitude, then one rounding (half a step: bf16 2^-8, fp32 2^-24). A gate's gradient
adds H products over threads, lanes and warps: (H / 32 + 16) * 2^-24 * magnitude is above every chain's length (a
thread's chain has at most 8 * ceil(H / 2048) + 8 additions in bf16, then 5 over lanes and 8 over warps)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import comm_overlapped_gemm_gb300 as tdx
    from oracle import products as P

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def code(t):
    return {BF: tdx.TDX_BF16, F32: tdx.TDX_FP32}[t]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def close(got, want, slack, dtype):
    g = f64(got)
    lim = slack + HALF[dtype] * (np.abs(want) + slack) + 2.0 ** -126
    assert (np.abs(g - want) <= lim).all(), float(np.max(np.abs(g - want) / lim))


def inputs(T, H, k, dtype, seed, spare=3, pad=0):
    g = torch.Generator().manual_seed(seed)
    R = T * k + spare
    Z = torch.randn(R, H + pad, generator=g).to(dtype).cuda()
    dest = torch.randperm(R, generator=g)[:T * k].to(torch.int32)
    gates = torch.rand(T, k, generator=g)
    dout = torch.randn(T, H + pad, generator=g).to(dtype).cuda()
    return R, Z, dest, gates, dout


# the last ones are large enough for several vectors a thread
CASES = [(1, 8, 1), (1, 7168, 8), (2, 16, 3), (33, 64, 16), (200, 1000, 8), (1000, 264, 2), (77, 4104, 9), (5, 20000, 4), (2501, 1000, 2),
         (1301, 2056, 4)]


@pytest.mark.parametrize("T,H,k", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("gated", [True, False])
def test_combine(T, H, k, dtype, out, gated):
    pad = 24 if T % 2 else 0
    R, Z, dest, gates, _ = inputs(T, H, k, dtype, T + H, pad=pad)
    if T > 1:   # entries outside add nothing; a row named twice counts twice
        dest[0], dest[T * k - 1], dest[1] = -1, R, dest[2]
    d, gt = dest.cuda(), gates.cuda() if gated else None
    got = torch.full((T, H + pad), 777.0, device="cuda", dtype=out)
    o = tdx.make_combine_opts(out_dtype=code(out), ld_z=H + pad, ld_out=H + pad)
    tdx.check(tdx.tdx_moe_combine(Z, d, gt, got, R, T, H, k, code(dtype), o))
    want, mag = P.combine(f64(Z)[:, :H], dest.numpy(), gates.double().numpy() if gated else None, T)
    close(got[:, :H], want, 17 * 2.0 ** -24 * mag, out)
    assert (got[:, H:] == got.new_tensor(777.0)).all()


@pytest.mark.parametrize("T,H,k", CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gated", [True, False])
def test_combine_bwd(T, H, k, dtype, gated):
    pad = 24 if T % 2 else 0
    R, Z, dest, gates, dout = inputs(T, H, k, dtype, T * 3 + H, pad=pad)
    if T > 1:
        dest[0], dest[T * k - 1] = -1, R
    d, gt = dest.cuda(), gates.cuda() if gated else None
    o = tdx.make_combine_opts(ld_z=H + pad, ld_out=H + pad)
    dZ = torch.full_like(Z, 777.0)
    dg = torch.full((T, k), 777.0, device="cuda")
    tdx.check(tdx.tdx_moe_combine_bwd(dout, Z, d, gt, dZ, dg, R, T, H, k, code(dtype), o))
    want, wg, mag = P.combine_bwd(f64(dout)[:, :H], f64(Z)[:, :H], dest.numpy(), gates.double().numpy() if gated else None)
    named = ~np.isnan(want[:, 0])
    close(dZ[torch.from_numpy(named).cuda()][:, :H], want[named], 2.0 ** -24 * np.abs(want[named]), dtype)
    assert (dZ[torch.from_numpy(~named).cuda()] == dZ.new_tensor(777.0)).all()
    assert (dZ[:, H:] == dZ.new_tensor(777.0)).all()
    assert (np.abs(f64(dg) - wg) <= (H / 32 + 16) * 2.0 ** -24 * mag).all()
    # each output alone, and dZ in place of Z
    dg2, z2 = torch.empty_like(dg), Z.clone()
    tdx.check(tdx.tdx_moe_combine_bwd(dout, Z, d, gt, None, dg2, R, T, H, k, code(dtype), o))
    tdx.check(tdx.tdx_moe_combine_bwd(dout, z2, d, gt, z2, dg, R, T, H, k, code(dtype), o))
    assert torch.equal(dg, dg2)
    at = torch.from_numpy(named).cuda()
    assert torch.equal(z2[at][:, :H], dZ[at][:, :H]) and torch.equal(z2[~at], Z[~at])
    z3 = torch.full_like(Z, 777.0)
    tdx.check(tdx.tdx_moe_combine_bwd(dout, None, d, gt, z3, None, R, T, H, k, code(dtype), o))
    assert torch.equal(z3, dZ)


def test_combine_no_rows():
    """R = 0: every entry is outside."""
    out = torch.full((3, 64), 5.0, dtype=BF, device="cuda")
    d = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    Z = torch.ones(1, 64, dtype=BF, device="cuda")
    tdx.check(tdx.tdx_moe_combine(Z, d, None, out, 0, 3, 64, 2, tdx.TDX_BF16))
    assert (out == 0).all()
    dg = torch.full((3, 2), 5.0, device="cuda")
    tdx.check(tdx.tdx_moe_combine_bwd(out, Z, d, None, Z, dg, 0, 3, 64, 2, tdx.TDX_BF16))
    assert (dg == 0).all() and (Z == 1).all()
