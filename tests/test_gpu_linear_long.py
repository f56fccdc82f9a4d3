"""GPU tests of products whose K passes one sum on the tensor cores: gated fp32 results of tiles that several CTAs
share, every column of which is summed and read by one warp.

Integer inputs, so that every sum is exact: v (kept in z) is compared bit for bit. silu(g) * u is then fp32 arithmetic
of exact forms, within 2^-21 * (4 + |g|) relative and one rounding of 2^-24."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import comm_overlapped_gemm_gb300 as tdx

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def ints(g, *shape, dtype=BF):
    return torch.randint(-4, 5, shape, generator=g, device="cuda", dtype=torch.int8).float().to(dtype)


# 16 tiles (8 of e4m3) of few rows: 4 to 8 CTAs share each, 16, 32 and 64 slices of K or more apiece: sums of 2, 3 and 5
# segments of 14 slices
@pytest.mark.parametrize("slices", [128, 256, 512])
@pytest.mark.parametrize("M", [1, 16, 128])
@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("grouped", [False, True])
def test_gated_fp32_results_on_clusters(slices, M, dtype, grouped):
    g = torch.Generator(device="cuda").manual_seed(slices + M)
    K, N = slices * (64 if dtype == BF else 128), 2048
    A, B = ints(g, M, K, dtype=dtype), ints(g, K, N, dtype=dtype)
    alpha = 2.0 ** -9
    want = (A.double() @ B.double()) * alpha
    gate, up = want[:, :N // 2], want[:, N // 2:]
    y = gate * torch.sigmoid(gate) * up
    lim = (2.0 ** -21 * (4 + gate.abs()) + 2.0 ** -24) * y.abs() + 2.0 ** -126
    code = tdx.TDX_BF16 if dtype == BF else tdx.TDX_FP8_E4M3
    o = tdx.make_linear_opts(out_dtype=tdx.TDX_FP32, act=tdx.TDX_ACT_SWIGLU, alpha=alpha)
    if grouped:
        B, off = torch.stack([torch.zeros_like(B), B]), torch.tensor([0, 0, M], dtype=torch.int32, device="cuda")
    first = None
    for _ in range(30):
        C, z = torch.empty(M, N // 2, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
        if grouped:
            tdx.check(tdx.tdx_grouped_gemm(A, off, B, None, None, C, z, M, K, N, 2, code, o))
        else:
            tdx.check(tdx.tdx_linear(A, B, None, None, None, C, z, M, K, N, code, o))
        assert torch.equal(z, want.float().to(BF))
        assert bool(((C.double() - y).abs() <= lim).all())
        first = C if first is None else first
        assert torch.equal(C, first)
