"""GPU tests of calls whose row tensors are empty: what the formulas leave is zeroed, nothing else is written."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import comm_overlapped_gemm_gb300 as tdx

BF, F32 = torch.bfloat16, torch.float32


def empty(*shape, dtype=BF):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    assert t.data_ptr() == 0
    return t


def full(*shape, dtype=F32):
    return torch.full(shape, 3.0, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dw", [F32, BF])
@pytest.mark.parametrize("acc", [0, 1])
@pytest.mark.parametrize("K,N", [(64, 128), (2048, 4096)])
def test_weight_gradients(dw, acc, K, N):
    o = tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32 if dw == F32 else tdx.TDX_BF16, accumulate=acc)
    want = 3.0 if acc else 0.0
    dB, B = full(K, N, dtype=dw), full(K, N, dtype=BF)
    tdx.check(tdx.tdx_linear_bwd(empty(0, N), empty(0, K), B, empty(0, K), empty(0, K), dB, 0, K, N, 0, o))
    assert bool((dB == want).all())
    dB, B, off = full(3, K, N, dtype=dw), full(3, K, N, dtype=BF), torch.zeros(4, dtype=torch.int32, device="cuda")
    tdx.check(tdx.tdx_grouped_gemm_bwd(empty(0, N), empty(0, K), off, B, empty(0, K), dB, 0, K, N, 3, 0, o))
    assert bool((dB == want).all())


@pytest.mark.parametrize("act", range(6))
def test_bias_gradient(act):
    cols = 64 if act == 5 else 128
    o, db = tdx.make_linear_opts(act=act), full(128)
    ws = torch.empty(tdx.tdx_linear_act_bwd_workspace_size(0, 128, 0, o), dtype=torch.uint8, device="cuda")
    tdx.check(tdx.tdx_linear_act_bwd(empty(0, cols), empty(0, 128), empty(0, 128), db, ws, 0, 128, 0, o))
    assert bool((db == 0).all())


def test_forward_products():
    B = full(2, 64, 128, dtype=BF)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    tdx.check(tdx.tdx_linear(empty(0, 64), B, None, empty(0, 128), empty(0, dtype=F32), empty(0, 128), empty(0, 128), 0,
                             64, 128, 0))
    tdx.check(tdx.tdx_grouped_gemm(empty(0, 64), off, B, empty(0, dtype=F32), None, empty(0, 128), None, 0, 64, 128, 2, 0))
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_combine(dtype):
    code = tdx.TDX_BF16 if dtype == BF else tdx.TDX_FP32
    T, H, k = 5, 64, 2
    dest, gates = torch.zeros(T, k, dtype=torch.int32, device="cuda"), full(T, k)
    out, dg, Z = full(T, H, dtype=BF), full(T, k), empty(0, H, dtype=dtype)
    tdx.check(tdx.tdx_moe_combine(Z, dest, gates, out, 0, T, H, k, code))
    assert bool((out == 0).all())
    dout = full(T, H, dtype=dtype)
    tdx.check(tdx.tdx_moe_combine_bwd(dout, Z, dest, gates, empty(0, H, dtype=dtype), dg, 0, T, H, k, code))
    assert bool((dg == 0).all())
    none, Z = torch.empty(0, k, dtype=torch.int32, device="cuda"), full(4, H, dtype=dtype)
    tdx.check(tdx.tdx_moe_combine(Z, none, empty(0, k, dtype=F32), empty(0, H), 4, 0, H, k, code))
    tdx.check(tdx.tdx_moe_combine_bwd(empty(0, H, dtype=dtype), Z, none, None, Z, empty(0, k, dtype=F32), 4, 0, H, k, code))
    assert bool((Z == 3).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_gradient(dtype):
    code, H = tdx.TDX_BF16 if dtype == BF else tdx.TDX_FP32, 64
    e, dw = empty(0, H, dtype=dtype), full(H)
    ws = torch.empty(tdx.tdx_rmsnorm_bwd_workspace_size(0, H, code), dtype=torch.uint8, device="cuda")
    tdx.check(tdx.tdx_rmsnorm_bwd(e, e, full(H, dtype=dtype), empty(0, dtype=F32), e, e, dw, ws, 0, H, code))
    assert bool((dw == 0).all())


def test_dispatch_without_tokens():
    """The offsets of no rows, and what follows them: zeros."""
    H, F, E, k = 64, 128, 8, 2
    B, off = full(E, H, F, dtype=BF), torch.full((E + 1,), 9, dtype=torch.int32, device="cuda")
    o = tdx.make_opts()
    ws = torch.empty(tdx.tdx_moe_workspace_size(1, 0, H, F, E, k, 0, o), dtype=torch.uint8, device="cuda")
    tdx.check(tdx.tdx_workspace_init(ws))
    ids = empty(0, k, dtype=torch.int32)
    tdx.check(tdx.tdx_moe_dispatch_gemm([empty(0, H)], [ids], B, empty(0, F), ids, off, ws, 1, 0, H, F, E, k, 0, o))
    assert bool((off == 0).all())
    dB = full(E, H, F)
    tdx.check(tdx.tdx_grouped_gemm_bwd(empty(0, F), empty(0, H), off, B, empty(0, H), dB, 0, H, F, E, 0,
                                       tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32)))
    assert bool((dB == 0).all())


@pytest.mark.parametrize("K", [0, 64])
def test_all_gather_without_rows_or_columns(K):
    """K = 0: C is zeroed."""
    W, M, N = 2, 64, 64
    C = full(W * M, N, dtype=BF)
    ws = torch.empty(tdx.tdx_workspace_size(tdx.OP_AG, W, M, K, N, 0), dtype=torch.uint8, device="cuda")
    tdx.check(tdx.tdx_workspace_init(ws))
    if K == 0:
        tdx.check(tdx.tdx_ag_gemm([empty(M, 0)] * W, empty(0, N), C, ws, W, M, 0, N, 0))
        assert bool((C == 0).all())
    else:
        tdx.check(tdx.tdx_ag_gemm([empty(0, K)] * W, full(K, N, dtype=BF), empty(0, N), ws, W, 0, K, N, 0))
    torch.cuda.synchronize()
