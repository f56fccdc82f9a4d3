"""Calls without rows, whose row tensors are empty and have no address: checked on the host, without a GPU. Addresses
are fake, and no call here gets as far as a launch."""
import pytest

from test_boundary import FAKE, _lib_or_skip


@pytest.fixture(scope="module")
def tdx():
    return _lib_or_skip()


@pytest.mark.parametrize("dtype", [0, 1])
def test_products(tdx, dtype):
    ok, inv = tdx.TDX_OK, tdx.TDX_ERR_INVALID_ARG
    assert tdx.tdx_linear(0, FAKE, FAKE, 0, 0, 0, 0, 0, 64, 128, dtype, None, 0) == ok
    assert tdx.tdx_linear(0, 0, 0, 0, 0, 0, 0, 0, 64, 128, dtype, None, 0) == inv       # B has K rows
    assert tdx.tdx_grouped_gemm(0, FAKE, FAKE, 0, 0, 0, 0, 0, 64, 128, 3, dtype, None, 0) == ok
    assert tdx.tdx_grouped_gemm(0, 0, FAKE, 0, 0, 0, 0, 0, 64, 128, 3, dtype, None, 0) == inv   # offsets have E + 1


def test_products_gradients(tdx):
    ok, inv = tdx.TDX_OK, tdx.TDX_ERR_INVALID_ARG
    assert tdx.tdx_linear_bwd(0, 0, FAKE, 0, 0, 0, 0, 64, 128, 0, None, 0) == ok
    assert tdx.tdx_grouped_gemm_bwd(0, 0, FAKE, FAKE, 0, 0, 0, 64, 128, 3, 0, None, 0) == ok
    assert tdx.tdx_linear_bwd(0, 0, FAKE, 0, 0, 0, 1, 64, 128, 0, None, 0) == inv
    for act in range(6):
        o = tdx.make_linear_opts(act=act)
        assert tdx.tdx_linear_act_bwd(0, 0, 0, 0, 0, 0, 128, 0, o, 0, workspace_bytes=0) == ok


def test_combine(tdx):
    ok, inv = tdx.TDX_OK, tdx.TDX_ERR_INVALID_ARG
    assert tdx.tdx_moe_combine(FAKE, 0, 0, 0, 8, 0, 64, 2, 0, None, 0) == ok
    assert tdx.tdx_moe_combine(0, 0, 0, 0, 0, 0, 64, 2, 0, None, 0) == ok
    assert tdx.tdx_moe_combine(0, 0, 0, 0, 8, 0, 64, 2, 0, None, 0) == inv              # 8 rows of Z
    assert tdx.tdx_moe_combine_bwd(0, FAKE, 0, 0, FAKE, 0, 8, 0, 64, 2, 0, None, 0) == ok
    assert tdx.tdx_moe_combine_bwd(0, 0, 0, 0, 0, 0, 0, 0, 64, 2, 0, None, 0) == ok
    assert tdx.tdx_moe_combine_bwd(FAKE, 0, FAKE, FAKE, 0, FAKE, 8, 4, 64, 2, 0, None, 0) == inv


def test_row_wise_operators(tdx):
    ok, inv = tdx.TDX_OK, tdx.TDX_ERR_INVALID_ARG
    assert tdx.tdx_rmsnorm(0, 0, FAKE, 0, 0, 0, 0, 0, 64, 0, None, 0) == ok
    assert tdx.tdx_rmsnorm(0, 0, 0, 0, 0, 0, 0, 0, 64, 0, None, 0) == inv                # the weight has no rows
    assert tdx.tdx_rmsnorm_bwd(0, 0, FAKE, 0, 0, 0, 0, FAKE, 0, 64, 0, None, 0, workspace_bytes=1 << 30) == inv
    assert tdx.tdx_moe_route(0, 0, 0, 0, FAKE, 0, 64, 8, 0, None, 0) == ok
    assert tdx.tdx_moe_route_bwd(0, 0, 0, 0, 0, 64, 8, 0, None, 0) == ok
    assert tdx.tdx_swiglu(0, 0, 0, 0, 0, 64, 0, None, 0) == ok
    assert tdx.tdx_swiglu(0, 0, 0, 0, 0, 64, 0, tdx.make_act_opts(topk=8), 0) == ok
    assert tdx.tdx_swiglu_bwd(0, 0, 0, 0, 64, 0, None, 0) == ok
