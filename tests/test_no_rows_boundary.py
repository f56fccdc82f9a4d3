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


def test_collectives(tdx):
    ok, inv, ws = tdx.TDX_OK, tdx.TDX_ERR_INVALID_ARG, dict(stream=0, workspace_bytes=1 << 40)

    def ag(shard, B, C, m, k, n):
        return tdx.tdx_ag_gemm([shard] * 2, B, C, FAKE, 2, m, k, n, 0, None, **ws)

    assert ag(0, FAKE, 0, 0, 64, 64) == ok and ag(FAKE, 0, 0, 64, 64, 0) == ok and ag(0, 0, 0, 0, 0, 0) == ok
    assert ag(0, FAKE, FAKE, 64, 64, 64) == inv and ag(FAKE, 0, FAKE, 64, 64, 64) == inv
    assert ag(0, 0, 0, 0, 64, 64) == inv and ag(0, 0, 0, 64, 0, 64) == inv      # B has K rows, C has M
    for f in (tdx.tdx_gemm_rs, tdx.tdx_gemm_ar):
        def rs(A, B, out, m, k, n):
            return f([A] * 2, [B] * 2, [out] * 2, FAKE, 2, m, k, n, 0, None, **ws)

        assert rs(0, FAKE, 0, 0, 64, 64) == ok and rs(FAKE, 0, 0, 256, 64, 0) == ok
        assert rs(0, FAKE, FAKE, 256, 64, 64) == inv and rs(0, 0, 0, 0, 64, 64) == inv
        assert rs(FAKE, FAKE, 0, 256, 64, 64) == inv


def test_expert_collectives(tdx):
    ok, inv, ws = tdx.TDX_OK, tdx.TDX_ERR_INVALID_ARG, dict(stream=0, workspace_bytes=1 << 40)

    def dispatch(p, T, B=FAKE):
        return tdx.tdx_moe_dispatch_gemm([p], [p], B, p, p, 0, FAKE, 1, T, 64, 128, 8, 2, 0, None, **ws)

    def combine(p, T, B=FAKE):
        return tdx.tdx_moe_gemm_combine(p, [p], B, [p], [p], FAKE, 1, T, 128, 64, 8, 2, 0, None, **ws)

    for call in (dispatch, combine):
        assert call(0, 0) == ok and call(0, 4) == inv and call(0, 0, B=0) == inv
