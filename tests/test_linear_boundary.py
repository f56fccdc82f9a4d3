"""Host-side checks of the arguments of the products without communication, without a GPU: every pointer
is a fake address that is never dereferenced, and a call that got as far as a launch would return
TDX_ERR_CUDA instead of the code expected here."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest

from test_boundary import FAKE, _lib_or_skip

HUGE = 1 << 40


@pytest.fixture(scope="module")
def tdx():
    return _lib_or_skip()


def test_defaults(tdx):
    o, c = tdx.tdx_linear_opts_default(), tdx.tdx_combine_opts_default()
    assert (o.out_dtype, o.act, o.alpha, o.out_scale, o.dw_dtype, o.accumulate) == (0, 0, 1.0, 1.0, 0, 0)
    assert (o.ld_a, o.ld_b, o.ld_c, o.ld_residual, o.ld_z, o.device_status) == (0, 0, 0, 0, 0, None)
    assert (c.out_dtype, c.ld_z, c.ld_out) == (0, 0, 0)
    for name in ("tdx_linear_opts_default", "tdx_combine_opts_default"):
        assert getattr(tdx._lib, name)(None) == tdx.TDX_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        tdx.make_linear_opts(beta=1.0)


def test_option_structs_match_the_header(tdx, tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "tdx.h"', "int main(void) {"]
    want = []
    for s in (tdx.tdx_linear_opts, tdx.tdx_combine_opts):
        src.append(f'printf("%zu\\n", sizeof({s.__name__}));')
        want.append(ctypes.sizeof(s))
        for f in s._fields_:
            src.append(f'printf("%zu\\n", offsetof({s.__name__}, {f[0]}));')
            want.append(getattr(s, f[0]).offset)
    for i, name in enumerate(("NONE", "RELU", "GELU", "GELU_TANH", "SILU", "SWIGLU")):
        src.append(f'printf("%d\\n", TDX_ACT_{name});')
        want.append(getattr(tdx, "TDX_ACT_" + name))
    (tmp_path / "o.c").write_text("\n".join(src) + "return 0; }\n")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-std=c99", "-I", inc, str(tmp_path / "o.c"), "-o", str(tmp_path / "o")], check=True)
    got = subprocess.run([str(tmp_path / "o")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == want


def linear(tdx, A=FAKE, B=FAKE, bias=0, res=0, rs=0, C=FAKE, z=0, M=4, K=64, N=128, dtype=0, **kw):
    return tdx.tdx_linear(A, B, bias, res, rs, C, z, M, K, N, dtype, tdx.make_linear_opts(**kw), stream=0)


def grouped(tdx, A=FAKE, off=FAKE, B=FAKE, rs=0, es=0, C=FAKE, z=0, R=4, K=64, N=128, E=3, dtype=0, **kw):
    return tdx.tdx_grouped_gemm(A, off, B, rs, es, C, z, R, K, N, E, dtype, tdx.make_linear_opts(**kw), stream=0)


def test_linear_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED
    for call, rows in ((linear, "M"), (grouped, "R")):
        for bad in ("A", "B", "C"):
            assert call(tdx, **{bad: 0}) == inv
            assert call(tdx, **{bad: FAKE + 8}) == ali
        assert call(tdx, z=FAKE + 8) == ali and call(tdx, rs=FAKE + 2) == ali
        assert call(tdx, **{rows: -1}) == inv and call(tdx, K=0) == inv and call(tdx, N=0) == inv and call(tdx, N=-8) == inv
        assert call(tdx, dtype=7) == inv and call(tdx, dtype=-1) == inv and call(tdx, dtype=tdx.TDX_FP32) == uns
        assert call(tdx, out_dtype=7) == inv and call(tdx, out_dtype=-1) == inv
        assert call(tdx, act=6) == inv and call(tdx, act=-1) == inv
        for a in (math.nan, math.inf, -math.inf):
            assert call(tdx, alpha=a) == inv
        for s in (0.0, -1.0, math.nan, math.inf, 1e-40):
            assert call(tdx, out_scale=s) == inv
        assert call(tdx, K=60) == ali and call(tdx, N=124) == ali
        assert call(tdx, dtype=1, K=72) == ali and call(tdx, dtype=1, N=136) == ali      # 16-byte rows of e4m3
        assert call(tdx, N=136, out_dtype=1) == ali                                       # of e4m3 outputs
        assert call(tdx, N=127, act=5) == inv and call(tdx, N=24, act=5) == ali           # halves of 12 columns
        assert call(tdx, dtype=1, N=48, act=5) == ali
        assert call(tdx, **{rows: (1 << 30) + 1}) == uns and call(tdx, K=(1 << 30) + 8) == uns
        for ld, least in (("ld_a", 64), ("ld_b", 128), ("ld_c", 128), ("ld_z", 128)):
            assert call(tdx, **{ld: least - 8}) == inv and call(tdx, **{ld: -least}) == inv
            assert call(tdx, **{ld: least + 4}) == ali
            assert call(tdx, **{ld: 1 << 62}) == inv
        assert call(tdx, ld_a=1 << 39) == uns and call(tdx, ld_b=1 << 39) == uns
        assert call(tdx, **{rows: 0}) == tdx.TDX_OK
        assert call(tdx, device_status=FAKE + 2) == ali
    assert linear(tdx, bias=FAKE + 8) == ali and linear(tdx, res=FAKE + 8) == ali
    assert linear(tdx, ld_residual=120) == inv and linear(tdx, ld_residual=132) == ali
    assert grouped(tdx, off=0) == inv and grouped(tdx, E=0) == inv and grouped(tdx, E=-1) == inv
    assert grouped(tdx, E=513) == uns and grouped(tdx, off=FAKE + 2) == ali and grouped(tdx, es=FAKE + 2) == ali
    assert grouped(tdx, ld_b=1 << 36) == uns        # experts 2^43 bytes apart


def test_linear_bwd_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED

    def lin(dz=FAKE, A=FAKE, B=FAKE, dA=FAKE, dB=FAKE, M=4, K=64, N=128, dtype=0, res=0, **kw):
        return tdx.tdx_linear_bwd(dz, A, B, res, dA, dB, M, K, N, dtype, tdx.make_linear_opts(**kw), stream=0)

    def grp(dz=FAKE, A=FAKE, B=FAKE, dA=FAKE, dB=FAKE, M=4, K=64, N=128, dtype=0, off=FAKE, E=2, **kw):
        return tdx.tdx_grouped_gemm_bwd(dz, A, off, B, dA, dB, M, K, N, E, dtype, tdx.make_linear_opts(**kw), stream=0)

    for call in (lin, grp):
        for bad in ("dz", "A", "B"):
            assert call(**{bad: 0}) == inv
        for bad in ("dz", "A", "B", "dA", "dB"):
            assert call(**{bad: FAKE + 8}) == ali
        assert call(dA=0, dB=0) == inv
        assert call(M=-1) == inv and call(K=0) == inv and call(N=0) == inv and call(dtype=9) == inv
        assert call(dtype=1) == uns and call(dtype=2) == uns and call(out_dtype=1) == uns and call(dw_dtype=1) == uns
        assert call(out_dtype=5) == inv and call(dw_dtype=5) == inv
        assert call(act=1) == inv and call(act=9) == inv
        assert call(accumulate=2) == inv and call(accumulate=-1) == inv and call(alpha=math.nan) == inv
        assert call(K=60) == ali and call(N=132) == ali
        for ld, least in (("ld_a", 64), ("ld_b", 128), ("ld_c", 64), ("ld_z", 128)):
            assert call(**{ld: least - 8}) == inv and call(**{ld: least + 4}) == ali
        assert call(device_status=FAKE + 2) == ali
        assert call(M=0, dB=0) == tdx.TDX_OK
    assert lin(res=FAKE, dA=0) == inv and lin(res=FAKE + 8) == ali and lin(res=FAKE, ld_residual=56) == inv
    assert grp(off=0) == inv and grp(E=0) == inv and grp(E=513) == uns and grp(off=FAKE + 2) == ali


def test_linear_act_bwd_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED

    def call(dy=FAKE, z=FAKE, dz=FAKE, db=FAKE, ws=FAKE, wsb=HUGE, M=4, N=128, dtype=0, **kw):
        kw.setdefault("act", tdx.TDX_ACT_SILU)
        return tdx.tdx_linear_act_bwd(dy, z, dz, db, ws, M, N, dtype, tdx.make_linear_opts(**kw), stream=0,
                                      workspace_bytes=wsb)

    assert call(dy=0) == inv and call(z=0) == inv and call(dz=0, db=0) == inv
    for bad in ("dy", "z", "dz", "db"):
        assert call(**{bad: FAKE + 8}) == ali
    assert call(M=-1) == inv and call(N=0) == inv and call(N=12) == ali and call(dtype=7) == inv
    assert call(dtype=1) == uns and call(dtype=2) == uns and call(N=1 << 29) == uns
    assert call(act=6) == inv and call(act=5, N=127) == inv and call(act=5, N=24) == ali
    need = tdx.tdx_linear_act_bwd_workspace_size(4, 128, 0, tdx.make_linear_opts(act=tdx.TDX_ACT_SILU))
    assert call(ws=0) == tdx.TDX_ERR_WORKSPACE and call(ws=FAKE + 64) == tdx.TDX_ERR_WORKSPACE
    assert call(wsb=need - 1) == tdx.TDX_ERR_WORKSPACE
    for ld in ("ld_c", "ld_z"):
        assert call(**{ld: 120}) == inv and call(**{ld: 132}) == ali
    assert call(M=0, db=0) == tdx.TDX_OK
    assert tdx._lib.tdx_linear_act_bwd_workspace_size(4, 128, 0, None, None) == inv
    with pytest.raises(tdx.TdxError):
        tdx.tdx_linear_act_bwd_workspace_size(-1, 128, 0)


def test_combine_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED

    def fwd(Z=FAKE, dest=FAKE, g=FAKE, out=FAKE, R=32, T=4, H=64, k=8, dtype=0, **kw):
        return tdx.tdx_moe_combine(Z, dest, g, out, R, T, H, k, dtype, tdx.make_combine_opts(**kw), stream=0)

    def bwd(dout=FAKE, Z=FAKE, dest=FAKE, g=FAKE, dZ=FAKE, dg=FAKE, R=32, T=4, H=64, k=8, dtype=0, **kw):
        return tdx.tdx_moe_combine_bwd(dout, Z, dest, g, dZ, dg, R, T, H, k, dtype, tdx.make_combine_opts(**kw), stream=0)

    for call in (fwd, bwd):
        assert call(dest=0) == inv and call(Z=0) == inv
        assert call(Z=FAKE + 8) == ali and call(dest=FAKE + 2) == ali and call(g=FAKE + 2) == ali
        assert call(R=-1) == inv and call(T=-1) == inv and call(H=0) == inv and call(k=0) == inv and call(k=17) == inv
        assert call(dtype=9) == inv and call(dtype=1) == uns and call(H=60) == ali
        for ld in ("ld_z", "ld_out"):
            assert call(**{ld: 56}) == inv and call(**{ld: 68}) == ali
        assert call(T=0) == tdx.TDX_OK
    assert fwd(out=0) == inv and fwd(out=FAKE + 8) == ali and fwd(out_dtype=1) == uns and fwd(out_dtype=9) == inv
    assert fwd(dtype=2, H=4) == ali            # 8-byte bf16 rows
    assert bwd(dout=0) == inv and bwd(dZ=0, dg=0) == inv and bwd(dout=FAKE + 8) == ali and bwd(dZ=FAKE + 8) == ali
    assert bwd(dg=FAKE + 2) == ali
