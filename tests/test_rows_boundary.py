"""Host-side checks of the row-wise operators' arguments, without a GPU: every pointer is a fake
address that is never dereferenced, and a call that got as far as a launch would return
TDX_ERR_CUDA instead of the code expected here."""
import ctypes
import math
import os

import pytest

from test_boundary import FAKE, _lib_or_skip

HUGE = 1 << 40


@pytest.fixture(scope="module")
def tdx():
    return _lib_or_skip()


def test_defaults(tdx):
    n, r, a = tdx.tdx_norm_opts_default(), tdx.tdx_route_opts_default(), tdx.tdx_act_opts_default()
    assert (n.out_dtype, n.eps, n.out_scale) == (tdx.TDX_BF16, pytest.approx(1e-6), 1.0)
    assert (n.ld_x, n.ld_residual, n.ld_h, n.ld_y) == (0, 0, 0, 0)
    assert (r.score, r.n_group, r.topk_group, r.group_top, r.renorm, r.scale, r.ld_logits) == (0, 1, 1, 1, 1, 1.0, 0)
    assert (a.out_dtype, a.out_scale, a.topk, a.ld_y, a.ld_out) == (tdx.TDX_BF16, 1.0, 0, 0, 0)
    for name in ("tdx_norm_opts_default", "tdx_route_opts_default", "tdx_act_opts_default"):
        assert getattr(tdx._lib, name)(None) == tdx.TDX_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        tdx.make_norm_opts(epsilon=1.0)


def test_option_structs_match_the_header(tdx, tmp_path):
    """The ctypes structures have the C structures' sizes and field offsets."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = [tdx.tdx_norm_opts, tdx.tdx_route_opts, tdx.tdx_act_opts]
    src = ['#include <stdio.h>', '#include <stddef.h>', '#include "tdx.h"', "int main(void) {"]
    want = []
    for s in structs:
        src.append(f'printf("%zu\\n", sizeof({s.__name__}));')
        want.append(ctypes.sizeof(s))
        for f in s._fields_:
            src.append(f'printf("%zu\\n", offsetof({s.__name__}, {f[0]}));')
            want.append(getattr(s, f[0]).offset)
    (tmp_path / "o.c").write_text("\n".join(src) + "return 0; }\n")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run([cc, "-std=c99", "-I", inc, str(tmp_path / "o.c"), "-o", str(tmp_path / "o")], check=True)
    got = subprocess.run([str(tmp_path / "o")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == want


def norm(tdx, x=FAKE, r=FAKE, w=FAKE, h=FAKE, y=FAKE, rs=0, rstd=FAKE, T=4, H=64, dtype=0, **kw):
    return tdx.tdx_rmsnorm(x, r, w, h, y, rs, rstd, T, H, dtype, tdx.make_norm_opts(**kw), stream=0)


def test_rmsnorm_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED
    for bad in ("x", "w", "y"):
        assert norm(tdx, **{bad: 0}) == inv
    assert norm(tdx, r=0) == inv                       # h_out without a residual
    assert norm(tdx, T=-1) == inv and norm(tdx, H=0) == inv and norm(tdx, H=-8) == inv
    assert norm(tdx, dtype=7) == inv and norm(tdx, out_dtype=7) == inv and norm(tdx, out_dtype=-1) == inv
    assert norm(tdx, dtype=tdx.TDX_FP8_E4M3) == uns
    for eps in (-1e-6, math.nan, math.inf):
        assert norm(tdx, eps=eps) == inv
    for s in (0.0, -1.0, math.nan, math.inf, 1e-40):
        assert norm(tdx, out_dtype=1, out_scale=s) == inv
    assert norm(tdx, H=(1 << 28) + 8) == uns
    assert norm(tdx, rs=FAKE) == inv                   # row scales without an e4m3 output
    assert norm(tdx, H=60) == ali                      # 120-byte rows
    assert norm(tdx, H=24, out_dtype=1) == ali         # 24-byte e4m3 rows
    for bad in ("x", "r", "w", "h", "y"):
        assert norm(tdx, **{bad: FAKE + 8}) == ali
    assert norm(tdx, rstd=FAKE + 2) == ali and norm(tdx, rs=FAKE + 2, out_dtype=1) == ali
    for ld in ("ld_x", "ld_residual", "ld_h", "ld_y"):
        assert norm(tdx, **{ld: 56}) == inv
        assert norm(tdx, **{ld: -64}) == inv
        assert norm(tdx, **{ld: 68}) == ali
        assert norm(tdx, **{ld: 1 << 62}) == inv
    assert norm(tdx, T=0) == tdx.TDX_OK                # nothing to launch


def test_rmsnorm_bwd_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED

    def bwd(dy=FAKE, h=FAKE, w=FAKE, rstd=FAKE, dr=0, dx=FAKE, dw=FAKE, ws=FAKE, wsb=HUGE, T=4, H=64, dtype=0, **kw):
        return tdx.tdx_rmsnorm_bwd(dy, h, w, rstd, dr, dx, dw, ws, T, H, dtype, tdx.make_norm_opts(**kw), stream=0,
                                   workspace_bytes=wsb)

    for bad in ("dy", "h", "w", "rstd", "dx", "dw"):
        assert bwd(**{bad: 0}) == inv
    for bad in ("dy", "h", "w", "dr", "dx", "dw"):
        assert bwd(**{bad: FAKE + 8}) == ali
    assert bwd(rstd=FAKE + 2) == ali and bwd(H=60) == ali
    assert bwd(T=-1) == inv and bwd(H=0) == inv and bwd(dtype=1) == uns and bwd(dtype=9) == inv
    assert bwd(H=32768 + 8) == uns
    need = tdx.tdx_rmsnorm_bwd_workspace_size(4, 64, 0)
    assert need >= 64 * 4
    assert bwd(ws=0) == tdx.TDX_ERR_WORKSPACE and bwd(ws=FAKE + 64) == tdx.TDX_ERR_WORKSPACE
    assert bwd(wsb=need - 1) == tdx.TDX_ERR_WORKSPACE
    for ld in ("ld_x", "ld_residual", "ld_h", "ld_y"):
        assert bwd(**{ld: 56}) == inv and bwd(**{ld: 68}) == ali
    for args in ((-1, 64, 0), (4, 0, 0), (4, 64, 9)):
        with pytest.raises(tdx.TdxError):
            tdx.tdx_rmsnorm_bwd_workspace_size(*args)
    assert tdx._lib.tdx_rmsnorm_bwd_workspace_size(4, 64, 0, None) == inv
    assert tdx.tdx_rmsnorm_bwd_workspace_size(0, 64, 0) > 0


def test_route_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED

    def route(x=FAKE, b=0, idx=FAKE, g=FAKE, c=0, T=4, E=64, k=8, dtype=2, **kw):
        return tdx.tdx_moe_route(x, b, idx, g, c, T, E, k, dtype, tdx.make_route_opts(**kw), stream=0)

    def bwd(x=FAKE, idx=FAKE, dg=FAKE, dx=FAKE, T=4, E=64, k=8, dtype=2, **kw):
        return tdx.tdx_moe_route_bwd(x, idx, dg, dx, T, E, k, dtype, tdx.make_route_opts(**kw), stream=0)

    for bad in ("x", "idx", "g"):
        assert route(**{bad: 0}) == inv
    for bad in ("x", "idx", "dg", "dx"):
        assert bwd(**{bad: 0}) == inv
        assert bwd(**{bad: FAKE + 2}) == ali
    assert bwd(x=FAKE + 1, dtype=0) == ali
    for f in (route, bwd):
        assert f(T=-1) == inv and f(E=0) == inv and f(k=0) == inv and f(k=65) == inv and f(dtype=9) == inv
        assert f(E=513) == uns and f(k=17) == uns and f(dtype=1) == uns
        assert f(E=512, n_group=64) == uns
        assert f(score=2) == inv and f(renorm=2) == inv and f(scale=math.nan) == inv and f(scale=math.inf) == inv
        assert f(n_group=0) == inv and f(n_group=7) == inv and f(n_group=8, topk_group=9) == inv
        assert f(topk_group=0) == inv and f(group_top=0) == inv and f(group_top=3) == inv
        assert f(ld_logits=63) == inv and f(ld_logits=-1) == inv and f(ld_logits=1 << 62) == inv
        assert f(T=0) == tdx.TDX_OK
    assert route(n_group=16, topk_group=1) == inv      # 8 of 4 experts
    for bad in ("x", "b", "idx", "g", "c"):
        assert route(**{bad: FAKE + 2}) == ali
    assert route(x=FAKE + 1, dtype=0) == ali


def test_swiglu_refusals(tdx):
    inv, ali, uns = tdx.TDX_ERR_INVALID_ARG, tdx.TDX_ERR_ALIGNMENT, tdx.TDX_ERR_UNSUPPORTED

    def act(y=FAKE, out=FAKE, rs=0, dest=0, R=8, I=64, dtype=0, **kw):
        return tdx.tdx_swiglu(y, out, rs, dest, R, I, dtype, tdx.make_act_opts(**kw), stream=0)

    def bwd(y=FAKE, do=FAKE, dy=FAKE, R=8, I=64, dtype=0, **kw):
        return tdx.tdx_swiglu_bwd(y, do, dy, R, I, dtype, tdx.make_act_opts(**kw), stream=0)

    assert act(y=0) == inv and act(out=0) == inv
    for bad in ("y", "do", "dy"):
        assert bwd(**{bad: 0}) == inv and bwd(**{bad: FAKE + 8}) == ali
    for f in (act, bwd):
        assert f(R=-1) == inv and f(I=0) == inv and f(dtype=5) == inv and f(dtype=1) == uns and f(I=60) == ali
        assert f(ld_y=120) == inv and f(ld_y=132) == ali and f(ld_out=56) == inv and f(ld_out=68) == ali
        assert f(R=0) == tdx.TDX_OK
        assert f(I=1 << 30) == inv
    assert act(I=24, out_dtype=1) == ali and act(out_dtype=9) == inv
    for s in (0.0, -2.0, math.nan, math.inf):
        assert act(out_dtype=1, out_scale=s) == inv
    assert act(topk=-1) == inv
    assert act(topk=2, rs=FAKE) == inv and act(topk=2, dest=FAKE) == inv and act(dest=FAKE, rs=FAKE) == inv
    assert act(topk=3, rs=FAKE, dest=FAKE) == inv      # 8 rows are no whole number of tokens
    assert act(topk=2, rs=FAKE + 2, dest=FAKE) == ali and act(topk=2, rs=FAKE, dest=FAKE + 2) == ali
    assert act(out=FAKE + 8) == ali and act(y=FAKE + 8) == ali


def test_first_stream_from_two_threads(tdx, monkeypatch):
    """While one thread looks torch's calls up for the first time, another may ask for the stream at any
    point: here after every bytecode of the first one's way."""
    import sys
    import torch
    for name, value in (("_cuda_getCurrentRawStream", lambda device: 4096 + device), ("_cuda_getDevice", lambda: 3)):
        monkeypatch.setattr(torch._C, name, value, raising=False)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(tdx, "_raw_stream", None)
    monkeypatch.setattr(tdx, "_device", None)
    seen, events = [], getattr(sys, "monitoring", None)
    if events is None:
        pytest.skip("no events of single instructions before Python 3.12")

    def other(code, offset):
        if tdx._raw_stream is not None:
            seen.append(tdx._stream(None))

    events.use_tool_id(events.DEBUGGER_ID, "two threads")
    try:
        events.register_callback(events.DEBUGGER_ID, events.events.INSTRUCTION, other)
        events.set_local_events(events.DEBUGGER_ID, tdx._first_stream.__code__, events.events.INSTRUCTION)
        first = tdx._stream(None)
    finally:
        events.set_local_events(events.DEBUGGER_ID, tdx._first_stream.__code__, 0)
        events.free_tool_id(events.DEBUGGER_ID)
    assert first == 4099 and seen and set(seen) == {4099}


@pytest.mark.parametrize("what", ["abc", b"abc", 1.5, [1], (1, 2), object()])
def test_what_is_no_tensor_and_no_address_is_refused(tdx, what):
    """ctypes would take text and bytes for the addresses of their characters."""
    with pytest.raises((AttributeError, TypeError)):
        norm(tdx, x=what, T=0)
    with pytest.raises((AttributeError, TypeError)):
        tdx.tdx_swiglu(FAKE, FAKE, None, what, 0, 64, 0, stream=0)
    with pytest.raises((AttributeError, TypeError)):
        tdx.tdx_ag_gemm([what], FAKE, FAKE, FAKE, 1, 128, 64, 64, 0, stream=0, workspace_bytes=0)
