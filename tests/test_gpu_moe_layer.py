"""The mixture-of-experts layer of examples/moe_layer.py (norm, router, dispatch, activation, combine)
against the fp64 oracles, step by step on the values the step before left on the device, and as a
whole in a replayed CUDA graph."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import comm_overlapped_gemm_gb300 as tdx
from oracle import moe as MO
from oracle import reference as R
from oracle import rows as RO
from gpu_util import host_bits

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("W,T,H,I,E,k,dtype,route", [
    (2, 40, 128, 64, 16, 4, "bf16", {}),
    (4, 33, 256, 128, 16, 2, "bf16", dict(score=1, n_group=4, topk_group=2, group_top=2, scale=2.5)),
    (2, 64, 256, 128, 8, 2, "e4m3", dict(score=1, renorm=0)),
])
def test_layer_step_by_step(W, T, H, I, E, k, dtype, route):
    layer, x, residual = example().random_layer(W, T, H, I, E, k, dtype, seed=W, **route)
    out, h = layer.forward(x, residual)
    layer.status()
    wh, _, wy = RO.rmsnorm(f64(x), f64(residual), f64(layer.norm), 1e-6)
    assert np.abs(f64(h) - wh).max() <= 2.0 ** -8 * np.abs(wh).max()
    assert (np.abs(f64(layer.y) - wy) <= 2.0 ** -7 * np.abs(wy) + 1e-6).all()
    logits = f64(layer.y) @ f64(layer.router)
    assert np.abs(f64(layer.logits) - logits).max() <= 1e-4 * np.abs(logits).max()
    ids, gates, margin = RO.route(f64(layer.logits), k, "sigmoid" if route.get("score") else "softmax",
                                  None if layer.bias is None else f64(layer.bias), route.get("n_group", 1),
                                  route.get("topk_group", 1), route.get("group_top", 1), bool(route.get("renorm", 1)),
                                  route.get("scale", 1.0))
    clear = margin > 2.0 ** -19
    assert clear.mean() >= 0.9
    got_ids = layer.idx.cpu().numpy()
    assert np.array_equal(got_ids[clear], ids[clear])
    assert np.allclose(f64(layer.gates)[clear], gates[clear], rtol=1e-5)
    assert np.array_equal(layer.counts.cpu().numpy(), np.bincount(got_ids.ravel(), minlength=E))
    topk = [a for a in got_ids.reshape(W, T, k)]
    if dtype == "e4m3":
        codes = layer.q.view(torch.uint8).cpu().numpy().reshape(W, T, H)
        up = layer.up.view(torch.uint8).cpu().numpy()
        Y, (_, _, dest, _) = MO.moe_dispatch_gemm(list(codes), topk, up, E, "e4m3", None,
                                                  [layer.up_opts.scale_b[e] for e in range(E)])
        tol = 2.0 ** -7
    else:
        Y, (_, _, dest, _) = MO.moe_dispatch_gemm(list(host_bits(layer.y).reshape(W, T, H)), topk, host_bits(layer.up), E)
        tol = 2.0 ** -7
    assert np.array_equal(layer.dest.cpu().numpy().reshape(W, T, k), np.stack(dest))
    assert np.abs(f64(layer.expert_in) - Y).max() <= tol * np.abs(Y).max()
    scale = None
    if dtype == "e4m3":
        scale = np.empty(W * T * k)
        scale[np.stack(dest).reshape(-1)] = np.repeat(f64(layer.q_scale), k)
    act = RO.swiglu(f64(layer.expert_in), scale)
    assert (np.abs(f64(layer.expert_act) - act) <= 2.0 ** -7 * np.abs(act) + 1e-6).all()
    want = np.concatenate(MO.moe_gemm_combine(host_bits(layer.expert_act), topk, host_bits(layer.down),
                                              list(layer.gates.cpu().numpy().reshape(W, T, k)), E, z_dtype="bf16"))
    assert np.abs(f64(out) - want).max() <= 1e-2 * np.abs(want).max()
    if dtype == "e4m3":
        # the whole in higher precision: what quantising tokens and weights costs stays small
        y = wy
        for s in range(W):
            for t in range(0, T, 17):
                r = s * T + t
                o = np.zeros(H)
                for j in range(k):
                    e = got_ids[r, j]
                    w = R.decode_e4m3(up[e]) * layer.up_opts.scale_b[e]
                    o += float(layer.gates[r, j]) * (RO.swiglu((y[r] @ w)[None])[0] @ f64(layer.down[e]))
                assert np.abs(f64(out)[r] - o).max() <= 0.15 * np.abs(o).max()


def test_layer_in_a_graph_and_two_layers_in_a_row():
    mod = example()
    layer, x, residual = mod.random_layer(4, 64, 256, 128, 16, 4, "bf16", seed=5)
    second, _, _ = mod.random_layer(4, 64, 256, 128, 16, 4, "bf16", seed=6)
    out, h = layer.forward(x, residual)
    out2, h2 = second.forward(out, h)
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, h, out2, h2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, r = layer.forward(x, residual)
        second.forward(o, r)
    for _ in range(3):
        for t in (out, h, out2, h2, layer.idx, second.gates):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        layer.status()
        second.status()
        assert all(torch.equal(a, b) for a, b in zip((out, h, out2, h2), want))
    # other inputs in the same buffers
    x.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out2, want[2])


def test_experts_and_router_take_one_norm():
    """The codes for the experts are those of the norm that the router's bf16 tokens come from (of the
    unrounded x + residual), also where a layer's own outputs are its next inputs."""
    layer, x, residual = example().random_layer(2, 64, 256, 128, 8, 2, "e4m3", seed=3, score=1, renorm=0)
    n, H = x.shape
    for _ in range(2):
        q, scale = torch.empty_like(layer.q), torch.empty_like(layer.q_scale)
        tdx.check(tdx.tdx_rmsnorm(x, residual, layer.norm, None, q, scale, None, n, H, 0, layer.quant_opts))
        want = x.double() + residual.double()
        want = want / (want.square().mean(1, keepdim=True) + 1e-6).sqrt() * layer.norm.double()
        out, h = layer.forward(x, residual)
        layer.status()
        assert torch.equal(layer.q.view(torch.uint8), q.view(torch.uint8)) and torch.equal(layer.q_scale, scale)
        near = (layer.y.double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8)
        assert bool(near.all())
        x, residual = out, h
