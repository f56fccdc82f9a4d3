"""A mixture-of-experts layer of a transformer on this library's calls, for W ranks of T tokens each.

    norm       tdx_rmsnorm             h = x + residual, y = norm(h)
    router     tdx_ag_gemm (fp32 C)    logits of all ranks' tokens, then tdx_moe_route
    experts    tdx_moe_dispatch_gemm   tokens to their experts and the gate/up product
               tdx_swiglu              the gated activation
               tdx_moe_gemm_combine    the down product and the gates' sum on the source rank

The output and h go into the next layer's tdx_rmsnorm as x and residual. With dtype "e4m3" the expert
tokens are quantised one by one (tdx_rmsnorm's row scales), multiplied without scales, and scaled
back in front of the activation, which finds each row's token through the dispatch's `dest`.

Run ``python examples/moe_layer.py`` on a GPU for one layer at a decoding size, captured in a CUDA graph.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import comm_overlapped_gemm_gb300 as tdx  # noqa: E402


class MoeLayer:
    """Weights, workspaces and buffers of one layer; ``forward`` allocates nothing.

    ``norm`` [H], ``router`` [H, E], ``bias`` [E] fp32 or None, ``up`` [E, H, 2 I] and ``down``
    [E, I, H]; all bf16 but the bias, ``up`` e4m3 with ``up_scale`` (E floats) for dtype "e4m3"."""

    def __init__(self, W, T, topk, norm, router, bias, up, down, dtype="bf16", up_scale=None, route=None, eps=1e-6):
        H, E = router.shape
        I = down.shape[1]
        self.W, self.T, self.H, self.E, self.I, self.k = W, T, H, E, I, topk
        self.norm, self.router, self.bias, self.up, self.down = norm, router, bias, up, down
        self.e4m3 = dtype == "e4m3"
        self.code = tdx.TDX_FP8_E4M3 if self.e4m3 else tdx.TDX_BF16
        n, dev = W * T, norm.device

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=dev)

        def workspace(nbytes):
            ws = empty(nbytes, dtype=torch.uint8)
            tdx.check(tdx.tdx_workspace_init(ws), "tdx_workspace_init")
            return ws

        self.h, self.y = empty(n, H), empty(n, H)
        self.q = empty(n, H, dtype=torch.float8_e4m3fn) if self.e4m3 else None
        self.q_scale = empty(n, dtype=torch.float32) if self.e4m3 else None
        self.logits = empty(n, E, dtype=torch.float32)
        self.idx = empty(n, topk, dtype=torch.int32)
        self.gates = empty(n, topk, dtype=torch.float32)
        self.counts = torch.zeros(E, dtype=torch.int32, device=dev)   # tokens per expert, added up over the calls
        self.dest = empty(n, topk, dtype=torch.int32)
        self.expert_in, self.expert_act = empty(n * topk, 2 * I), empty(n * topk, I)
        self.out = empty(n, H)
        self.norm_opts = tdx.make_norm_opts(eps=eps)
        self.quant_opts = tdx.make_norm_opts(eps=eps, out_dtype=tdx.TDX_FP8_E4M3)
        self.route_opts = tdx.make_route_opts(**(route or {}))
        self.act_opts = tdx.make_act_opts(topk=topk if self.e4m3 else 0)
        # epochs kept in the workspaces: one captured call replays in a graph
        self.gemm_opts = tdx.make_opts(epoch=tdx.TDX_EPOCH_DEVICE)
        self.logit_opts = tdx.make_opts(epoch=tdx.TDX_EPOCH_DEVICE, out_dtype=tdx.TDX_FP32)
        self.up_opts = tdx.make_opts(epoch=tdx.TDX_EPOCH_DEVICE, scale_b=up_scale) if self.e4m3 else self.gemm_opts
        self.ws_router = workspace(tdx.tdx_workspace_size(tdx.OP_AG, W, T, H, E, tdx.TDX_BF16, self.logit_opts))
        self.ws_up = workspace(tdx.tdx_moe_workspace_size(W, T, H, 2 * I, E, topk, self.code, self.up_opts))
        self.ws_down = workspace(tdx.tdx_moe_combine_workspace_size(W, T, I, H, E, topk, tdx.TDX_BF16, self.gemm_opts))

    def ranks(self, t):
        return list(t.view(self.W, self.T, -1))

    def forward(self, x, residual, stream=None):
        """x, residual: [W * T, H] bf16, rank after rank. Returns (out, h)."""
        W, T, H, E, I, k, n = self.W, self.T, self.H, self.E, self.I, self.k, self.W * self.T
        bf16 = tdx.TDX_BF16
        tokens = self.y
        if self.e4m3:
            # the same norm as codes, before h takes the place of a residual that is this layer's own
            tokens = self.q
            tdx.check(tdx.tdx_rmsnorm(x, residual, self.norm, None, self.q, self.q_scale, None, n, H, bf16,
                                      self.quant_opts, stream), "tdx_rmsnorm")
        tdx.check(tdx.tdx_rmsnorm(x, residual, self.norm, self.h, self.y, None, None, n, H, bf16, self.norm_opts, stream),
                  "tdx_rmsnorm")
        tdx.check(tdx.tdx_ag_gemm(self.ranks(self.y), self.router, self.logits, self.ws_router, W, T, H, E, bf16,
                                  self.logit_opts, stream), "tdx_ag_gemm")
        tdx.check(tdx.tdx_moe_route(self.logits, self.bias, self.idx, self.gates, self.counts, n, E, k, tdx.TDX_FP32,
                                    self.route_opts, stream), "tdx_moe_route")
        tdx.check(tdx.tdx_moe_dispatch_gemm(self.ranks(tokens), self.ranks(self.idx), self.up, self.expert_in, self.dest,
                                            None, self.ws_up, W, T, H, 2 * I, E, k, self.code, self.up_opts, stream),
                  "tdx_moe_dispatch_gemm")
        tdx.check(tdx.tdx_swiglu(self.expert_in, self.expert_act, self.q_scale, self.dest if self.e4m3 else None, n * k, I,
                                 bf16, self.act_opts, stream), "tdx_swiglu")
        tdx.check(tdx.tdx_moe_gemm_combine(self.expert_act, self.ranks(self.idx), self.down, self.ranks(self.gates),
                                           self.ranks(self.out), self.ws_down, W, T, I, H, E, k, bf16, self.gemm_opts,
                                           stream), "tdx_moe_gemm_combine")
        return self.out, self.h

    def status(self):
        """Raise if a call met an error on the device (synchronises)."""
        for ws in (self.ws_router, self.ws_up, self.ws_down):
            st, detail = tdx.tdx_read_device_status(ws)
            if st != tdx.TDX_OK:
                raise tdx.TdxError(st, f"device status {detail}")


def random_layer(W, T, H, I, E, topk, dtype="bf16", seed=0, **route):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)

    up, up_scale = randn(E, H, 2 * I, std=H ** -0.5), None
    if dtype == "e4m3":
        up_scale = [float(s) for s in up.float().abs().amax(dim=(1, 2)) / 448.0]
        up = torch.stack([(w.float() / s).to(torch.float8_e4m3fn) for w, s in zip(up, up_scale)])
    bias = None
    if route.get("score") == tdx.TDX_SCORE_SIGMOID:
        bias = randn(E, std=0.05).float()
    layer = MoeLayer(W, T, topk, 1.0 + randn(H, std=0.1), randn(H, E, std=H ** -0.5), bias, up,
                     randn(E, I, H, std=I ** -0.5), dtype, up_scale, route)
    return layer, randn(W * T, H), randn(W * T, H)


def main():
    W, T, H, I, E, topk = 8, 128, 7168, 1024, 64, 8
    for dtype in ("bf16", "e4m3"):
        layer, x, residual = random_layer(W, T, H, I, E, topk, dtype)
        layer.forward(x, residual)
        layer.status()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward(x, residual)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for _ in range(3):
            graph.replay()
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        layer.status()
        print(f"{dtype}: {W} x {T} tokens, {H} wide, {topk} of {E} experts of {I}: {start.elapsed_time(end) / 20 * 1e3:.0f} us a layer")


if __name__ == "__main__":
    main()
