"""One training step of a mixture-of-experts block on this library's calls: forwards, then every gradient.

    forwards   tdx_rmsnorm, tdx_linear (router), tdx_moe_route, tdx_moe_dispatch_gemm, tdx_swiglu,
               tdx_moe_gemm_combine
    backwards  tdx_moe_combine_bwd         the experts' rows and the gates
               tdx_grouped_gemm_bwd        down product: its input and its weights
               tdx_swiglu_bwd
               tdx_grouped_gemm_bwd        gate/up product
               tdx_moe_combine             without gates: the dispatch's gradient, each token's rows added up
               tdx_moe_route_bwd, tdx_linear_bwd   router, its input gradient added to the experts'
               tdx_rmsnorm_bwd

The forward calls leave what the gradients need where they worked: the dispatched tokens in the dispatch's
workspace, the experts' outputs in the combine's. Run ``python examples/moe_training.py`` on a GPU for one step,
captured in a CUDA graph.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import comm_overlapped_gemm_gb300 as tdx  # noqa: E402

BF16 = tdx.TDX_BF16


class MoeBlock:
    """Weights (bf16: ``norm`` [H], ``router`` [H, E], ``up`` [E, H, 2 I], ``down`` [E, I, H]), workspaces and
    buffers of a block for n tokens; neither direction allocates anything. Weight gradients are fp32 and are added
    to (``zero_grad`` clears them)."""

    def __init__(self, n, topk, norm, router, up, down, eps=1e-6):
        H, E = router.shape
        I = down.shape[1]
        self.n, self.H, self.E, self.I, self.k = n, H, E, I, topk
        self.norm, self.router, self.up, self.down = norm, router, up, down
        rows, dev = n * topk, norm.device

        def empty(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=dev)

        def workspace(nbytes):
            ws = empty(nbytes, dtype=torch.uint8)
            tdx.check(tdx.tdx_workspace_init(ws), "tdx_workspace_init")
            return ws

        fp32 = torch.float32
        self.h, self.y, self.rstd = empty(n, H), empty(n, H), empty(n, dtype=fp32)
        self.logits, self.idx, self.gates = empty(n, E), empty(n, topk, dtype=torch.int32), empty(n, topk, dtype=fp32)
        self.dest, self.offsets = empty(n, topk, dtype=torch.int32), empty(E + 1, dtype=torch.int32)
        self.expert_in, self.expert_act, self.out = empty(rows, 2 * I), empty(rows, I), empty(n, H)
        self.d_rows, self.d_gates, self.d_act = empty(rows, H), empty(n, topk, dtype=fp32), empty(rows, I)
        self.d_logits, self.d_y, self.d_x = empty(n, E), empty(n, H), empty(n, H)
        self.grads = {name: torch.zeros(w.shape, dtype=fp32, device=dev)
                      for name, w in (("norm", norm), ("router", router), ("up", up), ("down", down))}
        self.norm_opts = tdx.make_norm_opts(eps=eps)
        self.opts = tdx.make_opts(epoch=tdx.TDX_EPOCH_DEVICE)
        # set if a wait inside a product's kernel runs out: without it nothing would tell
        self.word = torch.zeros(1, dtype=torch.int32, device=dev)
        self.fwd_opts = tdx.make_linear_opts(device_status=self.word)
        self.bwd_opts = tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32, accumulate=1, device_status=self.word)
        up_size, down_size = (1, n, H, 2 * I, E, topk, BF16, self.opts), (1, n, I, H, E, topk, BF16, self.opts)
        self.ws_up = workspace(tdx.tdx_moe_workspace_size(*up_size))
        self.ws_down = workspace(tdx.tdx_moe_combine_workspace_size(*down_size))
        self.ws_norm = workspace(tdx.tdx_rmsnorm_bwd_workspace_size(n, H, BF16))

        def inside(ws, at):   # the rows that a call keeps in its workspace
            return ws[at:at + rows * H * 2].view(torch.bfloat16).view(rows, H)

        self.expert_tokens = inside(self.ws_up, tdx.tdx_moe_plan_info(*up_size)["off_R"])
        self.expert_out = inside(self.ws_down, tdx.tdx_moe_combine_plan_info(*down_size)["off_R"])
        self.d_norm = empty(H, dtype=fp32)

    def zero_grad(self):
        for g in self.grads.values():
            g.zero_()

    def forward(self, x, residual, stream=None):
        """x, residual: [n, H] bf16. Returns (out, h)."""
        n, H, E, I, k = self.n, self.H, self.E, self.I, self.k
        tdx.check(tdx.tdx_rmsnorm(x, residual, self.norm, self.h, self.y, None, self.rstd, n, H, BF16, self.norm_opts,
                                  stream), "tdx_rmsnorm")
        tdx.check(tdx.tdx_linear(self.y, self.router, None, None, None, self.logits, None, n, H, E, BF16,
                                 self.fwd_opts, stream), "tdx_linear")
        tdx.check(tdx.tdx_moe_route(self.logits, None, self.idx, self.gates, None, n, E, k, BF16, None, stream),
                  "tdx_moe_route")
        tdx.check(tdx.tdx_moe_dispatch_gemm([self.y], [self.idx], self.up, self.expert_in, self.dest, self.offsets,
                                            self.ws_up, 1, n, H, 2 * I, E, k, BF16, self.opts, stream),
                  "tdx_moe_dispatch_gemm")
        tdx.check(tdx.tdx_swiglu(self.expert_in, self.expert_act, None, None, n * k, I, BF16, None, stream), "tdx_swiglu")
        tdx.check(tdx.tdx_moe_gemm_combine(self.expert_act, [self.idx], self.down, [self.gates], [self.out], self.ws_down,
                                           1, n, I, H, E, k, BF16, self.opts, stream), "tdx_moe_gemm_combine")
        return self.out, self.h

    def backward(self, d_out, d_h, stream=None):
        """Gradients by out and h (of the residual stream, or None). Returns the gradient by x and residual alike
        and adds to ``grads``."""
        n, H, E, I, k, rows = self.n, self.H, self.E, self.I, self.k, self.n * self.k
        g = self.grads
        tdx.check(tdx.tdx_moe_combine_bwd(d_out, self.expert_out, self.dest, self.gates, self.d_rows, self.d_gates, rows,
                                          n, H, k, BF16, None, stream), "tdx_moe_combine_bwd")
        tdx.check(tdx.tdx_grouped_gemm_bwd(self.d_rows, self.expert_act, self.offsets, self.down, self.d_act, g["down"],
                                           rows, I, H, E, BF16, self.bwd_opts, stream), "tdx_grouped_gemm_bwd")
        tdx.check(tdx.tdx_swiglu_bwd(self.expert_in, self.d_act, self.expert_in, rows, I, BF16, None, stream),
                  "tdx_swiglu_bwd")
        tdx.check(tdx.tdx_grouped_gemm_bwd(self.expert_in, self.expert_tokens, self.offsets, self.up, self.d_rows, g["up"],
                                           rows, H, 2 * I, E, BF16, self.bwd_opts, stream), "tdx_grouped_gemm_bwd")
        tdx.check(tdx.tdx_moe_combine(self.d_rows, self.dest, None, self.d_y, rows, n, H, k, BF16, None, stream),
                  "tdx_moe_combine")
        tdx.check(tdx.tdx_moe_route_bwd(self.logits, self.idx, self.d_gates, self.d_logits, n, E, k, BF16, None, stream),
                  "tdx_moe_route_bwd")
        tdx.check(tdx.tdx_linear_bwd(self.d_logits, self.y, self.router, self.d_y, self.d_y, g["router"], n, H, E, BF16,
                                     self.bwd_opts, stream), "tdx_linear_bwd")
        tdx.check(tdx.tdx_rmsnorm_bwd(self.d_y, self.h, self.norm, self.rstd, d_h, self.d_x, self.d_norm, self.ws_norm, n,
                                      H, BF16, self.norm_opts, stream), "tdx_rmsnorm_bwd")
        g["norm"] += self.d_norm
        return self.d_x

    def status(self):
        """Raise if a call met an error on the device (synchronises)."""
        for ws in (self.ws_up, self.ws_down):
            st, detail = tdx.tdx_read_device_status(ws)
            if st != tdx.TDX_OK:
                raise tdx.TdxError(st, f"device status {detail}")
        tdx.check(int(self.word), "device status of the products")


def random_block(n, H, I, E, topk, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)

    block = MoeBlock(n, topk, 1.0 + randn(H, std=0.1), randn(H, E, std=H ** -0.5), randn(E, H, 2 * I, std=H ** -0.5),
                     randn(E, I, H, std=I ** -0.5))
    return block, randn(n, H), randn(n, H), randn(n, H, std=0.1), randn(n, H, std=0.1)


def main():
    n, H, I, E, topk = 4096, 2048, 1024, 32, 8
    block, x, residual, d_out, d_h = random_block(n, H, I, E, topk)

    def step():
        block.forward(x, residual)
        block.backward(d_out, d_h)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    block.status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    block.status()
    us = start.elapsed_time(end) / 20 * 1e3
    flops = 3 * 2 * n * topk * 3 * H * I
    print(f"{n} tokens, {H} wide, {topk} of {E} experts of {I}: {us:.0f} us a step, {flops / us / 1e6:.0f} TFLOP/s in the experts")


if __name__ == "__main__":
    main()
