"""Runs of the products without communication as a user has them: a mixture-of-experts block and a dense block
through a training step against 64-bit automatic differentiation, captured graphs, several streams, outputs past
2^31 elements."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import comm_overlapped_gemm_gb300 as tdx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def example():
    spec = importlib.util.spec_from_file_location("moe_training", os.path.join(ROOT, "examples", "moe_training.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def off(got, want):
    """Relative distance in the 2-norm."""
    g, w = got.detach().double().cpu(), want.detach().double().cpu()
    return float((g - w).norm() / w.norm())


def moe64(block, x, residual, idx):
    """The block in 64 bits with the given expert ids; leaves require gradients."""
    leaves = {k: getattr(block, k).double().cpu().requires_grad_(True) for k in ("norm", "router", "up", "down")}
    leaves["x"] = x.double().cpu().requires_grad_(True)
    h = leaves["x"] + residual.double().cpu()
    y = h * torch.rsqrt(h.pow(2).mean(-1, keepdim=True) + 1e-6) * leaves["norm"]
    s = torch.softmax(y @ leaves["router"], -1).gather(1, idx)
    gates = s / s.sum(-1, keepdim=True)
    out = torch.zeros_like(h)
    for e in range(block.E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if len(t) == 0:
            continue
        v = y[t] @ leaves["up"][e]
        act = torch.nn.functional.silu(v[:, :block.I]) * v[:, block.I:]
        out = out.index_add(0, t, gates[t, j, None] * (act @ leaves["down"][e]))
    return out, h, leaves


@pytest.mark.parametrize("n,H,I,E,k", [(40, 64, 32, 8, 2), (333, 256, 128, 16, 4), (1000, 512, 256, 8, 3)])
def test_moe_block_training_step(n, H, I, E, k):
    """Values pass at most ten roundings to bf16 on their way to a gradient (y, logits, the two products, the
    activation, the experts' rows, and their gradients back), each of at most 2^-8 relative and 2^-9.8 in the mean
    square; sums of independent ones add in squares, and no step of the block stretches a relative error in the norm
    by more than about 2: 2 * sqrt(10) * 2^-8 = 2.5%."""
    block, x, residual, d_out, d_h = example().random_block(n, H, I, E, k, seed=n)
    out, h = block.forward(x, residual)
    dx = block.backward(d_out, d_h)
    block.status()
    idx = block.idx.cpu().long()
    w_out, w_h, leaves = moe64(block, x, residual, idx)
    ((w_out * d_out.double().cpu()).sum() + (w_h * d_h.double().cpu()).sum()).backward()
    lim = 0.025
    assert off(out, w_out) <= lim and off(h, w_h) <= 2.0 ** -8
    assert off(dx, leaves["x"].grad) <= lim
    for name, got in block.grads.items():
        assert off(got, leaves[name].grad) <= lim, name
    # the same gradients against differences of the 64-bit loss along the kernel's own gradient
    for name in ("up", "down", "router"):
        step = block.grads[name].double().cpu()
        eps = 1e-6 / float(step.norm())

        def loss(sign):
            keep = leaves[name].data.clone()
            moved = type("B", (), dict(E=E, I=I, **{m: getattr(block, m) for m in ("norm", "router", "up", "down")}))()
            setattr(moved, name, (keep + sign * eps * step))
            o, hh, _ = moe64(moved, x, residual, idx)
            return float(((o * d_out.double().cpu()).sum() + (hh * d_h.double().cpu()).sum()).detach())

        slope = (loss(1.0) - loss(-1.0)) / (2 * eps)
        assert abs(slope - float(step.pow(2).sum())) <= 2 * lim * float(step.pow(2).sum()), name
    # a second backward pass adds to the weights' gradients
    first = {m: v.clone() for m, v in block.grads.items()}
    block.forward(x, residual)
    block.backward(d_out, d_h)
    for m, v in block.grads.items():
        assert off(v, 2 * first[m]) <= 2.0 ** -22 + 1e-7, m


def test_moe_block_in_a_graph():
    mod = example()
    block, x, residual, d_out, d_h = mod.random_block(200, 256, 128, 16, 4, seed=1)

    def step():
        block.forward(x, residual)
        return block.backward(d_out, d_h)

    dx = step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (block.out, dx, block.grads["up"], block.grads["down"], block.grads["router"])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        block.zero_grad()
        block.out.zero_()
        block.d_x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        block.status()
        got = (block.out, block.d_x, block.grads["up"], block.grads["down"], block.grads["router"])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


class Dense:
    """x + gelu(norm-free x @ up + b) @ down, with its gradients; buffers made once."""

    def __init__(self, M, H, F, seed, dev="cuda"):
        g = torch.Generator(device=dev).manual_seed(seed)

        def randn(*s, std=1.0):
            return (torch.randn(*s, generator=g, device=dev) * std).to(BF)

        self.M, self.H, self.F = M, H, F
        self.x, self.up, self.down = randn(M, H), randn(H, F, std=H ** -0.5), randn(F, H, std=F ** -0.5)
        self.b, self.dout = randn(F, std=0.5), randn(M, H, std=0.1)

        def empty(*s, dtype=BF):
            return torch.empty(*s, dtype=dtype, device=dev)

        self.z, self.a, self.out = empty(M, F), empty(M, F), empty(M, H)
        self.da, self.dz, self.dx, self.db = empty(M, F), empty(M, F), empty(M, H), empty(F, dtype=torch.float32)
        self.dup, self.ddown = empty(H, F, dtype=torch.float32), empty(F, H, dtype=torch.float32)
        self.act = tdx.make_linear_opts(act=tdx.TDX_ACT_GELU_TANH)
        self.bwd = tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32)
        self.ws = torch.empty(tdx.tdx_linear_act_bwd_workspace_size(M, F, 0, self.act), dtype=torch.uint8, device=dev)

    def run(self):
        M, H, F = self.M, self.H, self.F
        tdx.check(tdx.tdx_linear(self.x, self.up, self.b, None, None, self.a, self.z, M, H, F, 0, self.act))
        tdx.check(tdx.tdx_linear(self.a, self.down, None, self.x, None, self.out, None, M, F, H, 0))
        tdx.check(tdx.tdx_linear_bwd(self.dout, self.a, self.down, None, self.da, self.ddown, M, F, H, 0, self.bwd))
        tdx.check(tdx.tdx_linear_act_bwd(self.da, self.z, self.dz, self.db, self.ws, M, F, 0, self.act))
        tdx.check(tdx.tdx_linear_bwd(self.dz, self.x, self.up, self.dout, self.dx, self.dup, M, H, F, 0, self.bwd))

    def results(self):
        return [self.out, self.dx, self.db, self.dup, self.ddown]

    def wipe(self):
        for t in self.results() + [self.z, self.a, self.da, self.dz]:
            t.fill_(float("nan"))


@pytest.mark.parametrize("M,H,F", [(1, 64, 128), (77, 256, 520), (1021, 512, 1024)])
def test_dense_block_training_step(M, H, F):
    """At most four roundings to bf16 lie on the way to each result (a, z, da, dz): as above, 2 * sqrt(4) * 2^-8."""
    d = Dense(M, H, F, seed=M)
    d.run()
    leaf = {k: getattr(d, k).double().cpu().requires_grad_(True) for k in ("x", "up", "down", "b")}
    a = torch.nn.functional.gelu(leaf["x"] @ leaf["up"] + leaf["b"], approximate="tanh")
    out = leaf["x"] + a @ leaf["down"]
    (out * d.dout.double().cpu()).sum().backward()
    lim = 2 * 2 * 2.0 ** -8
    for got, want in ((d.out, out), (d.dx, leaf["x"].grad), (d.db, leaf["b"].grad), (d.dup, leaf["up"].grad),
                      (d.ddown, leaf["down"].grad)):
        assert off(got, want) <= lim


def test_dense_block_replayed_beside_eager_calls():
    """The two products of one gradient overlap on the GPU; what follows reads both."""
    d = Dense(300, 512, 1024, seed=2)
    d.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in d.results()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.run()
    for i in range(10):
        d.wipe()
        graph.replay() if i % 2 else d.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(d.results(), want))
    for _ in range(20):   # back to back, nothing in between
        d.run()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(d.results(), want))


def test_blocks_on_two_streams():
    blocks = [Dense(200 + 100 * i, 256, 512 + 512 * i, seed=i) for i in range(3)]
    want = []
    for b in blocks:
        b.run()
        want.append([t.clone() for t in b.results()])
        b.wipe()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(20):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        assert all(torch.equal(x, y) for x, y in zip(b.results(), w))


def test_a_gradient_followed_at_once_by_its_reader():
    """tdx_linear_bwd's second kernel starts beside its first and ends after it: a kernel of another kind that
    follows sees the first one's output whole."""
    g = torch.Generator(device="cuda").manual_seed(4)
    M, K, N = 2048, 2048, 64     # dA: 128 tiles of one K slice; dB: few tiles, done early
    dz = torch.randn(M, N, generator=g, device="cuda").to(BF)
    A, B = torch.randn(M, K, generator=g, device="cuda").to(BF), torch.randn(K, N, generator=g, device="cuda").to(BF)
    dA, dB, out = torch.empty_like(A), torch.empty_like(B), torch.empty_like(A)
    dest = torch.arange(M, dtype=torch.int32, device="cuda")
    want = None
    for i in range(30):
        dA.fill_(float("nan"))
        tdx.check(tdx.tdx_linear_bwd(dz, A, B, None, dA, dB, M, K, N, 0))
        tdx.check(tdx.tdx_moe_combine(dA, dest, None, out, M, M, K, 1, 0))
        torch.cuda.synchronize()
        want = out.clone() if want is None else want
        assert torch.equal(out, want) and torch.equal(out, dA)


def test_offsets_past_32_bits():
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    M, K, N = 270001, 64, 8192                     # 2.2e9 outputs
    A = torch.randint(-4, 5, (M, K), device="cuda").to(BF)
    B = torch.randint(-4, 5, (K, N), device="cuda").to(BF)
    C = torch.empty(M, N, dtype=BF, device="cuda")
    tdx.check(tdx.tdx_linear(A, B, None, None, None, C, None, M, K, N, 0))
    for at in (slice(0, 300), slice(262000, 262300), slice(M - 300, M)):
        assert torch.equal(C[at].float(), (A[at].float() @ B.float()).to(BF).float())
    # its gradients: the rows of dz and dA, and of dB's sums
    dz = C
    dz.copy_(torch.randint(-2, 3, (1, N), device="cuda").to(BF).expand(M, N))
    dA, dB = torch.empty_like(A), torch.empty(K, N, device="cuda")
    tdx.check(tdx.tdx_linear_bwd(dz, A, B, None, dA, dB, M, K, N, 0, tdx.make_linear_opts(dw_dtype=tdx.TDX_FP32)))
    assert torch.equal(dA[-300:].double(), (dz[-300:].double() @ B.double().t()).to(BF).double())
    assert torch.equal(dB.double(), A.double().sum(0)[:, None] * dz[0].double()[None])
    del A, C, dz, dA
    # experts' weights past 2^31 elements
    E, K, N, R = 260, 1024, 8192, 300
    W = torch.zeros(E, K, N, dtype=BF, device="cuda")
    W[0] = 1.0
    W[E - 1].copy_(torch.randint(-4, 5, (K, N), device="cuda").to(BF))
    X = torch.randint(-4, 5, (R, K), device="cuda").to(BF)
    off_ = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off_[1:] = 100
    off_[E] = R
    Y = torch.empty(R, N, device="cuda")
    tdx.check(tdx.tdx_grouped_gemm(X, off_, W, None, None, Y, None, R, K, N, E, 0,
                                   tdx.make_linear_opts(out_dtype=tdx.TDX_FP32)))
    assert torch.equal(Y[100:].double(), X[100:].double() @ W[E - 1].double())
    dW = torch.full_like(W, 7.0)
    dY = torch.randint(-4, 5, (R, N), device="cuda").to(BF)
    tdx.check(tdx.tdx_grouped_gemm_bwd(dY, X, off_, W, None, dW, R, K, N, E, 0))
    assert torch.equal(dW[E - 1].double(), (X[100:].double().t() @ dY[100:].double()).to(BF).double())
    assert bool((dW[5] == 0).all()) and bool((dW[E - 2] == 0).all())


FIRST_CALLS = """
import torch
import comm_overlapped_gemm_gb300 as tdx
def rn(*s): return torch.randn(*s, device="cuda", dtype=torch.bfloat16)
A, B, x, W, big = rn(300, 512), rn(512, 1024), rn(1, 8192), rn(8192, 2048), rn(2048, 2048)
C, y, out, dA, dB = rn(300, 1024), rn(1, 2048), rn(2048, 2048), torch.empty_like(A), torch.empty_like(B)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    tdx.check(tdx.tdx_linear(A, B, None, None, None, C, None, 300, 512, 1024, 0))
    tdx.check(tdx.tdx_linear_bwd(C, A, B, None, dA, dB, 300, 512, 1024, 0))
    tdx.check(tdx.tdx_linear(x, W, None, None, None, y, None, 1, 8192, 2048, 0))      # clusters
    tdx.check(tdx.tdx_linear(big, big, None, None, None, out, None, 2048, 2048, 2048, 0))   # pairs
g.replay()
torch.cuda.synchronize()
for got, want in ((C, A.double() @ B.double()), (dA, C.double() @ B.double().t()), (dB, A.double().t() @ C.double()),
                  (y, x.double() @ W.double()), (out, big.double() @ big.double())):
    assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -8
"""


def test_first_calls_of_a_process_under_capture():
    """Kernels' limits and the clusters that fit are asked for at the first call, which may be a captured one."""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads():
    import threading
    blocks = [Dense(300, 256, 1024, seed=7), Dense(170, 512, 512, seed=8)]
    want = []
    for b in blocks:
        b.run()
        want.append([t.clone() for t in b.results()])
        b.wipe()
    torch.cuda.synchronize()
    bad = []

    def work(b):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    b.run()
        except Exception as e:   # noqa: BLE001  (reported below, in the test's own thread)
            bad.append(e)

    threads = [threading.Thread(target=work, args=(b,)) for b in blocks]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad
    for b, w in zip(blocks, want):
        assert all(torch.equal(x, y) for x, y in zip(b.results(), w))


def test_moe_block_tells_of_a_wait_that_ran_out():
    """Every product of the example has its status word, and status() reads it."""
    block, x, residual, d_out, d_h = example().random_block(64, 128, 64, 8, 2, seed=3)
    block.forward(x, residual)
    block.backward(d_out, d_h)
    block.status()
    assert all(o.device_status == block.word.data_ptr() for o in (block.fwd_opts, block.bwd_opts))
    block.word.fill_(tdx.TDX_ERR_TIMEOUT)
    with pytest.raises(tdx.TdxError):
        block.status()
    block.word.zero_()
    block.forward(x, residual)
    block.status()
