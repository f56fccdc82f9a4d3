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


# ------------------------------------------------------------------------- results of 8 and 16 bits
def near(got, want, half, K, slope=1.0):
    """Terms of one sign, in sums of at most 65536 of K. The tensor cores add 16 products or more at a time and may lose
    2^-22 of the sum so far with each addition: at most 65536 / 16 * 2^-22 * 1/2 = 2^-11 of a sum that grows evenly. The
    sums are added in fp32, 2^-24 each. Then one rounding."""
    lim = slope * (2.0 ** -11 + K / 65536 * 2.0 ** -24) + half
    off = ((got.double() - want) / want).abs().max()
    assert float(off) <= lim, (float(off), lim)


def positive(g, *shape, dtype=BF):
    return torch.empty(shape, device="cuda", dtype=BF).uniform_(0.5, 1.5, generator=g).to(dtype)


def test_weight_gradient_of_millions_of_rows():
    """All rows go to the first of 512 experts, whose one tile then is one CTA's."""
    g = torch.Generator(device="cuda").manual_seed(1)
    R, K, N, E = (1 << 22) + 37, 64, 72, 512
    X, dY = positive(g, R, K), positive(g, R, N)
    off = torch.full((E + 1,), R, dtype=torch.int32, device="cuda")
    off[0] = 0
    want = sum(X[a:a + (1 << 20)].double().t() @ dY[a:a + (1 << 20)].double() for a in range(0, R, 1 << 20))
    dB = torch.full((E, K, N), 3.0, dtype=BF, device="cuda")
    tdx.check(tdx.tdx_grouped_gemm_bwd(dY, X, off, None, None, dB, R, K, N, E, 0))
    near(dB[0], want, 2.0 ** -8, R)
    assert bool((dB[1:] == 0).all())
    old = torch.ones_like(dB)   # added to, and negligible beside the sum
    tdx.check(tdx.tdx_grouped_gemm_bwd(dY, X, off, None, None, old, R, K, N, E, 0, tdx.make_linear_opts(accumulate=1)))
    near(old[0], want, 2.0 ** -8 + 1e-6, R)
    assert bool((old[1:] == 1).all())


# 320 tiles of a single CTA or 80 of a pair: every tile's sum is one CTA's or pair's own
@pytest.mark.parametrize("K", [(1 << 20) + 16, (1 << 16) + 1040])
@pytest.mark.parametrize("out", [BF, E4])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_forward_products_of_long_rows(K, out, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    M, N = 2048, 2560
    A, B = positive(g, M, K, dtype=dtype), positive(g, K, N, dtype=dtype)
    rows, cols = slice(1000, 1064), slice(1300, 1364)
    want = A[rows].double() @ B[:, cols].double()
    code = {BF: tdx.TDX_BF16, E4: tdx.TDX_FP8_E4M3}
    scale = float(want.max()) / 256
    C = torch.empty(M, N, dtype=out, device="cuda")
    o = tdx.make_linear_opts(out_dtype=code[out], out_scale=scale if out == E4 else 1.0)
    tdx.check(tdx.tdx_linear(A, B, None, None, None, C, None, M, K, N, code[dtype], o))
    got = C[rows, cols].double() * (scale if out == E4 else 1.0)
    near(got, want, 2.0 ** -8 if out == BF else 2.0 ** -4 + 2.0 ** -22, K)
    # gated, with a bias and z: v of about 1, whose silu's slope is below 1.1
    bias = positive(g, N)
    o = tdx.make_linear_opts(act=tdx.TDX_ACT_SWIGLU, alpha=1.0 / K)
    C, z = torch.empty(M, N // 2, dtype=BF, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    tdx.check(tdx.tdx_linear(A, B, bias, None, None, C, z, M, K, N, code[dtype], o))
    cols = slice(100, 164)
    up = slice(cols.start + N // 2, cols.stop + N // 2)
    v, u = ((A[rows].double() @ B[:, c].double()) / K + bias[c].double() for c in (cols, up))
    near(z[rows, cols], v, 2.0 ** -8 + 2.0 ** -22, K)
    near(z[rows, up], u, 2.0 ** -8 + 2.0 ** -22, K)
    # relative slope of silu at v > 0: 1 + v (1 - sigmoid(v)) <= 1.28, and the up half's 1
    near(C[rows, cols], v * torch.sigmoid(v) * u, 2.0 ** -8 + 2.0 ** -18, K, slope=2.3)


def test_input_gradient_of_long_rows():
    g = torch.Generator(device="cuda").manual_seed(3)
    M, K, N = 2048, 2560, (1 << 20) + 8
    dz, B = positive(g, M, N), positive(g, K, N)
    dA = torch.empty(M, K, dtype=BF, device="cuda")
    tdx.check(tdx.tdx_linear_bwd(dz, None, B, None, dA, None, M, K, N, 0))
    rows, cols = slice(1000, 1064), slice(1300, 1364)
    near(dA[rows, cols], dz[rows].double() @ B[cols].double().t(), 2.0 ** -8, N)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_one_row_of_a_long_product(act, dtype):
    """One tile of a cluster: each CTA's share of K is a long sum of its own."""
    g = torch.Generator(device="cuda").manual_seed(4)
    K, N = (1 << 20) + 4112, 256
    A, B = positive(g, 3, K, dtype=dtype), positive(g, K, N, dtype=dtype)
    code = tdx.TDX_BF16 if dtype == BF else tdx.TDX_FP8_E4M3
    want = A.double() @ B.double() / K
    cols = N if act == "none" else N // 2
    o = tdx.make_linear_opts(act=tdx.TDX_ACT_NONE if act == "none" else tdx.TDX_ACT_SWIGLU, alpha=1.0 / K)
    first = None
    for _ in range(10):
        C, z = torch.empty(3, cols, dtype=BF, device="cuda"), torch.empty(3, N, dtype=BF, device="cuda")
        tdx.check(tdx.tdx_linear(A, B, None, None, None, C, z, 3, K, N, code, o))
        near(z, want, 2.0 ** -8 + 2.0 ** -22, K)
        if act == "swiglu":
            gate, up = want[:, :cols], want[:, cols:]
            near(C, gate * torch.sigmoid(gate) * up, 2.0 ** -8 + 2.0 ** -18, K, slope=2.3)
        first = C if first is None else first
        assert torch.equal(C, first)


def test_long_and_short_tiles_in_turn():
    """Runs of all lengths through the same CTAs: a tile of several sums takes both accumulators, the next one either."""
    g = torch.Generator(device="cuda").manual_seed(5)
    counts = ([70000, 3, 0, 200000, 64, 131072, 65536, 1, 65537] + [40] * 90) * 5
    E, K, N = len(counts), 64, 256
    R = sum(counts)
    X = torch.randint(-4, 5, (R, K), generator=g, device="cuda", dtype=torch.int8).to(BF)
    dY = torch.randint(-4, 5, (R, N), generator=g, device="cuda", dtype=torch.int8).to(BF)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    at = off.tolist()
    dB = torch.full((E, K, N), 777.0, dtype=BF, device="cuda")
    tdx.check(tdx.tdx_grouped_gemm_bwd(dY, X, off, None, None, dB, R, K, N, E, 0))
    for e in range(E):   # sums of integers below 2^24: exact
        want = X[at[e]:at[e + 1]].double().t() @ dY[at[e]:at[e + 1]].double()
        assert torch.equal(dB[e].float(), want.float().to(BF).float()), e


def test_kernels_of_seconds():
    """A weight gradient over 2^30 rows of one expert, whose tile takes over 4 s, and one with rows for the same CTA
    after it: no wait runs out. Sums of ones in steps of 2^16: exact."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    R, K, N, E = 1 << 30, 8, 8, 512
    off = torch.full((E + 1,), R - 128, dtype=torch.int32, device="cuda")
    off[0] = 0
    off[sms + 1:] = R - 59            # 69 rows: a whole slice of 64 and a tail
    X = torch.ones(R, K, dtype=BF, device="cuda")
    X[R - 128:] = 3.0
    dB, status = torch.full((E, K, N), 5.0, dtype=BF, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    o = tdx.make_linear_opts(device_status=status)
    tdx.check(tdx.tdx_grouped_gemm_bwd(X, X, off, None, None, dB, R, K, N, E, 0, o))
    assert int(status) == 0
    want = torch.zeros(E)
    want[0], want[sms] = R - 128, 9 * 69
    assert torch.equal(dB, want.to(BF).cuda()[:, None, None].expand(E, K, N))


@pytest.mark.parametrize("acc", [0, 1])
def test_weight_gradients_of_long_runs_on_pairs(acc):
    """Tiles of pairs whose runs are long and short, with tails, beside the input gradient; and one layer's."""
    g = torch.Generator(device="cuda").manual_seed(6)
    counts, K, N = [70001, 30, 131079], 2048, 2056
    R, E = sum(counts), len(counts)

    def ints8(*shape):
        return torch.randint(-4, 5, shape, generator=g, device="cuda", dtype=torch.int8).to(BF)

    X, dY, B = ints8(R, K), ints8(R, N), ints8(E, K, N)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    at = off.tolist()
    old = ints8(E, K, N)
    dB, dX = old.clone(), torch.empty_like(X)
    o = tdx.make_linear_opts(accumulate=acc)
    tdx.check(tdx.tdx_grouped_gemm_bwd(dY, X, off, B, dX, dB, R, K, N, E, 0, o))
    some = torch.tensor([0, 1, 127, 128, 255, 256, 1000, 1023, 1024, 2000, 2047], device="cuda")
    for e in range(E):   # sums of integers below 2^24: exact
        rows = slice(at[e], at[e + 1])
        want = X[rows][:, some].double().t() @ dY[rows].double() + acc * old[e][some].double()
        assert torch.equal(dB[e][some].float(), want.float().to(BF).float()), e
        last = slice(at[e + 1] - 20, at[e + 1])
        assert torch.equal(dX[last].float(), (dY[last].double() @ B[e].double().t()).float().to(BF).float()), e
    dB = old[0].clone()
    tdx.check(tdx.tdx_linear_bwd(dY, X, None, None, None, dB, R, K, N, 0, o))
    want = X[:, some].double().t() @ dY.double() + acc * old[0][some].double()
    assert torch.equal(dB[some].float(), want.float().to(BF).float())
