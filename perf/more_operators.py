"""The products a model's dense and expert blocks train and answer with, as measured cases: the
linear layer (product with bias, activation and residual in its epilogue), the products grouped by
expert over ragged rows, and the weighted sum of a token's expert rows, each forwards and backwards.

``run`` computes a case in its plain form (elementary torch operations in fp32, rounded once at
the end) where ``own`` is false and through the library's entry points where it is true;
``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
GELU_C, GELU_D = math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # the output projection of one token of a decoding step, added to the residual stream
        dict(name="linear_one_token", op="linear", M=1, K=8192, N=8192, dtype="bf16", out="bf16", act="none",
             bias=False, res=True, z=False, rows=False),
        # the first product of a GELU block over an odd number of packed training tokens, z kept for its gradient
        dict(name="linear_gelu_packed", op="linear", M=1021, K=3584, N=8192, dtype="bf16", out="bf16",
             act="gelu_tanh", bias=True, res=False, z=True, rows=False),
        # the gated block's first product of a prompt: 8 x 1024 tokens, gate and up halves of 3584
        dict(name="linear_swiglu_prompt", op="linear", M=8192, K=8192, N=7168, dtype="bf16", out="bf16",
             act="swiglu", bias=False, res=False, z=False, rows=False),
        # an e4m3 product of tokens scaled one by one, 8 x 2048 of them, added to the residual stream
        dict(name="linear_e4m3_prompt", op="linear", M=16384, K=8192, N=8192, dtype="e4m3", out="bf16", act="none",
             bias=False, res=True, z=False, rows=True),
        # the activation's and the bias's gradient of a training batch
        dict(name="linear_act_bwd", op="linear_act_bwd", M=16381, N=8192, dtype="bf16", act="gelu_tanh", bias=True),
        # gradients of a small layer over packed tokens, weights' gradient in fp32
        dict(name="linear_bwd_small", op="linear_bwd", M=1021, K=1024, N=1024, dtype="bf16", dw="fp32", res=False),
        # gradients of the gated block's first product over a training batch
        dict(name="linear_bwd", op="linear_bwd", M=8192, K=8192, N=7168, dtype="bf16", dw="bf16", res=True),
        # one token's eight rows, eight of 64 experts
        dict(name="grouped_one_token", op="grouped", R=8, K=7168, N=2048, E=64, dtype="bf16", out="bf16", act="none",
             rows=False, z=False),
        # an odd number of routed rows over 64 uneven experts, some empty, gate and up halves of 2048
        dict(name="grouped_prompt", op="grouped", R=65521, K=7168, N=4096, E=64, dtype="bf16", out="bf16",
             act="swiglu", rows=False, z=False),
        # gradients of 16 experts' second product in training
        dict(name="grouped_bwd", op="grouped_bwd", R=32749, K=2048, N=7168, E=16, dtype="bf16", dw="bf16"),
        # the sum of each token's eight expert rows
        dict(name="combine_prompt", op="combine", T=8192, H=7168, k=8, dtype="bf16", gates=True),
        # its gradient: the experts' rows and the gates
        dict(name="combine_bwd", op="combine_bwd", T=8191, H=7168, k=8, dtype="bf16", gates=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


_ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_act_bwd", "linear_bwd", "grouped", "grouped", "grouped_bwd",
                     "combine", "combine_bwd"])
    if op in ("linear", "linear_bwd"):
        c = dict(op=op, M=_log(rng, 1, 8192), K=16 * _log(rng, 4, 512), N=32 * _log(rng, 2, 256))
        if op == "linear_bwd":
            c.update(dtype="bf16", dw=rng.choice(["bf16", "fp32"]), res=rng.random() < 0.5)
            return c
        c["dtype"] = rng.choice(["bf16", "bf16", "e4m3"])
        c["out"] = rng.choice(["bf16", "bf16", "fp32", "e4m3"])
        c.update(act=rng.choice(_ACTS), bias=rng.random() < 0.5, res=rng.random() < 0.5, z=rng.random() < 0.4,
                 rows=c["dtype"] == "e4m3" and rng.random() < 0.7)
        return c
    if op == "linear_act_bwd":
        N = 32 * _log(rng, 2, 512)
        return dict(op=op, M=_log(rng, 1, min(32768, (1 << 27) // N)), N=N, dtype="bf16", act=rng.choice(_ACTS),
                    bias=rng.random() < 0.7)
    if op in ("grouped", "grouped_bwd"):
        E = _log(rng, 1, 128)
        K = 16 * _log(rng, 4, 256)
        N = 32 * _log(rng, 2, max(2, min(128, (1 << 24) // (E * K))))
        c = dict(op=op, R=_log(rng, 1, 32768), K=K, N=N, E=E)
        if op == "grouped_bwd":
            c.update(dtype="bf16", dw=rng.choice(["bf16", "fp32"]))
            return c
        c["dtype"] = rng.choice(["bf16", "bf16", "e4m3"])
        c["out"] = rng.choice(["bf16", "bf16", "fp32"])
        c.update(act=rng.choice(["none", "none", "silu", "swiglu"]), rows=c["dtype"] == "e4m3" and rng.random() < 0.7,
                 z=rng.random() < 0.3)
        return c
    k = rng.choice([1, 2, 4, 6, 8, 8, 16])
    H = 16 * _log(rng, 4, 512)
    return dict(op=op, T=_log(rng, 1, min(32768, (1 << 28) // (H * k))), H=H, k=k, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                gates=rng.random() < 0.7)


def _width(name):
    return {"bf16": 2, "fp32": 4, "e4m3": 1}[name]


def _out_cols(case):
    return case["N"] // 2 if case["act"] == "swiglu" else case["N"]


def work(case):
    op, e = case["op"], _width(case["dtype"])
    if op == "linear":
        M, K, N, O = case["M"], case["K"], case["N"], _out_cols(case)
        b = (M * K + K * N) * e + M * O * _width(case["out"])
        b += (2 * N if case["bias"] else 0) + (2 * M * O if case["res"] else 0) + (2 * M * N if case["z"] else 0)
        return {"bytes": b + (4 * M if case["rows"] else 0), "flops": 2 * M * K * N}
    if op == "linear_act_bwd":
        M, N, O = case["M"], case["N"], _out_cols(case)
        z = 0 if case["act"] == "none" else M * N
        return {"bytes": 2 * (M * O + 2 * z) + (4 * N if case["bias"] else 0), "flops": 12 * M * N}
    if op == "linear_bwd":
        M, K, N = case["M"], case["K"], case["N"]
        b = 2 * (M * N + M * K + K * N + M * K + (M * K if case["res"] else 0)) + K * N * _width(case["dw"])
        return {"bytes": b, "flops": 4 * M * K * N}
    if op == "grouped":
        R, K, N, E = case["R"], case["K"], case["N"], min(case["E"], case["R"])
        b = (R * K + E * K * N) * e + R * _out_cols(case) * _width(case["out"]) + (2 * R * N if case["z"] else 0)
        return {"bytes": b, "flops": 2 * R * K * N}
    if op == "grouped_bwd":
        R, K, N, E = case["R"], case["K"], case["N"], case["E"]
        b = 2 * (R * N + 2 * R * K + min(E, R) * K * N) + E * K * N * _width(case["dw"])
        return {"bytes": b, "flops": 4 * R * K * N}
    n, k = case["T"] * case["H"], case["k"]
    if op == "combine":
        return {"bytes": (k + 1) * n * e + (8 if case["gates"] else 4) * case["T"] * k, "flops": 2 * k * n}
    return {"bytes": ((2 * k if case["gates"] else k) + 1) * n * e + (12 if case["gates"] else 4) * case["T"] * k,
            "flops": (3 if case["gates"] else 0) * k * n}


# ------------------------------------------------------------------------------------- inputs
_TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _expert_rows(g, R, E):
    """Rows of each expert: uneven shares, every fourth expert likely empty when there are several."""
    share = torch.rand(E, generator=g).add_(0.05)
    if E > 4:
        share[torch.rand(E, generator=g) < 0.2] = 0.0
    if float(share.sum()) == 0.0:
        share[0] = 1.0
    ids = torch.multinomial(share, R, replacement=True, generator=g)
    return torch.bincount(ids, minlength=E)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    op = case["op"]

    def randn(*shape, dtype=torch.bfloat16, scale=1.0):
        if dtype == torch.float8_e4m3fn:   # codes of values scaled to the type's range
            return torch.cat([torch.randn(*part, generator=g, device="cuda").mul_(64.0).clamp_(-E4M3_MAX, E4M3_MAX)
                              .to(dtype) for part in _parts(shape)])
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype).mul_(scale)

    s = {"case": case, "alpha": 1.0}
    e4 = case["dtype"] == "e4m3"
    dt = _TORCH[case["dtype"]]
    if op in ("linear", "linear_bwd"):
        M, K, N = case["M"], case["K"], case["N"]
        s["A"] = randn(M, K, dtype=dt)
        s["B"] = randn(K, N, dtype=dt, scale=0.02)
        if op == "linear":
            s["bias"] = randn(N, scale=0.5) if case["bias"] else None
            s["res"] = randn(M, _out_cols(case)) if case["res"] else None
        else:
            s["dz"] = randn(M, N, scale=0.01)
            s["res"] = randn(M, K, scale=0.01) if case["res"] else None
    elif op == "linear_act_bwd":
        s["zin"] = randn(case["M"], case["N"]) if case["act"] != "none" else None
        s["dy"] = randn(case["M"], _out_cols(case), scale=0.01)
    elif op in ("grouped", "grouped_bwd"):
        R, K, N, E = case["R"], case["K"], case["N"], case["E"]
        rows = _expert_rows(host, R, E)
        s["rows"] = rows.tolist()
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.long), rows.cumsum(0)]).to(torch.int32).cuda()
        s["A"] = randn(R, K, dtype=dt)
        s["B"] = randn(E, K, N, dtype=dt, scale=0.02)
        if op == "grouped_bwd":
            s["dz"] = randn(R, N, scale=0.01)
        elif e4:
            s["expert_scale"] = torch.rand(E, generator=g, device="cuda").add_(0.5).mul_(0.02 / 64.0)
    else:
        T, H, k = case["T"], case["H"], case["k"]
        s["Z"] = randn(T * k, H, dtype=dt)
        s["dest"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
        s["gates"] = torch.rand(T, k, generator=g, device="cuda").add_(0.01) if case["gates"] else None
        if op == "combine_bwd":
            s["dout"] = randn(T, H, dtype=dt, scale=0.01)
    if e4:
        s["row_scale"] = torch.rand(s["A"].shape[0], generator=g, device="cuda").add_(0.5).mul_(1.0 / 64.0) \
            if case["rows"] else None
        if op == "linear":
            s["alpha"] = 0.02 / 64.0
        if not case["rows"]:
            s["alpha"] /= 64.0
    return s


def _parts(shape):
    """The shape cut along its first dimension into pieces of at most 2^28 values."""
    step = max(1, (1 << 28) // max(1, math.prod(shape[1:])))
    return [(min(step, shape[0] - a),) + tuple(shape[1:]) for a in range(0, shape[0], step)]


def _out_scale(case):
    return 0.0625 if case["out"] == "e4m3" else 1.0


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    if op in ("linear", "grouped"):
        M = s["A"].shape[0]
        s["C"] = empty(M, _out_cols(case), dtype=_TORCH[case["out"]])
        s["z"] = empty(M, case["N"]) if case["z"] else None
    elif op == "linear_act_bwd":
        s["dz"] = empty(case["M"], case["N"]) if case["act"] != "none" else None
        s["dbias"] = empty(case["N"], dtype=torch.float32) if case["bias"] or case["act"] == "none" else None
    elif op in ("linear_bwd", "grouped_bwd"):
        s["dA"] = torch.empty_like(s["A"])
        s["dB"] = torch.empty_like(s["B"], dtype=_TORCH[case["dw"]])
    elif op == "combine":
        s["out"] = empty(case["T"], case["H"], dtype=_TORCH[case["dtype"]])
    else:
        s["dZ"] = torch.empty_like(s["Z"])
        s["dgates"] = torch.empty_like(s["gates"]) if case["gates"] else None
    if own:
        import comm_overlapped_gemm_gb300 as tdx
        code = {"bf16": tdx.TDX_BF16, "fp32": tdx.TDX_FP32, "e4m3": tdx.TDX_FP8_E4M3}
        act = {"none": tdx.TDX_ACT_NONE, "relu": tdx.TDX_ACT_RELU, "gelu": tdx.TDX_ACT_GELU,
               "gelu_tanh": tdx.TDX_ACT_GELU_TANH, "silu": tdx.TDX_ACT_SILU, "swiglu": tdx.TDX_ACT_SWIGLU}
        s["tdx"], s["dt"] = tdx, code[case["dtype"]]
        if op in ("linear", "grouped"):
            s["opts"] = tdx.make_linear_opts(out_dtype=code[case["out"]], act=act[case["act"]], alpha=s["alpha"],
                                             out_scale=_out_scale(case))
        elif op == "linear_act_bwd":
            s["opts"] = tdx.make_linear_opts(act=act[case["act"]])
            n = tdx.tdx_linear_act_bwd_workspace_size(case["M"], case["N"], s["dt"], s["opts"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        elif op in ("linear_bwd", "grouped_bwd"):
            s["opts"] = tdx.make_linear_opts(dw_dtype=code[case["dw"]])
        else:
            s["opts"] = tdx.make_combine_opts(out_dtype=s["dt"])
    return s


# ----------------------------------------------------------------------------------- own calls
def _own(s):
    c, tdx = s["case"], s["tdx"]
    op = c["op"]
    if op == "linear":
        tdx.check(tdx.tdx_linear(s["A"], s["B"], s["bias"], s["res"], s.get("row_scale"), s["C"], s["z"], c["M"],
                                 c["K"], c["N"], s["dt"], s["opts"]))
        return {"C": s["C"], "z": s["z"]}
    if op == "linear_act_bwd":
        tdx.check(tdx.tdx_linear_act_bwd(s["dy"], s["zin"], s["dz"], s["dbias"], s["ws"], c["M"], c["N"], s["dt"],
                                         s["opts"]))
        return {"dz": s["dz"], "dbias": s["dbias"]}
    if op == "linear_bwd":
        tdx.check(tdx.tdx_linear_bwd(s["dz"], s["A"], s["B"], s["res"], s["dA"], s["dB"], c["M"], c["K"], c["N"],
                                     s["dt"], s["opts"]))
        return {"dA": s["dA"], "dB": s["dB"]}
    if op == "grouped":
        tdx.check(tdx.tdx_grouped_gemm(s["A"], s["offsets"], s["B"], s.get("row_scale"), s.get("expert_scale"), s["C"],
                                       s["z"], c["R"], c["K"], c["N"], c["E"], s["dt"], s["opts"]))
        return {"C": s["C"], "z": s["z"]}
    if op == "grouped_bwd":
        tdx.check(tdx.tdx_grouped_gemm_bwd(s["dz"], s["A"], s["offsets"], s["B"], s["dA"], s["dB"], c["R"], c["K"],
                                           c["N"], c["E"], s["dt"], s["opts"]))
        return {"dA": s["dA"], "dB": s["dB"]}
    R = c["T"] * c["k"]
    if op == "combine":
        tdx.check(tdx.tdx_moe_combine(s["Z"], s["dest"], s["gates"], s["out"], R, c["T"], c["H"], c["k"], s["dt"],
                                      s["opts"]))
        return {"out": s["out"]}
    tdx.check(tdx.tdx_moe_combine_bwd(s["dout"], s["Z"], s["dest"], s["gates"], s["dZ"], s["dgates"], R, c["T"],
                                      c["H"], c["k"], s["dt"], s["opts"]))
    return {"dZ": s["dZ"], "dgates": s["dgates"]}


# ---------------------------------------------------------------------------------- plain form
def _e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _act(name, z):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * _sigmoid(2.0 * GELU_C * (z + GELU_D * z * z * z))
    if name == "silu":
        return z * _sigmoid(z)
    if name == "swiglu":
        half = z.shape[1] // 2
        return z[:, :half] * _sigmoid(z[:, :half]) * z[:, half:]
    return z


def _finish(s, acc, row_scale, bias, res):
    """The epilogue of a product: scales, bias, activation, residual, one rounding."""
    c = s["case"]
    if s["alpha"] != 1.0:
        acc = acc * s["alpha"]
    if row_scale is not None:
        acc = acc * row_scale[:, None]
    if bias is not None:
        acc = acc + bias.float()
    y = _act(c["act"], acc)
    if res is not None:
        y = y + res.float()
    y = _e4m3(y / _out_scale(c)) if c["out"] == "e4m3" else y.to(_TORCH[c["out"]])
    return y, acc.to(torch.bfloat16) if c["z"] else None


def _plain_linear(s):
    y, z = _finish(s, s["A"].float() @ s["B"].float(), s.get("row_scale"), s["bias"], s["res"])
    return {"C": y, "z": z}


def _plain_act_bwd(s):
    c = s["case"]
    dy = s["dy"].float()
    if c["act"] == "none":
        return {"dz": None, "dbias": dy.sum(0)}
    z = s["zin"].float()
    if c["act"] == "relu":
        dz = torch.where(z > 0, dy, torch.zeros_like(dy))
    elif c["act"] == "gelu":
        dz = dy * (0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    elif c["act"] == "gelu_tanh":
        p = _sigmoid(2.0 * GELU_C * (z + GELU_D * z * z * z))
        dz = dy * (p + z * p * (1.0 - p) * (2.0 * GELU_C * (1.0 + 3.0 * GELU_D * z * z)))
    elif c["act"] == "silu":
        p = _sigmoid(z)
        dz = dy * p * (1.0 + z * (1.0 - p))
    else:
        half = c["N"] // 2
        g, u = z[:, :half], z[:, half:]
        p = _sigmoid(g)
        dz = torch.cat([dy * u * p * (1.0 + g * (1.0 - p)), dy * g * p], 1)
    return {"dz": dz.to(torch.bfloat16), "dbias": dz.sum(0) if c["bias"] else None}


def _plain_linear_bwd(s):
    dz = s["dz"].float()
    dA = dz @ s["B"].float().t()
    if s["res"] is not None:
        dA = dA + s["res"].float()
    return {"dA": dA.to(torch.bfloat16), "dB": (s["A"].float().t() @ dz).to(_TORCH[s["case"]["dw"]])}


def _plain_grouped(s):
    c = s["case"]
    ys, zs, at = [], [], 0
    for e, n in enumerate(s["rows"]):
        if n == 0:
            continue
        acc = s["A"][at:at + n].float() @ s["B"][e].float()
        if "expert_scale" in s:
            acc = acc * s["expert_scale"][e]
        rs = s.get("row_scale")
        y, z = _finish(s, acc, None if rs is None else rs[at:at + n], None, None)
        ys.append(y)
        zs.append(z)
        at += n
    return {"C": torch.cat(ys), "z": torch.cat(zs) if c["z"] else None}


def _plain_grouped_bwd(s):
    dA, dB, at = [], [], 0
    dw = _TORCH[s["case"]["dw"]]
    for e, n in enumerate(s["rows"]):
        dz = s["dz"][at:at + n].float()
        dA.append((dz @ s["B"][e].float().t()).to(torch.bfloat16))
        dB.append((s["A"][at:at + n].float().t() @ dz).to(dw))
        at += n
    return {"dA": torch.cat(dA), "dB": torch.stack(dB)}


def _plain_combine(s):
    c = s["case"]
    at = s["dest"].long().view(c["T"], c["k"])
    out = torch.zeros(c["T"], c["H"], device="cuda")
    for j in range(c["k"]):
        z = s["Z"][at[:, j]].float()
        out = out + (z if s["gates"] is None else z * s["gates"][:, j, None])
    return {"out": out.to(_TORCH[c["dtype"]])}


def _plain_combine_bwd(s):
    c = s["case"]
    at = s["dest"].long().view(c["T"], c["k"])
    dout = s["dout"].float()
    dZ = torch.empty_like(s["Z"])
    dg = []
    for j in range(c["k"]):
        dZ[at[:, j]] = (dout if s["gates"] is None else dout * s["gates"][:, j, None]).to(dZ.dtype)
        if s["gates"] is not None:
            dg.append((dout * s["Z"][at[:, j]].float()).sum(1))
    return {"dZ": dZ, "dgates": torch.stack(dg, 1) if dg else None}


_PLAIN = {"linear": _plain_linear, "linear_act_bwd": _plain_act_bwd, "linear_bwd": _plain_linear_bwd,
          "grouped": _plain_grouped, "grouped_bwd": _plain_grouped_bwd, "combine": _plain_combine,
          "combine_bwd": _plain_combine_bwd}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------------------- in 64 bits
def _act64(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z.clamp_min(0.0)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        # 1 + tanh(u) = 2 sigmoid(2u), which does not cancel
        return z * torch.sigmoid((z + z.pow(3) * GELU_D) * (2.0 * GELU_C))
    gate, up = (z, None) if name == "silu" else z.chunk(2, 1)
    y = gate * torch.sigmoid(gate)
    return y if up is None else y * up


def _epilogue64(case, s, z, res):
    y = _act64(case["act"], z)
    if res is not None:
        y = y + res.double()
    if case["out"] == "e4m3":
        y = (y / _out_scale(case)).clamp(-E4M3_MAX, E4M3_MAX)
    return y


def _linear64(case, s):
    z = torch.matmul(s["A"].double(), s["B"].double()).mul_(s["alpha"])
    if s.get("row_scale") is not None:
        z *= s["row_scale"].double().unsqueeze(1)
    if s["bias"] is not None:
        z += s["bias"].double()
    return {"C": _epilogue64(case, s, z, s["res"]), "z": z if case["z"] else None}


def _act_bwd64(case, s):
    dy = s["dy"].double()
    if case["act"] == "none":
        return {"dz": None, "dbias": torch.einsum("mn->n", dy)}
    # the activation's own derivative, by automatic differentiation in pieces of rows
    dz = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
    step = max(1, (1 << 25) // case["N"])
    for a in range(0, case["M"], step):
        with torch.enable_grad():
            z = s["zin"][a:a + step].double().requires_grad_(True)
            (dz[a:a + step],) = torch.autograd.grad(_act64(case["act"], z), z, dy[a:a + step])
    return {"dz": dz, "dbias": torch.einsum("mn->n", dz) if case["bias"] else None}


def _linear_bwd64(case, s):
    dz = s["dz"].double()
    dA = torch.einsum("mn,kn->mk", dz, s["B"].double())
    if s["res"] is not None:
        dA += s["res"].double()
    return {"dA": dA, "dB": torch.einsum("mk,mn->kn", s["A"].double(), dz)}


def _grouped64(case, s):
    bounds = s["offsets"].tolist()
    z = torch.empty(case["R"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            f = float(s["expert_scale"][e]) if "expert_scale" in s else 1.0
            z[lo:hi] = torch.matmul(s["A"][lo:hi].double(), s["B"][e].double()) * (s["alpha"] * f)
    if s.get("row_scale") is not None:
        z *= s["row_scale"].double().unsqueeze(1)
    return {"C": _epilogue64(case, s, z, None), "z": z if case["z"] else None}


def _grouped_bwd64(case, s):
    bounds = s["offsets"].tolist()
    dA = torch.empty(case["R"], case["K"], dtype=torch.float64, device="cuda")
    dB = torch.zeros(case["E"], case["K"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            dz = s["dz"][lo:hi].double()
            dA[lo:hi] = torch.einsum("rn,kn->rk", dz, s["B"][e].double())
            dB[e] = torch.einsum("rk,rn->kn", s["A"][lo:hi].double(), dz)
    return {"dA": dA, "dB": dB}


def _token_pieces(case):
    step = max(1, (1 << 26) // (case["H"] * case["k"]))
    return [(a, min(case["T"], a + step)) for a in range(0, case["T"], step)]


def _combine64(case, s):
    k, parts = case["k"], []
    for a, b in _token_pieces(case):
        z = s["Z"].index_select(0, s["dest"][a * k:b * k].long()).double().view(b - a, k, case["H"])
        w = torch.ones(b - a, k, dtype=torch.float64, device="cuda") if s["gates"] is None else s["gates"][a:b].double()
        parts.append(torch.einsum("tk,tkh->th", w, z))
    return {"out": torch.cat(parts)}


def _combine_bwd64(case, s):
    k = case["k"]
    dZ = torch.empty(case["T"] * k, case["H"], dtype=torch.float64, device="cuda")
    dg = []
    for a, b in _token_pieces(case):
        at = s["dest"][a * k:b * k].long()
        dout = s["dout"][a:b].double()
        w = torch.ones(b - a, k, dtype=torch.float64, device="cuda") if s["gates"] is None else s["gates"][a:b].double()
        dZ.index_copy_(0, at, torch.einsum("tk,th->tkh", w, dout).reshape(-1, case["H"]))
        if s["gates"] is not None:
            dg.append(torch.einsum("th,tkh->tk", dout, s["Z"].index_select(0, at).double().view(b - a, k, -1)))
    return {"dZ": dZ, "dgates": torch.cat(dg) if dg else None}


_EXACT = {"linear": _linear64, "linear_act_bwd": _act_bwd64, "linear_bwd": _linear_bwd64, "grouped": _grouped64,
          "grouped_bwd": _grouped_bwd64, "combine": _combine64, "combine_bwd": _combine_bwd64}


def exact(case, seed):
    return _EXACT[case["op"]](case, _inputs(case, seed))
