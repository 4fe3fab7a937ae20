"""The 8-bit operators around the MoE layer, as cases that can be run and timed.

Three operators belong together here: the root-mean-square norm that makes the layer's input (with
the residual's addition before it and the rounding to 8 bits behind it), the matrix product of
8-bit integers with one scale per token and one per output channel, and the experts' feed-forward
network made of such products.  `run` computes them from elementary torch operations, or, where
`own` is true, through the library's entry points.
"""
import math

import torch

own = False

# ------------------------------------------------------------------------------------- cases
#
# norm:   out = norm(x + residual) * w for T tokens of H channels, in the input format of a layer
#         ("bf16"; "e4m3" with a power-of-two scale per 128 channels; "int8" with a scale per token).
# linear: out[M, N] = a[M, K] w[N, K]^T, int8 codes times a_scale[M] and w_scale[N] (+ bias).  `pad`
#         codes of other data lie between the rows of a.
# ffn:    the experts' SwiGLU network on T*K rows bucketed by expert, int8.  `cap` > 0: every expert
#         owns cap rows (masked layout), else the buckets are padded to 128 rows.  `skew` is the
#         standard deviation of the experts' log popularity.


def listed():
    return [
        # one token of a decode step, the latency of a single launch
        {"name": "norm_bf16_one_token", "op": "norm", "T": 1, "H": 7168, "to": "bf16", "residual": True},
        # a decode batch in front of an int8 layer
        {"name": "norm_int8_decode", "op": "norm", "T": 128, "H": 7168, "to": "int8", "residual": True},
        # the first norm of a stack (no residual yet), a ragged number of tokens, 33 blocks of channels
        {"name": "norm_e4m3_first", "op": "norm", "T": 1023, "H": 4224, "to": "e4m3", "residual": False},
        # a long prefill in front of an e4m3 layer
        {"name": "norm_e4m3_prefill", "op": "norm", "T": 16384, "H": 7168, "to": "e4m3", "residual": True},
        # one token through a projection: the weights are read once, nothing else counts
        {"name": "linear_one_token", "op": "linear", "M": 1, "N": 4096, "K": 7168, "to": "bf16", "bias": False, "pad": 0},
        # odd sizes, a part of wider rows, fp32 for a head that sums on
        {"name": "linear_ragged", "op": "linear", "M": 77, "N": 1031, "K": 1552, "to": "fp32", "bias": True, "pad": 48},
        # a decode batch through a projection
        {"name": "linear_decode", "op": "linear", "M": 128, "N": 7168, "K": 4096, "to": "bf16", "bias": False, "pad": 0},
        # a prefill through the wide projection of a dense feed-forward network
        {"name": "linear_prefill", "op": "linear", "M": 8192, "N": 14336, "K": 4096, "to": "fp16", "bias": False, "pad": 0},
        # a handful of tokens through small experts in the masked layout
        {"name": "ffn_small_masked", "op": "ffn", "T": 33, "H": 256, "I": 128, "E": 8, "K": 2, "cap": 128, "skew": 1.0},
        # a decode step of 256 experts: all experts' weights for four rows each
        {"name": "ffn_decode", "op": "ffn", "T": 128, "H": 7168, "I": 2048, "E": 256, "K": 8, "cap": 0, "skew": 0.3},
        # a prefill over 128 narrow experts of uneven load
        {"name": "ffn_prefill", "op": "ffn", "T": 16384, "H": 4096, "I": 1536, "E": 128, "K": 8, "cap": 0, "skew": 0.4},
        # a prefill over eight wide experts
        {"name": "ffn_prefill_wide", "op": "ffn", "T": 4096, "H": 4096, "I": 14336, "E": 8, "K": 2, "cap": 0, "skew": 0.2},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "ffn"])
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 16384), "H": 128 * _log(rng, 1, 56), "to": rng.choice(["bf16", "e4m3", "int8"]),
                "residual": rng.random() < 0.7}
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 17, 14336), "K": 16 * _log(rng, 2, 448),
                "to": rng.choice(["bf16", "fp16", "fp32"]), "bias": rng.random() < 0.5, "pad": 16 * rng.choice([0, 0, 1, 3, 8])}
    while True:
        E = _log(rng, 1, 256)
        c = {"op": op, "T": _log(rng, 1, 16384), "H": 128 * _log(rng, 1, 56), "I": 128 * _log(rng, 1, 112), "E": E,
             "K": min(E, rng.randint(1, 8)), "cap": 0, "skew": round(rng.uniform(0.0, 0.5), 2)}
        if rng.random() < 0.3:  # room for every token in every expert
            c["cap"] = (c["T"] + 127) // 128 * 128
        flops = 6 * c["T"] * c["K"] * c["H"] * c["I"]
        rows = c["E"] * c["cap"] if c["cap"] else 3 * c["T"] * c["K"] + 128 * E
        if flops <= 4e12 and E * c["H"] * c["I"] <= 1.5e9 and rows * max(c["H"], 3 * c["I"]) <= 2e9:
            return c


# ------------------------------------------------------------------------------------ inputs
_OUT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _codes(shape, g, std=36.0):
    """Codes of normally distributed values whose rows' largest lies near 127."""
    return torch.randn(shape, generator=g, device="cuda").mul_(std).round_().clamp_(-127, 127).to(torch.int8)


def _weights(n, rows, cols, g):
    """n matrices of codes [rows, cols], and a scale for each row, of weights of standard deviation 0.02."""
    q = torch.empty((n, rows, cols), dtype=torch.int8, device="cuda")
    for e in range(n):
        q[e] = _codes((rows, cols), g)
    s = (0.02 / 36.0) * (0.8 + 0.4 * torch.rand((n, rows), generator=g, device="cuda"))
    return q, s


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    loud = torch.ones(H, device="cuda")  # a few channels are much larger than the others
    loud[torch.randperm(H, generator=g, device="cuda")[: max(1, H // 128)]] = 20.0
    st = {"x": (torch.randn((T, H), generator=g, device="cuda") * loud).to(torch.bfloat16), "residual": None,
          "w": (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)}
    if c["residual"]:
        st["residual"] = (torch.randn((T, H), generator=g, device="cuda") * loud * 4.0).to(torch.bfloat16)
    st["eps"] = 1e-6
    st["sum"] = torch.empty_like(st["x"]) if c["residual"] else None
    st["out"] = torch.empty((T, H), dtype={"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}[c["to"]],
                            device="cuda")
    st["scale"] = None
    if c["to"] != "bf16":
        st["scale"] = torch.empty((T, H // 128) if c["to"] == "e4m3" else (T,), dtype=torch.float32, device="cuda")
    st["values"] = torch.empty_like(st["x"])
    return st


def _prepare_linear(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    st = {"a": _codes((M, K + c["pad"]), g)[:, :K], "a_scale": (4.0 / 127.0) * (0.5 + torch.rand(M, generator=g, device="cuda"))}
    w, s = _weights(1, N, K, g)
    st["w"], st["w_scale"] = w[0], s[0]
    st["bias"] = torch.randn(N, generator=g, device="cuda") if c["bias"] else None
    st["out"] = torch.empty((M, N), dtype=_OUT[c["to"]], device="cuda")
    return st


def _prepare_ffn(c, g):
    T, H, I, E, K, cap = c["T"], c["H"], c["I"], c["E"], c["K"], c["cap"]
    # the router's choice: K different experts for each token, by popularity
    taste = torch.randn(E, generator=g, device="cuda") * c["skew"]
    luck = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)))
    ids = (luck + taste).topk(K, dim=1).indices
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    room = torch.full_like(counts, cap) if cap else (counts + 127) // 128 * 128
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = room.cumsum(0)
    rows = E * cap if cap else T * K + E * 127
    most = int(counts.max())
    # real row r is number `at[r]` of the [E, most] table of rows, and row `real[r]` of the buckets
    slot = torch.arange(most, device="cuda")
    valid = slot[None, :] < counts[:, None]
    table = (offsets[:E, None] + slot[None, :]).clamp_(max=rows - 1)
    at = valid.reshape(-1).nonzero().reshape(-1)
    real = table.reshape(-1)[at]
    x = torch.zeros((rows, H), dtype=torch.int8, device="cuda")
    x_scale = torch.ones(rows, device="cuda")
    for i in range(0, real.numel(), 16384):
        r = real[i:i + 16384]
        x[r] = _codes((r.numel(), H), g)
        x_scale[r] = (4.0 / 127.0) * (0.5 + torch.rand(r.numel(), generator=g, device="cuda"))
    st = {"x": x, "x_scale": x_scale, "counts": counts.to(torch.int32), "offsets": offsets.to(torch.int32),
          "table": table, "at": at, "real": real}
    st["w_gate"], st["s_gate"] = _weights(E, I, H, g)
    st["w_up"], st["s_up"] = _weights(E, I, H, g)
    st["w_down"], st["s_down"] = _weights(E, H, I, g)
    st["y"] = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    st["ws"] = torch.zeros(_workspace_bytes(c, rows), dtype=torch.uint8, device="cuda")
    return st


def _workspace_bytes(c, rows):
    """More than the library asks for any of these cases (its own answer is asked for where it runs)."""
    T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
    return rows * (12 * I + 8 * H + 1024) + 256 * 14 * I + T * (4 * H + 128 * E + 64 * K) + T * K * E // 32 + 64 * E + (1 << 20)


def prepare(case, seed):
    st = {"norm": _prepare_norm, "linear": _prepare_linear, "ffn": _prepare_ffn}[case["op"]](case, _gen(seed))
    st["case"] = case
    return st


# -------------------------------------------------------------------------------- plain forms
def _plain_norm(st):
    c = st["case"]
    # the codes' borders and the scales' powers of two are decided in 64 bits
    wide = torch.float32 if c["to"] == "bf16" else torch.float64
    z = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(torch.bfloat16)
    v = z.to(wide)
    y = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + st["eps"]) * st["w"].to(wide)
    res = {} if st["residual"] is None else {"sum": z}
    if c["to"] == "bf16":
        return {**res, "out": y.to(torch.bfloat16)}
    if c["to"] == "e4m3":
        b = y.reshape(c["T"], c["H"] // 128, 128)
        m, e = torch.frexp(b.abs().amax(dim=2) / 448.0)
        s = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
        s = torch.where(m > 0, s, torch.ones_like(s))
        q = (b / s[:, :, None]).reshape(c["T"], c["H"]).float().to(torch.float8_e4m3fn)
        return {**res, "out": q, "scale": s.float()}
    amax = y.abs().amax(dim=1)
    s = torch.where(amax > 0, amax / 127.0, torch.ones_like(amax))
    q = torch.round(y / s[:, None])
    return {**res, "out": (q * s.float()[:, None]).to(torch.bfloat16), "scale": s.float()}


def _plain_linear(st):
    acc = st["a"].float() @ st["w"].float().t()
    y = acc * st["a_scale"][:, None] * st["w_scale"][None, :]
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(st["out"].dtype)


def _plain_ffn(st):
    x = st["x"][st["table"]].float()  # [E, most, H], with rows of others behind each expert's own
    xs = st["x_scale"][st["table"]][:, :, None]
    gate = torch.bmm(x, st["w_gate"].float().transpose(1, 2)) * xs * st["s_gate"][:, None, :]
    up = torch.bmm(x, st["w_up"].float().transpose(1, 2)) * xs * st["s_up"][:, None, :]
    h = gate / (1.0 + torch.exp(-gate)) * up
    amax = h.abs().amax(dim=2, keepdim=True)
    hs = torch.where(amax > 0, amax / 127.0, torch.ones_like(amax))
    q = torch.round(h / hs)
    y = torch.bmm(q, st["w_down"].float().transpose(1, 2)) * hs * st["s_down"][:, None, :]
    out = torch.zeros_like(st["y"])
    out[st["real"]] = y.reshape(-1, y.shape[2])[st["at"]].to(torch.bfloat16)
    return out


# ------------------------------------------------------------------------- the library's calls
def _params(B, W, c, T, H, I, E, K, cap):
    dtype = {"bf16": W.DTYPE_BF16, "e4m3": W.DTYPE_FP8, "int8": W.DTYPE_INT8}[c.get("to", "int8")]
    return B.params(W.Workload("operators", T=T, H=H, I=I, E=E, K=K, dtype=dtype, masked_cap=cap))


def _own_norm(st):
    from mixture_experts_ffn_08_b200 import binding as B, workloads as W
    c = st["case"]
    if "p" not in st:
        st["p"] = _params(B, W, c, c["T"], c["H"], 128, 1, 1, 0)
    B.check(B.moe_add_rms_norm(st["p"], st["x"], st["residual"], st["w"], st["eps"], st["sum"], st["out"], st["scale"]))
    res = {} if st["residual"] is None else {"sum": st["sum"]}
    if c["to"] == "bf16":
        return {**res, "out": st["out"]}
    out = st["out"]
    if c["to"] == "int8":
        out = torch.mul(out, st["scale"][:, None], out=st["values"])
    return {**res, "out": out, "scale": st["scale"]}


def _own_linear(st):
    from mixture_experts_ffn_08_b200 import binding as B
    c = st["case"]
    kind = {"bf16": B.MOE_OUT_BF16, "fp16": B.MOE_OUT_FP16, "fp32": B.MOE_OUT_FP32}[c["to"]]
    B.check(B.moe_linear_int8(c["M"], c["N"], c["K"], st["a"], c["K"] + c["pad"], st["a_scale"], st["w"], c["K"], st["w_scale"],
                              st["bias"], st["out"], c["N"], kind, None))
    return st["out"]


def _own_ffn(st):
    from mixture_experts_ffn_08_b200 import binding as B, workloads as W
    c = st["case"]
    if "p" not in st:
        st["p"] = _params(B, W, c, c["T"], c["H"], c["I"], c["E"], c["K"], c["cap"])
        if B.moe_workspace_size(st["p"]) > st["ws"].numel():
            st["ws"] = torch.zeros(B.moe_workspace_size(st["p"]), dtype=torch.uint8, device="cuda")
    B.check(B.moe_expert_ffn(st["p"], st["x"], st["x_scale"], st["offsets"], st["counts"], st["w_gate"], st["w_up"], st["w_down"],
                             st["s_gate"], st["s_up"], st["s_down"], st["y"], st["ws"], st["ws"].numel()))
    return st["y"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "ffn": _own_ffn}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "ffn": _plain_ffn}[op](state)


# --------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["H"]
        bytes_ = 2 * n + (4 * n if c["residual"] else 0) + 2 * c["H"]
        bytes_ += {"bf16": 2 * n, "e4m3": n + 4 * n // 128, "int8": n + 4 * c["T"]}[c["to"]]
        return {"bytes": bytes_, "flops": 5 * n}
    if c["op"] == "linear":
        size = 4 if c["to"] == "fp32" else 2
        return {"bytes": c["M"] * c["K"] + c["N"] * c["K"] + size * c["M"] * c["N"] + 4 * (c["M"] + c["N"] * (2 if c["bias"] else 1)),
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
    active = E * (1.0 - (1.0 - K / E) ** T)  # experts with a row, for an even load
    return {"bytes": active * (3 * H * I + 4 * (2 * I + H)) + T * K * (3 * H + 4), "flops": 6 * T * K * H * I}


# ------------------------------------------------------------------------------ in 64 bits
def _grid_e4m3(v):
    """The nearest e4m3 value, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_norm(c, st):
    x = st["x"].double()
    res = {}
    if c["residual"]:
        x = (x + st["residual"].double()).to(torch.bfloat16)  # the sum is stored in bf16 and the norm is of that
        res = {"sum": x.double()}
        x = x.double()
    y = st["w"].double() * (x / torch.sqrt(x.square().sum(dim=1, keepdim=True) / c["H"] + st["eps"]))
    if c["to"] == "bf16":
        return {**res, "out": y}
    if c["to"] == "int8":
        s = y.abs().amax(dim=1) / 127.0
        s[s == 0] = 1.0
        return {**res, "out": torch.round(y / s[:, None]) * s[:, None], "scale": s}
    blocks = y.unflatten(1, (-1, 128))
    top = blocks.abs().amax(dim=2)
    s = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
    s[top == 0] = 1.0
    return {**res, "out": _grid_e4m3(blocks / s[:, :, None]).flatten(1), "scale": s}


def _exact_linear(c, st):
    out = torch.empty((c["M"], c["N"]), dtype=torch.float64, device="cuda")
    w = st["w"].double() * st["w_scale"].double()[:, None]
    for i in range(0, c["M"], 2048):
        out[i:i + 2048] = (st["a"][i:i + 2048].double() * st["a_scale"][i:i + 2048, None].double()) @ w.t()
    return out if st["bias"] is None else out.add_(st["bias"].double())


def _exact_ffn(c, st):
    out = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
    counts, offsets = st["counts"].tolist(), st["offsets"].tolist()
    for e in range(c["E"]):
        if not counts[e]:
            continue
        r = slice(offsets[e], offsets[e] + counts[e])
        x = st["x"][r].double() * st["x_scale"][r, None].double()
        g = x @ (st["w_gate"][e].double() * st["s_gate"][e, :, None].double()).t()
        u = x @ (st["w_up"][e].double() * st["s_up"][e, :, None].double()).t()
        h = g * torch.sigmoid(g) * u
        s = h.abs().amax(dim=1, keepdim=True) / 127.0
        s[s == 0] = 1.0
        out[r] = (torch.round(h / s) * s) @ (st["w_down"][e].double() * st["s_down"][e, :, None].double()).t()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "ffn": _exact_ffn}[case["op"]](case, st)
