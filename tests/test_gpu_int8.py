"""The int8 product, the int8 experts and the int8 layer against plain forms in 64 bits.

Bounds of the product: the sum is an exact integer; its conversion to fp32, the product of the
scales and the multiply-add round by 2^-24 each, then the output type by half a step."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_08_b200 import binding as B
from mixture_experts_ffn_08_b200 import inputs, workloads as W
from oracle import moe_oracle as o
from tests import int8_help as I8
from tests import parity as P

pytestmark = pytest.mark.gpu

KIND = {torch.bfloat16: B.MOE_OUT_BF16, torch.float16: B.MOE_OUT_FP16, torch.float32: B.MOE_OUT_FP32}


def linear(a, lda, sa, w, ldw, sw, bias, out, ldo, M, N, K, status=None, stream=None):
    B.check(B.moe_linear_int8(M, N, K, a, lda, sa, w, ldw, sw, bias, out, ldo, KIND[out.dtype], status, stream))


def linear_case(M, N, K, dtype=torch.bfloat16, bias=True, pad=(0, 0, 0), seed=0):
    """Inputs in wider rows, an output in wider rows, and the product's value and bound."""
    g = I8.gen(seed)
    a = I8.codes((M, K + pad[0]), g)
    w = I8.codes((N, K + pad[1]), g)
    sa, sw = I8.scales(M, g), I8.scales(N, g)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    out = torch.full((M, N + pad[2]), 55.0, dtype=dtype, device="cuda")
    acc = P.f64(a[:, :K]) @ P.f64(w[:, :K]).T  # integers below 2^31: exact in fp64
    prod = acc * P.f64(sa)[:, None] * P.f64(sw)[None, :]
    ref = prod + (P.f64(b)[None, :] if bias else 0.0)
    tol = np.abs(prod) * 2.0 ** -22.9 + np.abs(ref) * (2.0 ** -24 + I8.HALF_STEP[dtype]) * (1 + 2.0 ** -10) + 1e-7 * (
        dtype == torch.float16)
    return (a, K + pad[0], sa, w, K + pad[1], sw, b, out, N + pad[2], M, N, K), ref, tol


def check_linear(args, ref, tol):
    out, N = args[7], args[10]
    got = P.f64(out)
    assert (np.abs(got[:, :N] - ref) <= tol).all(), float(np.max(np.abs(got[:, :N] - ref) / tol))
    assert (got[:, N:] == 55.0).all()


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 100, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (31, 48), (33, 128), (64, 112), (255, 272), (1031, 1552), (2304, 384)])
def test_linear_sizes(M, N, K):
    dtype = (torch.bfloat16, torch.float16, torch.float32)[(M + N) % 3]
    args, ref, tol = linear_case(M, N, K, dtype, bias=M % 2 == 0, pad=((0, 0, 0), (16, 48, 5))[M % 2], seed=M)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    linear(*args, status=st)
    check_linear(args, ref, tol)
    assert st.item() == 0


@pytest.mark.parametrize("M,N,K", [(1100, 4200, 272), (2048, 2560, 1024), (2500, 2049, 144), (513, 9500, 80), (5000, 300, 64),
                                   (257, 2600, 4096), (20000, 40, 16), (100, 20000, 64), (16, 40000, 128)])
@pytest.mark.parametrize("dtype", list(KIND))
def test_linear_large(M, N, K, dtype):
    args, ref, tol = linear_case(M, N, K, dtype, pad=(32, 0, 3 if dtype == torch.bfloat16 else 8), seed=M)
    linear(*args)
    check_linear(args, ref, tol)


@pytest.mark.parametrize("M,N,K", [(8, 4096, 7168), (16, 64, 4096), (33, 40, 2048), (128, 300, 8192), (20, 1000, 512),
                                   (300, 2304, 384), (600, 1500, 2048), (5, 16, 16), (100, 4700, 640), (30, 4700, 640),
                                   (64, 2300, 1008), (128, 7168, 4096), (1, 5, 16), (4, 1000, 9008), (2, 333, 4112)])
@pytest.mark.parametrize("dtype", list(KIND))
def test_linear_few_rows(M, N, K, dtype):
    """One round of tiles: every width, one to eight parts of K, odd ends; and the one-row forms."""
    args, ref, tol = linear_case(M, N, K, dtype, pad=(16, 16, 0 if dtype == torch.float16 else 1), seed=M)
    linear(*args)
    check_linear(args, ref, tol)


# Shapes for which the launch rule (on 148 SMs) takes each tile width, number of A rows and number
# of parts; the first three have one to four rows on either side of the dot products' limit.
TILES = [(2, 256, 8208), (3, 301, 4112), (4, 4200, 2048),
         (5, 16, 32), (6, 17, 704), (7, 19, 800), (33, 16, 32), (37, 1096, 912), (34, 17, 896),
         (66, 16, 32), (130, 606, 1520), (68, 18, 976),
         (5, 4826, 32), (9, 2645, 1168), (32, 1064, 784), (35, 5155, 32), (37, 2399, 1968), (64, 1052, 1808),
         (142, 2378, 32), (65, 2393, 3344), (67, 1048, 3536),
         (5, 9484, 32), (13, 4969, 2000), (31, 2471, 1840), (33, 9890, 32), (35, 5156, 3552), (63, 2514, 3728),
         (129, 4819, 32), (67, 4753, 7984), (127, 2776, 7952), (120, 19001, 144), (16, 38100, 64)]


@pytest.mark.parametrize("M,N,K", TILES)
def test_linear_tiles(M, N, K):
    for i, dtype in enumerate(KIND):
        args, ref, tol = linear_case(M, N, K, dtype, bias=i == 1, pad=(0, 16, (0, 1, 8)[(M + i) % 3]), seed=M + i)
        linear(*args)
        check_linear(args, ref, tol)


@pytest.mark.parametrize("M", [1, 3, 20, 200])
def test_linear_longest_sum(M):
    """K = 131056 with every code -128: the sum 2147221504 is the largest that 32 bits hold here."""
    N, K = 40, 131056
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one_a, one_w = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    out = torch.zeros((M, N), device="cuda")
    linear(a, K, one_a, w, K, one_w, None, out, N, M, N, K)
    ref = np.where(np.arange(N) % 2 == 0, 128.0 * 128 * K, -128.0 * 127 * K)
    assert (np.abs(P.f64(out) - ref) <= np.abs(ref) * 2.0 ** -23).all()


@pytest.mark.parametrize("M", [1, 40, 600])
def test_linear_special_scales(M):
    """Infinite and NaN scales stay in their rows and columns; fp16 past its range is infinite."""
    N, K = 300, 64
    (a, lda, sa, w, ldw, sw, _, _, _, _, _, _), _, _ = linear_case(M, N, K, bias=False)
    a[:, 0], w[:, 0] = 127, 127
    a[:, 1:], w[:, 1:] = 0, 0
    sa.fill_(1.0)
    sw.fill_(0.001)
    sw[5], sw[6], sw[7], sw[8] = float("nan"), float("inf"), 0.0, 100.0
    out = torch.empty((M, N), dtype=torch.float16, device="cuda")
    linear(a, lda, sa, w, ldw, sw, None, out, N, M, N, K)
    col = out[:, 5:9].float()
    assert torch.isnan(col[:, 0]).all() and torch.isinf(col[:, 1]).all() and (col[:, 2] == 0).all()
    assert torch.isinf(col[:, 3]).all()
    rest = torch.cat([out[:, :5], out[:, 9:]], 1).float()
    assert (rest - 16.129).abs().max() <= 16.129 * (2.0 ** -11 + 2.0 ** -22)
    sa[0] = float("nan")
    linear(a, lda, sa, w, ldw, sw, None, out, N, M, N, K)
    assert torch.isnan(out[0]).all() and not torch.isnan(out[1:, 9:]).any()


@pytest.mark.parametrize("M", [1, 8, 60, 1500])
def test_linear_unaligned_output_and_parts(M):
    """An output that starts anywhere, inside a wider matrix: nothing beside it changes."""
    N, K = 130, 256
    for dtype in KIND:
        args, ref, tol = linear_case(M, N, K, dtype)
        big = torch.full((M, 3 * N + 7), 55.0, dtype=dtype, device="cuda")
        part = big[:, 1:]
        linear(*args[:7], part, 3 * N + 7, M, N, K)
        got = P.f64(big)
        assert (np.abs(got[:, 1:N + 1] - ref) <= tol).all()
        assert (got[:, 0] == 55.0).all() and (got[:, N + 1:] == 55.0).all()


def test_linear_streams_and_graph():
    """Two calls at once on two streams, and a captured one: the same bits as one after the other."""
    cases = [linear_case(*mnk, seed=i) for i, mnk in enumerate([(2, 700, 512), (70, 512, 2048), (1500, 2600, 512)])]
    want = []
    for args, ref, tol in cases:
        linear(*args)
        check_linear(args, ref, tol)
        want.append(args[7].clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for args, _, _ in cases:
            args[7].fill_(55.0)
        torch.cuda.synchronize()
        for s, (args, _, _) in zip(streams, cases):
            linear(*args, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(args[7], t) for (args, _, _), t in zip(cases, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for args, _, _ in cases:
            linear(*args)
    for _ in range(2):
        for args, _, _ in cases:
            args[7].fill_(55.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(args[7], t) for (args, _, _), t in zip(cases, want))


# ------------------------------------------------------------------------------------ experts
def bucketed(wl, d, ids):
    """moe_permute of the int8 x."""
    p = B.params(wl)
    ws = P.alloc_ws(p)
    rows = B.moe_max_padded_rows(p)
    ids = torch.as_tensor(np.asarray(ids), dtype=torch.int32, device="cuda")
    r = dict(counts=torch.empty(wl.E, dtype=torch.int32, device="cuda"),
             offs=torch.empty(wl.E + 1, dtype=torch.int32, device="cuda"),
             rop=torch.empty(wl.T * wl.K, dtype=torch.int32, device="cuda"),
             por=torch.full((rows,), -7, dtype=torch.int32, device="cuda"),
             xp=torch.full((rows, wl.H), 99, dtype=torch.int8, device="cuda"),
             xps=torch.full((rows,), 99.0, dtype=torch.float32, device="cuda"), ws=ws, ids=ids)
    B.check(B.moe_permute(p, ids, d["x_q"], d["x_scale"], r["counts"], r["offs"], r["rop"], r["por"], r["xp"], r["xps"],
                          ws, ws.numel()))
    return r


def run_ffn(wl, d, r, counts=True, offsets=True, ws=None, stream=None):
    p = B.params(wl)
    ws = r["ws"] if ws is None else ws
    y = torch.full((B.moe_max_padded_rows(p), wl.H), 33.0, dtype=torch.bfloat16, device="cuda")
    B.check(B.moe_expert_ffn(p, r["xp"], r["xps"], r["offs"] if offsets else None, r["counts"] if counts else None,
                             *I8.weight_args(d), y, ws, ws.numel(), stream))
    torch.cuda.synchronize()
    assert B.moe_get_device_status(ws) == 0
    return y


def rows_of_experts(wl, r):
    counts, offs = r["counts"].cpu().numpy(), r["offs"].cpu().numpy()
    return {e: np.arange(offs[e], offs[e] + counts[e]) for e in range(wl.E)}


def check_ffn(wl, d, r, y, what=""):
    rows = rows_of_experts(wl, r)
    x = o.dequant_rows(r["xp"].cpu().numpy(), r["xps"].cpu().numpy())
    got = P.f64(y)
    I8.check_ffn(got, rows, x, I8.expert_weights_fn(d), what)
    real = np.zeros(len(got), bool)
    for v in rows.values():
        real[v] = True
    assert (got[~real] == 33.0).all(), f"{what}: rows without a pair were written"


def skewed_ids(wl, seed, empty=0):
    """K different experts per token; the first `empty` experts get nothing, the last one a lot."""
    rng = np.random.default_rng(seed)
    ids = np.empty((wl.T, wl.K), np.int64)
    for t in range(wl.T):
        w = np.ones(wl.E - empty)
        w[-1] = 6.0
        ids[t] = empty + rng.choice(wl.E - empty, size=wl.K, replace=False, p=w / w.sum())
    return ids


@pytest.mark.parametrize("T,H,I,E,K,cap,empty", [
    (1, 128, 128, 1, 1, 0, 0), (1, 256, 128, 8, 2, 0, 0), (1, 256, 256, 8, 2, 128, 0), (33, 256, 128, 8, 2, 128, 3),
    (48, 384, 384, 16, 4, 0, 5), (129, 128, 640, 3, 2, 0, 0), (130, 640, 128, 4, 1, 256, 1), (40, 256, 128, 300, 8, 0, 0),
    (400, 256, 384, 3, 2, 0, 1),      # several M-tiles, an odd last one
    (700, 384, 256, 4, 2, 768, 0),    # the same in the masked layout
    (2000, 2560, 1280, 5, 2, 0, 1),   # enough tiles for pairs of CTAs in both products
    (2000, 2560, 1280, 5, 2, 2048, 0),
    (1500, 256, 256, 5, 3, 0, 2), (300, 1152, 128, 1, 1, 0, 0), (257, 128, 128, 1, 1, 0, 0),
    (64, 512, 512, 64, 2, 0, 1), (200, 2176, 384, 8, 2, 0, 0), (7, 1920, 640, 16, 4, 128, 1),
    (9, 128, 16512, 2, 1, 0, 0), (70, 128, 16640, 2, 2, 128, 0), (70, 128, 4224, 4, 2, 0, 1), (70, 128, 1152, 4, 2, 128, 1)])
def test_expert_ffn(T, H, I, E, K, cap, empty):
    wl = I8.INT8_SMALL.with_(T=T, H=H, I=I, E=E, K=K, masked_cap=cap)
    d = inputs.make_inputs(wl, seed=T, device="cuda")
    r = bucketed(wl, d, skewed_ids(wl, T, empty))
    # the rows carry the token's codes and scale
    por = r["por"].cpu().numpy()
    total = E * cap if cap else int(r["offs"][E])
    real = np.flatnonzero(por[:total] >= 0)
    toks = por[real] // K
    assert torch.equal(r["xp"][real].cpu(), d["x_q"][toks].cpu()) and torch.equal(r["xps"][real].cpu(), d["x_scale"][toks].cpu())
    y = run_ffn(wl, d, r)
    check_ffn(wl, d, r, y, str(wl))
    assert torch.equal(run_ffn(wl, d, r), y)
    if cap:
        assert torch.equal(run_ffn(wl, d, r, offsets=False), y)
    else:  # without counts the pad rows are computed too, the real rows stay
        z = run_ffn(wl, d, r, counts=False)
        assert torch.equal(z[real], y[real])


def test_expert_ffn_full_width():
    """The channels of the largest configurations, few experts, and rows of every small number."""
    for H, I in ((7168, 2048), (4096, 14336)):
        wl = I8.INT8_SMALL.with_(T=70, H=H, I=I, E=4, K=1)
        d = inputs.make_inputs(wl, seed=1, device="cuda")
        ids = np.repeat(np.arange(4), [1, 32, 33, 4])[:, None]
        r = bucketed(wl, d, ids)
        check_ffn(wl, d, r, run_ffn(wl, d, r), str(wl))


@pytest.mark.parametrize("T", [60, 700])
def test_expert_ffn_special_rows(T):
    """A zero row gives zeros; a row with a NaN or infinite scale gives NaN and nothing else does."""
    wl = I8.INT8_SMALL.with_(T=T, E=2, K=1)
    d = inputs.make_inputs(wl, seed=2, device="cuda")
    d["x_q"][3] = 0
    d["x_scale"][4], d["x_scale"][5] = float("nan"), float("inf")
    r = bucketed(wl, d, np.arange(T)[:, None] % 2)
    y = run_ffn(wl, d, r).float()
    rop = r["rop"].cpu().numpy()
    assert (y[rop[3]] == 0).all()
    assert torch.isnan(y[rop[4]]).all() and torch.isnan(y[rop[5]]).all()
    others = [rop[t] for t in range(T) if t not in (3, 4, 5)]
    assert torch.isfinite(y[others]).all()


@pytest.mark.parametrize("cap", [0, 128])
def test_expert_ffn_counts_past_the_layout(cap):
    """A count past its expert's rows, or a negative one, reads and writes nothing beyond them."""
    wl = I8.INT8_SMALL.with_(T=100, E=4, K=1, masked_cap=cap)
    d = inputs.make_inputs(wl, seed=2, device="cuda")
    r = bucketed(wl, d, np.arange(100)[:, None] % 3)
    y = run_ffn(wl, d, r)
    wrong = dict(r, counts=torch.tensor([1000000, -5, int(r["counts"][2]), 999999], dtype=torch.int32, device="cuda"))
    z = run_ffn(wl, d, wrong)
    rows = rows_of_experts(wl, r)
    assert torch.equal(z[rows[0]], y[rows[0]]) and torch.equal(z[rows[2]], y[rows[2]])
    assert (z[rows[1]] == 33.0).all()
    end = 4 * cap if cap else int(r["offs"][4])
    assert (z[end:] == 33.0).all()


def test_expert_ffn_same_expert_twice():
    """A token that names one expert K times fills K rows of its bucket."""
    wl = I8.INT8_SMALL.with_(T=70, E=4, K=3)
    d = inputs.make_inputs(wl, seed=3, device="cuda")
    r = bucketed(wl, d, np.full((70, 3), 2))
    check_ffn(wl, d, r, run_ffn(wl, d, r), "same expert")


def test_expert_ffn_streams_and_graphs():
    """Two layers at once, each with its workspace; two captured graphs that share one workspace
    replayed one after the other: the same bits."""
    cases = []
    for i, kw in enumerate((dict(T=40), dict(T=900, E=3))):
        wl = I8.INT8_SMALL.with_(**kw)
        d = inputs.make_inputs(wl, seed=i, device="cuda")
        r = bucketed(wl, d, skewed_ids(wl, i))
        cases.append((wl, d, r, run_ffn(wl, d, r), torch.cuda.Stream()))
    ys = [torch.zeros_like(c[3]) for c in cases]

    def call(i, stream, ws):
        wl, d, r, _, _ = cases[i]
        B.check(B.moe_expert_ffn(B.params(wl), r["xp"], r["xps"], r["offs"], r["counts"], *I8.weight_args(d), ys[i], ws,
                                 ws.numel(), stream))

    def check():
        torch.cuda.synchronize()
        for (wl, d, r, want, _), y in zip(cases, ys):
            for rows in rows_of_experts(wl, r).values():
                assert torch.equal(y[rows], want[rows])
            y.zero_()

    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        call(i, c[4], c[2]["ws"])
    check()
    shared = max((c[2]["ws"] for c in cases), key=lambda t: t.numel())
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, None, shared)
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
        check()


FIRST = """
import torch
from mixture_experts_ffn_08_b200 import binding as B, workloads as W
for M, N, K in ((1, 512, 512), (8, 512, 4096), (128, 2048, 1024), (500, 4096, 256), (4096, 4096, 128), (16, 20000, 128)):
    a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda")
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    one_a, one_w, out = torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), torch.zeros((M, N), device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.check(B.moe_linear_int8(M, N, K, a, K, one_a, w, K, one_w, None, out, N, B.MOE_OUT_FP32, None))
    g.replay()
    assert torch.equal(out.double(), a.double() @ w.double().T), (M, N, K)
for T, H, dtype in ((1, 7168, W.DTYPE_BF16), (300, 1024, W.DTYPE_BF16), (20, 20480, W.DTYPE_BF16)):
    p = B.params(W.Workload("first", T=T, H=H, I=128, E=2, K=1, dtype=dtype))
    x = torch.randn((T, H), device="cuda").bfloat16()
    w, out, again = torch.ones(H, device="cuda").bfloat16(), torch.zeros_like(x), torch.zeros_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.check(B.moe_add_rms_norm(p, x, None, w, 1e-6, None, out, None))
    g.replay()
    B.check(B.moe_add_rms_norm(p, x, None, w, 1e-6, None, again, None))
    assert torch.equal(out, again) and out.float().abs().sum() > 0
print("captured")
"""


def test_first_call_inside_a_capture():
    """A process whose first call of each kernel is captured: its one-time settings need no stream."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


# -------------------------------------------------------------------------------------- layer
LAYERS = [dict(), dict(T=1), dict(T=5, E=300, K=8, n_group=4, topk_group=2, group_topn=2, score_fn=W.SCORE_SIGMOID, has_bias=True),
          dict(T=300, E=4, masked_cap=384), dict(T=700, E=4, H=512, I=384), dict(T=1100, E=4), dict(T=40, skewed=True, E=16)]


@pytest.mark.parametrize("change", LAYERS, ids=str)
def test_layer(change):
    wl = I8.INT8_SMALL.with_(**change)
    d = inputs.make_inputs(wl, seed=4, device="cuda")
    r = I8.run_layer(wl, d)
    assert B.moe_get_device_status(r["ws"]) == 0
    x = o.dequant_rows(d["x_q"].cpu().numpy(), d["x_scale"].cpu().numpy())
    s = o.scores(o.router_logits(x, P.f64(d["w_r"])), wl.score_fn)
    ids = r["ids"].cpu().numpy()
    bias = P.f64(d["bias"]) if d["bias"] is not None else None
    _, wt = P.check_routing(ids, r["w"].cpu().numpy(), s, bias, wl)
    ref = o.forward_given_routing(x, ids, wt, I8.expert_weights_fn(d), wl.E, None, h_format="int8")
    P.check_close(P.f64(r["out"]), ref, P.FP8_MAX_TOL, "int8 layer")
    # the stages one by one give the layer's bits
    b = bucketed(wl, d, ids)
    y = run_ffn(wl, d, b)
    out = torch.empty_like(r["out"])
    B.check(B.moe_combine(B.params(wl), y, b["rop"], r["w"], None, out))
    assert torch.equal(out, r["out"]) and torch.equal(b["counts"], r["counts"])


def test_layer_masked_overflow():
    """An expert with more pairs than its rows keeps the first ones; the others add nothing."""
    wl = I8.INT8_SMALL.with_(T=300, E=1, K=1, masked_cap=128)
    d = inputs.make_inputs(wl, seed=6, device="cuda")
    r = I8.run_layer(wl, d)
    assert B.moe_get_device_status(r["ws"]) == B.MOE_DEV_CAPACITY and r["counts"].tolist() == [128]
    full = I8.run_layer(wl.with_(masked_cap=0), d)
    assert torch.equal(r["out"][:128], full["out"][:128]) and (r["out"][128:] == 0).all()


def test_layer_from_host_memory():
    wl = I8.INT8_SMALL
    p = B.params(wl)
    batches = [inputs.make_inputs(wl, seed=s, device="cuda") for s in range(3)]
    d = batches[0]
    ws = P.alloc_ws(p)
    want = []
    for b in batches:
        out = torch.empty((wl.T, wl.H), dtype=torch.bfloat16, device="cuda")
        B.check(B.moe_layer_forward(p, b["x_q"], b["x_scale"], *I8.layer_args(d)[2:], out, None, None, None, ws, ws.numel()))
        want.append(out.cpu())
    xs = [b["x_q"].cpu().pin_memory() for b in batches]
    ss = [b["x_scale"].cpu().pin_memory() for b in batches]
    outs = [torch.empty((wl.T, wl.H), dtype=torch.bfloat16).pin_memory() for _ in batches]
    B.check(B.moe_layer_forward_host(p, xs[1], ss[1], *I8.layer_args(d)[2:], outs[1], ws, ws.numel()))
    torch.cuda.synchronize()
    assert torch.equal(outs[1], want[1])
    B.check(B.moe_layer_forward_host_batches(p, xs, ss, *I8.layer_args(d)[2:], outs, ws, ws.numel()))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_permute_without_a_workspace():
    wl = I8.INT8_SMALL.with_(T=130)
    d = inputs.make_inputs(wl, seed=5, device="cuda")
    r = bucketed(wl, d, skewed_ids(wl, 5))
    xp, xps = torch.zeros_like(r["xp"]), torch.zeros_like(r["xps"])
    bufs = [torch.empty_like(r[n]) for n in ("counts", "offs", "rop", "por")]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.check(B.moe_permute_noalloc(B.params(wl), r["ids"], d["x_q"], d["x_scale"], *bufs, xp, xps, st))
    total = int(r["offs"][wl.E])
    assert torch.equal(xp[:total], r["xp"][:total]) and torch.equal(xps[:total], r["xps"][:total]) and st.item() == 0


@pytest.mark.parametrize("dtype", [W.DTYPE_BF16, W.DTYPE_FP8, W.DTYPE_FP8_FP4, W.DTYPE_INT8])
@pytest.mark.parametrize("T", [1, 70, 600])
def test_norm_layer_is_the_norm_and_the_layer(dtype, T):
    """moe_norm_layer_forward against its two calls, bit for bit, and through a captured graph."""
    wl = W.Workload("norm_layer", T=T, H=384, I=256, E=4, K=2, dtype=dtype,
                    I_shared=128 if dtype == W.DTYPE_BF16 else 0)
    d = inputs.make_inputs(wl, seed=6, device="cuda")
    if dtype == W.DTYPE_INT8:
        tail = I8.layer_args(d)[2:]
    else:
        a = P.device_inputs_ptrs(d, wl)
        tail = tuple(a[n] for n in ("w_r", "bias", "w_gate", "w_up", "w_down", "w_gate_scale", "w_up_scale", "w_down_scale",
                                    "ws_gate", "ws_up", "ws_down"))
    g = I8.gen(7)
    x = torch.randn((T, wl.H), generator=g, device="cuda").bfloat16()
    res = torch.randn((T, wl.H), generator=g, device="cuda").bfloat16()
    w = torch.rand(wl.H, generator=g, device="cuda").bfloat16()
    p = B.params(wl)
    y = torch.empty((T, wl.H), dtype=torch.bfloat16 if dtype == W.DTYPE_BF16 else torch.int8, device="cuda")
    ys = None if dtype == W.DTYPE_BF16 else torch.empty(T * (1 if dtype == W.DTYPE_INT8 else wl.H // 128), device="cuda")
    z, want = torch.empty_like(x), torch.empty_like(x)
    ids, wt = torch.empty((T, 2), dtype=torch.int32, device="cuda"), torch.empty((T, 2), device="cuda")
    counts = torch.empty(4, dtype=torch.int32, device="cuda")
    n = B.moe_workspace_size_norm(p)
    assert B.moe_workspace_size(p) < n <= B.moe_workspace_size_host(p)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    B.check(B.moe_clear_device_status(ws))
    B.check(B.moe_add_rms_norm(p, x, res, w, 1e-6, z, y, ys))
    B.check(B.moe_layer_forward(p, y, ys, *tail, want, ids, wt, counts, ws, ws.numel()))
    out, z2 = torch.zeros_like(x), torch.zeros_like(x)
    ids2, wt2, counts2 = torch.zeros_like(ids), torch.zeros_like(wt), torch.zeros_like(counts)

    def call():
        B.check(B.moe_norm_layer_forward(p, x, res, w, 1e-6, z2, *tail, out, ids2, wt2, counts2, ws, ws.numel()))

    def check():
        torch.cuda.synchronize()
        for a, b in ((out, want), (z2, z), (ids2, ids), (wt2, wt), (counts2, counts)):
            assert torch.equal(a, b)
            a.zero_()
        assert B.moe_get_device_status(ws) == 0

    call()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        graph.replay()
        check()
    # launches: the layer's, and the norm
    B.check(B.moe_trace_enable(0xFFFFFFFF, 64))
    call()
    B.moe_trace_disable()
    seen = [k for k, _ in B.moe_trace_collect()]
    assert len(seen) == B.moe_layer_launch_count(p) + 1 and seen[0] == B.K_NORM


@pytest.mark.parametrize("dtype", [W.DTYPE_FP8, W.DTYPE_INT8])
def test_norm_layer_keeps_a_bad_token_to_itself(dtype):
    """One token with a NaN: the other tokens' outputs are the ones without it, bit for bit."""
    wl = W.Workload("norm_layer", T=90, H=256, I=128, E=4, K=2, dtype=dtype)
    d = inputs.make_inputs(wl, seed=9, device="cuda")
    g = I8.gen(9)
    x = torch.randn((wl.T, wl.H), generator=g, device="cuda").bfloat16()
    w = torch.ones(wl.H, device="cuda").bfloat16()
    p = B.params(wl)
    ws = torch.empty(B.moe_workspace_size_norm(p), dtype=torch.uint8, device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            x[17, 3] = float("nan")
        B.check(B.moe_clear_device_status(ws))
        out = torch.zeros_like(x)
        B.check(B.moe_norm_layer_forward(p, x, None, w, 1e-6, None, *I8.layer_args(d)[2:], out, None, None, None, ws, ws.numel()))
        torch.cuda.synchronize()
        outs.append(out)
    rest = torch.arange(wl.T, device="cuda") != 17
    assert torch.equal(outs[0][rest], outs[1][rest])


def test_two_layers_in_a_row():
    """Two int8 layers as a decoder runs them: the residual stream and the norms between, against
    the chain in 64 bits on the kernels' own routing.  The bound is the layers' own, twice."""
    wl = I8.INT8_SMALL.with_(T=50, H=256, I=256)
    p = B.params(wl)
    g = I8.gen(8)
    x = torch.randn((wl.T, wl.H), generator=g, device="cuda").bfloat16()
    res = torch.zeros_like(x)
    ws = torch.empty(B.moe_workspace_size_norm(p), dtype=torch.uint8, device="cuda")
    B.check(B.moe_clear_device_status(ws))
    for layer in range(2):
        d = inputs.make_inputs(wl, seed=20 + layer, device="cuda")
        w = (1 + 0.1 * torch.randn(wl.H, generator=g, device="cuda")).bfloat16()
        before = (P.f64(x), P.f64(res))
        out = torch.empty_like(x)
        ids = torch.empty((wl.T, wl.K), dtype=torch.int32, device="cuda")
        wt = torch.empty((wl.T, wl.K), device="cuda")
        B.check(B.moe_norm_layer_forward(p, x, res, w, 1e-6, res, *I8.layer_args(d)[2:], out, ids, wt, None, ws, ws.numel()))
        z, y = o.add_rms_norm(*before, P.f64(w), 1e-6)
        np.testing.assert_array_equal(P.f64(res), z)
        ref = o.forward_given_routing(o.quantize_rows_int8(y), ids.cpu().numpy(), P.f64(wt), I8.expert_weights_fn(d), wl.E, None,
                                      h_format="int8")
        P.check_close(P.f64(out), ref, P.FP8_MAX_TOL, f"layer {layer}")
        x = out
