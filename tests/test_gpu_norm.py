"""moe_add_rms_norm against its formula in 64 bits.

Bounds: z, a sum of two bf16 numbers rounded to bf16, is exact.  y carries the roundings of
rstd (2^-24) and of one product (2^-24; z w is exact): 2^-22 of itself with room, and then half
a step of the format: bf16 2^-8 of the value, e4m3 2^-4 of the value or 2^-10 of the scale
(subnormal codes), int8 half a code.  An e4m3 scale is the power of two exactly; the sum of
squares is good to 2^-24, so only an amax within 2^-22 of a border may take the other one."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_08_b200 import binding as B
from mixture_experts_ffn_08_b200 import workloads as W
from oracle import moe_oracle as o
from tests import int8_help as I8
from tests import parity as P

pytestmark = pytest.mark.gpu

EPS = 1e-6
FORMATS = {"bf16": W.DTYPE_BF16, "e4m3": W.DTYPE_FP8, "fp4": W.DTYPE_FP8_FP4, "int8": W.DTYPE_INT8}
STEP = 2.0 ** -22


def params(T, H, fmt):
    return B.params(W.Workload("norm", T=T, H=H, I=128, E=2, K=1, dtype=FORMATS[fmt]))


def inputs(T, H, seed=0, residual=True, spread=1.0):
    g = I8.gen(seed)
    loud = torch.where(torch.rand(H, generator=g, device="cuda") < 0.02, 30.0, 1.0)
    x = (torch.randn((T, H), generator=g, device="cuda") * loud * spread).bfloat16()
    r = (torch.randn((T, H), generator=g, device="cuda") * loud * 4 * spread).bfloat16() if residual else None
    w = (1.0 + 0.3 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    return x, r, w


def outputs(T, H, fmt):
    out = torch.full((T, H), 77, dtype=torch.bfloat16 if fmt == "bf16" else torch.int8, device="cuda")
    scale = None
    if fmt != "bf16":
        scale = torch.full((T, H // 128) if fmt in ("e4m3", "fp4") else (T,), -1.0, device="cuda")
    return out, scale


def check(fmt, x, r, w, out, scale, eps=EPS):
    z, y = o.add_rms_norm(P.f64(x), None if r is None else P.f64(r), P.f64(w), eps)
    T, H = y.shape
    if fmt == "bf16":
        assert (np.abs(P.f64(out) - y) <= np.abs(y) * (2.0 ** -8 + STEP) + 1e-38).all()
        return z
    if fmt == "int8":
        s = o.int8_scale(np.abs(y).max(axis=1))
        got_s = P.f64(scale)
        assert (np.abs(got_s - s) <= s * STEP).all()
        v = y / s[:, None]
        q = P.f64(out)
        assert np.abs(q).max() <= 127
        assert (np.abs(q - v) <= 0.5 + np.abs(v) * STEP).all()
        return z
    amax = np.abs(y.reshape(T, H // 128, 128)).max(axis=2)
    s, got_s = o.pow2_scale(amax), P.f64(scale)
    near = np.abs(amax / (448.0 * s) - 1) <= STEP
    near |= np.abs(amax / (224.0 * s) - 1) <= STEP
    assert ((got_s == s) | near & ((got_s == 2 * s) | (got_s == s / 2))).all()
    sb = np.repeat(got_s, 128, axis=1)
    v = o.decode_e4m3(out.view(torch.uint8).cpu().numpy()) * sb
    assert (np.abs(v - y) <= np.maximum(np.abs(y) * 2.0 ** -4, sb * 2.0 ** -10) * (1 + 2.0 ** -10)).all()
    return z


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (3, 384), (5, 8192), (2, 8320), (700, 1152), (1500, 4224),
                                 (2, 16384), (2, 16512), (300, 20608), (3, 26624), (2, 26752), (2, 32896)])
def test_formula(fmt, T, H):
    """Sizes of every variant: one vector per thread, two, four, and rows past the registers."""
    for residual in (True, False):
        x, r, w = inputs(T, H, seed=T + H, residual=residual)
        out, scale = outputs(T, H, fmt)
        total = torch.zeros_like(x) if residual else None
        B.check(B.moe_add_rms_norm(params(T, H, fmt), x, r, w, EPS, total, out, scale))
        z = check(fmt, x, r, w, out, scale)
        if residual:
            np.testing.assert_array_equal(P.f64(total), z)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("T,H", [(4, 1024), (600, 1024), (200, 16640), (3, 33024)])
def test_in_place_and_without_the_sum(fmt, T, H):
    x, r, w = inputs(T, H, seed=3)
    p = params(T, H, fmt)
    want, want_s = outputs(T, H, fmt)
    total = torch.empty_like(x)
    B.check(B.moe_add_rms_norm(p, x, r, w, EPS, total, want, want_s))
    for where in ("residual", "x", "none"):
        x2, r2 = x.clone(), r.clone()
        out, scale = outputs(T, H, fmt)
        B.check(B.moe_add_rms_norm(p, x2, r2, w, EPS, {"residual": r2, "x": x2, "none": None}[where], out, scale))
        assert torch.equal(out, want) and (scale is None or torch.equal(scale, want_s))
        assert torch.equal(r2, total if where == "residual" else r)
        assert torch.equal(x2, total if where == "x" else x)
    if fmt == "bf16":  # the output over x
        out, _ = outputs(T, H, fmt)
        B.check(B.moe_add_rms_norm(p, x, None, w, EPS, None, out, None))
        x2 = x.clone()
        B.check(B.moe_add_rms_norm(p, x2, None, w, EPS, None, x2, None))
        assert torch.equal(x2, out)


@pytest.mark.parametrize("T", [6, 700])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_zero_and_non_finite_rows(fmt, T):
    H = 256
    x, _, w = inputs(T, H, seed=9, residual=False)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3, 0] = 3e38   # its square passes fp32
    x[4] = x[4] * 1e-30
    out, scale = outputs(T, H, fmt)
    B.check(B.moe_add_rms_norm(params(T, H, fmt), x, None, w, EPS, None, out, scale))
    good = [0, 4] + list(range(5, T))
    check(fmt, x[good], None, w, out[good], None if scale is None else scale[good])
    if fmt == "bf16":
        assert torch.isnan(out[1]).all() and torch.isnan(out[2, 200]) and (out[0] == 0).all()
    else:
        assert (out[:4] == 0).all() and torch.isnan(scale[1:4]).all() and (scale[0] == 1).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int8"])
def test_tiny_outputs_and_weights(fmt):
    """Weights down to the smallest numbers: scales stay normal numbers, codes follow them."""
    T, H = 4, 256
    x, _, w = inputs(T, H, seed=4, residual=False)
    for factor in (1e-20, 1e-33, 0.0):
        wt = (w.float() * factor).bfloat16()
        out, scale = outputs(T, H, fmt)
        B.check(B.moe_add_rms_norm(params(T, H, fmt), x, None, wt, EPS, None, out, scale))
        check(fmt, x, None, wt, out, scale)
    # outputs below 127 * 2^-126: the scale stops at 2^-126 and the codes shrink
    wt = (w.float() * 2e-38).bfloat16()
    out, scale = outputs(T, H, fmt)
    B.check(B.moe_add_rms_norm(params(T, H, fmt), x, None, wt, EPS, None, out, scale))
    _, y = o.add_rms_norm(P.f64(x), None, P.f64(wt), EPS)
    if fmt == "int8":
        assert (scale == 2.0 ** -126).all()
        v = y * 2.0 ** 126
        assert (np.abs(P.f64(out) - v) <= 0.5 + np.abs(v) * STEP).all()
    elif fmt == "e4m3":
        assert (scale >= 2.0 ** -126).all()


def test_eps_and_scaling():
    """eps decides for small rows; the 8-bit codes of a row do not depend on its size."""
    T, H = 8, 512
    x, _, w = inputs(T, H, seed=5, residual=False, spread=1e-4)
    for eps in (1e-12, 1e-5, 1.0):
        out, _ = outputs(T, H, "bf16")
        B.check(B.moe_add_rms_norm(params(T, H, "bf16"), x, None, w, eps, None, out, None))
        check("bf16", x, None, w, out, None, eps=float(np.float32(eps)))
    q1, s1 = outputs(T, H, "int8")
    q2, s2 = outputs(T, H, "int8")
    p = params(T, H, "int8")
    B.check(B.moe_add_rms_norm(p, x, None, w, EPS, None, q1, s1))
    B.check(B.moe_add_rms_norm(p, x * 64, None, w, EPS, None, q2, s2))
    assert torch.equal(q1, q2) and (s2 > s1).all()


def test_streams_and_graph():
    """On another stream, captured and replayed, two graphs of the same buffers: the same bits."""
    T, H = 33, 1024
    x, r, w = inputs(T, H, seed=6)
    p = params(T, H, "int8")
    want, want_s = outputs(T, H, "int8")
    B.check(B.moe_add_rms_norm(p, x, r, w, EPS, None, want, want_s))
    torch.cuda.synchronize()
    out, scale = outputs(T, H, "int8")
    s = torch.cuda.Stream()
    B.check(B.moe_add_rms_norm(p, x, r, w, EPS, None, out, scale, s))
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(scale, want_s)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.check(B.moe_add_rms_norm(p, x, r, w, EPS, None, out, scale))
        graphs.append(g)
    for g in graphs:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(scale, want_s)


def test_two_threads():
    """Rows of different lengths from two threads at once, each on its own stream."""
    import threading
    failed = []

    def run(H):
        x, r, w = inputs(200, H, seed=H)
        p = params(200, H, "int8")
        want, want_s = outputs(200, H, "int8")
        B.check(B.moe_add_rms_norm(p, x, r, w, EPS, None, want, want_s))
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        out, scale = outputs(200, H, "int8")
        torch.cuda.synchronize()
        try:
            for _ in range(300):
                B.check(B.moe_add_rms_norm(p, x, r, w, EPS, None, out, scale, s))
            s.synchronize()
            assert torch.equal(out, want) and torch.equal(scale, want_s)
        except Exception as e:  # (a thread's exception is otherwise lost)
            failed.append(e)

    threads = [threading.Thread(target=run, args=(H,)) for H in (8192, 16384)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_feeds_the_e4m3_layer():
    """The e4m3 output is what the generator's quantiser makes of the same values."""
    from mixture_experts_ffn_08_b200 import inputs as gen_inputs
    T, H = 64, 1024
    x, r, w = inputs(T, H, seed=7)
    out, scale = outputs(T, H, "e4m3")
    B.check(B.moe_add_rms_norm(params(T, H, "e4m3"), x, r, w, EPS, None, out, scale))
    _, y = o.add_rms_norm(P.f64(x), P.f64(r), P.f64(w), EPS)
    q, s = gen_inputs.quantize_blocks_e4m3(torch.from_numpy(y), 1)
    assert torch.equal(s.float(), scale.cpu())
    # rounding the exact y once in fp64 may give the neighbouring code only next to a border
    assert (q != out.view(torch.uint8).cpu()).float().mean() < 1e-4
