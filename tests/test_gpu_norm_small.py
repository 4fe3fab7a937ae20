"""moe_add_rms_norm where its intermediate values are far from 1, and where a code is a tie.

e4m3: the bounds of test_gpu_norm.py, with scales that stop at 2^-126.  The products z w of these
inputs are exact in fp32 (inputs that would not be are zeros), so nothing else rounds."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_08_b200 import binding as B
from mixture_experts_ffn_08_b200 import inputs, workloads as W
from oracle import moe_oracle as o
from tests import int8_help as I8
from tests import parity as P

pytestmark = pytest.mark.gpu

EPS = 1e-6
STEP = 2.0 ** -22
SMALLEST = 2.0 ** -133  # of bf16


def params(T, H, dtype):
    return B.params(W.Workload("norm", T=T, H=H, I=128, E=2, K=1, dtype=dtype))


def exact_products(x, w):
    """x with zeros where z w is not exact in fp32."""
    prod = x.double() * w.double()
    return torch.where(prod.float().double() == prod, x, torch.zeros_like(x))


def small_inputs(kind, T, H, g):
    x = torch.randn((T, H), generator=g, device="cuda")
    w = 1.0 + 0.3 * torch.randn(H, generator=g, device="cuda")
    x[torch.rand((T, H), generator=g, device="cuda") < 0.3] = 0.0
    if kind == "rows":                 # whole rows
        x *= 1e-37
    elif kind == "one number":         # zeros and one smallest number
        x.zero_()
        x[:, H // 2] = SMALLEST
        x[::2, H // 2] = -SMALLEST
    elif kind == "weights":            # rows of 0.01 to 0.1, weights of 1e-36
        x *= torch.logspace(-2, -1, T, device="cuda")[:, None]
        w *= 1e-36
    elif kind == "block":              # one block of rows that are otherwise of size 0.05
        x *= 0.05
        x[:, -128:] *= 1e-35
    elif kind == "range":              # every size from 1e-38 to 1e-10
        x *= torch.logspace(-38, -10, T, device="cuda")[:, None]
    x, w = x.bfloat16(), w.bfloat16()
    return exact_products(x, w), w


@pytest.mark.parametrize("kind", ["rows", "one number", "weights", "block", "range"])
@pytest.mark.parametrize("dtype", [W.DTYPE_FP8, W.DTYPE_FP8_FP4])
@pytest.mark.parametrize("T,H", [(6, 256), (400, 384), (5, 8320), (300, 8320), (3, 20608), (4, 26752)])
def test_e4m3_of_small_values(kind, dtype, T, H):
    """rstd times the inverse of a block's scale passes fp32's range; the codes do not."""
    x, w = small_inputs(kind, T, H, I8.gen(T + H))
    assert (x != 0).any()
    out = torch.full((T, H), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((T, H // 128), -1.0, device="cuda")
    B.check(B.moe_add_rms_norm(params(T, H, dtype), x, None, w, EPS, None, out, scale))
    _, y = o.add_rms_norm(P.f64(x), None, P.f64(w), EPS)
    amax = np.abs(y.reshape(T, H // 128, 128)).max(axis=2)
    s, got_s = np.maximum(o.pow2_scale(amax), 2.0 ** -126), P.f64(scale)
    near = np.abs(amax / (448.0 * s) - 1) <= STEP
    near |= np.abs(amax / (224.0 * s) - 1) <= STEP
    assert ((got_s == s) | near & ((got_s == 2 * s) | (got_s == s / 2))).all()
    sb = np.repeat(got_s, 128, axis=1)
    v = o.decode_e4m3(out.view(torch.uint8).cpu().numpy()) * sb
    assert np.isfinite(v).all()
    assert (np.abs(v - y) <= np.maximum(np.abs(y) * 2.0 ** -4, sb * 2.0 ** -10) * (1 + 2.0 ** -10)).all()


def test_e4m3_layer_of_a_token_with_one_smallest_number():
    """The norm in front of the e4m3 layer: the token's output is a number."""
    wl = W.Workload("norm_layer", T=9, H=256, I=128, E=4, K=2, dtype=W.DTYPE_FP8)
    d = inputs.make_inputs(wl, seed=9, device="cuda")
    x = torch.randn((wl.T, wl.H), generator=I8.gen(1), device="cuda").bfloat16()
    x[4] = 0
    x[4, 17] = SMALLEST
    w = torch.ones(wl.H, device="cuda").bfloat16()
    p = B.params(wl)
    ws = torch.empty(B.moe_workspace_size_norm(p), dtype=torch.uint8, device="cuda")
    B.check(B.moe_clear_device_status(ws))
    out = torch.full_like(x, float("nan"))
    B.check(B.moe_norm_layer_forward(p, x, None, w, EPS, None, *I8.layer_args(d)[2:], out, None, None, None, ws, ws.numel()))
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and B.moe_get_device_status(ws) == 0


def int8_codes(x, w):
    """Codes of the norm, and those of 127 z w / max |z w| in fp64: z w and its multiples are exact, and a
    quotient that is not a tie lies more than 2^-30 from one, so rounding it decides as the exact one would."""
    T, H = x.shape
    out = torch.full((T, H), 77, dtype=torch.int8, device="cuda")
    scale = torch.empty(T, device="cuda")
    B.check(B.moe_add_rms_norm(params(T, H, W.DTYPE_INT8), x, None, w, EPS, None, out, scale))
    zw = P.f64(x) * P.f64(w)[None, :]
    return P.f64(out), np.round(127.0 * zw / np.abs(zw).max(axis=1, keepdims=True))


@pytest.mark.parametrize("T,H", [(3, 256), (200, 256), (3, 8320), (2, 20608), (2, 26752)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -112])
def test_int8_ties_go_to_even(T, H, size):
    """Every (2 k + 1) / 2 as the value of a code, for a largest product whose inverse rounds up or down."""
    odd = torch.arange(1, 254, 2, dtype=torch.float32)
    row = torch.cat([odd, -odd, torch.tensor([254.0, 0.0])]).repeat((H + 255) // 256)[:H]
    x = (row * size).cuda().bfloat16().repeat(T, 1)
    for q in range(1, 256, 2 if H == 256 else 46):
        got, want = int8_codes(x, torch.full((H,), float(q), device="cuda").bfloat16())
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("T,H", [(2000, 1024), (100, 7168), (300, 8320), (200, 20608), (100, 26752)])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -112])
def test_int8_codes_are_the_nearest(T, H, size):
    g = I8.gen(T)
    x = (torch.randn((T, H), generator=g, device="cuda") * size).bfloat16()
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    got, want = int8_codes(exact_products(x, w), w)
    np.testing.assert_array_equal(got, want)
