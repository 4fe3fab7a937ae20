"""The int8 product with scales far from 1, and the same row in products of every height.

The bound in fp32: the sum's conversion, its product with the row's scale and the multiply-add with
the channel's round by 2^-24 each; a result below 2^-126 by half of 2^-149 besides."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_08_b200 import binding as B
from tests import int8_help as I8
from tests import parity as P

pytestmark = pytest.mark.gpu

KIND = {torch.bfloat16: B.MOE_OUT_BF16, torch.float16: B.MOE_OUT_FP16, torch.float32: B.MOE_OUT_FP32}


def product(a, sa, w, sw, bias, dtype):
    M, K = a.shape
    N = w.shape[0]
    out = torch.full((M, N), 55.0, dtype=dtype, device="cuda")
    B.check(B.moe_linear_int8(M, N, K, a, K, sa, w, K, sw, bias, out, N, KIND[dtype], None))
    return out


@pytest.mark.parametrize("sa,sw", [(2.0 ** -126, 5e-4), (1e-23, 1e-23), (1e-30, 1e-20), (2.0 ** -120, 1e30), (1e20, 1e-35),
                                   (1e25, 1e25)])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 8, 200, 700])
def test_scales_whose_product_leaves_fp32(M, sa, sw):
    """The smallest scales that the norm writes, and large ones with a sum of zero."""
    N, K = 2600, 512
    g = I8.gen(M)
    a, w = I8.codes((M, K), g), I8.codes((N, K), g)
    if sa > 1 and sw > 1:
        a.zero_()
    ta = torch.full((M,), sa, device="cuda")
    tw = sw * (1 + torch.rand(N, generator=g, device="cuda"))
    out = P.f64(product(a, ta, w, tw, None, torch.float32))
    ref = (P.f64(a) @ P.f64(w).T) * P.f64(ta)[:, None] * P.f64(tw)[None, :]
    assert (np.abs(out - ref) <= np.abs(ref) * 2.0 ** -22 + 2.0 ** -149).all()


@pytest.mark.parametrize("N,K", [(700, 2048), (9600, 256), (7100, 512)])
@pytest.mark.parametrize("bias", [False, True])
def test_a_row_does_not_depend_on_the_others(N, K, bias):
    """Dot products, split tiles and persistent tiles round alike: one row's bits at every M."""
    g = I8.gen(N)
    a, w = I8.codes((800, K), g), I8.codes((N, K), g)
    sa, sw = I8.scales(800, g), I8.scales(N, g)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    for dtype in KIND:
        want = product(a, sa, w, sw, b, dtype)
        for M in (1, 2, 3, 4, 5, 30, 60, 128, 129, 300):
            assert torch.equal(product(a[:M], sa[:M], w, sw, b, dtype), want[:M]), (M, dtype)
