"""The int8 and norm entry points without a GPU: sizes, refusals, and pins of the oracle's pieces."""
import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_ffn_08_b200 import binding as B
from mixture_experts_ffn_08_b200 import inputs, workloads as W
from oracle import moe_oracle as o

INT8 = W.Workload("int8", T=8, H=256, I=128, E=4, K=2, dtype=W.DTYPE_INT8)
OK, INVALID, UNSUPPORTED = 0, 1, 2
ADDR = 4096  # never read: every call below is refused, or is empty


@pytest.fixture(scope="module")
def lib():
    return B.lib(require_gpu=False)


def test_workspaces(lib):
    p = B.params(INT8)
    a, n, h = B.moe_workspace_size(p), B.moe_workspace_size_norm(p), B.moe_workspace_size_host(p)
    rows = B.moe_max_padded_rows(p)
    assert a >= rows * (5 * INT8.I + INT8.H) and a + 8 * 256 <= n <= h
    for wl in (W.TINY, W.TINY.with_(dtype=W.DTYPE_FP8)):
        q = B.params(wl)
        assert B.moe_workspace_size(q) < B.moe_workspace_size_norm(q) < B.moe_workspace_size_host(q)
    assert B.moe_workspace_size_norm(B.params(INT8.with_(H=100))) == 0


def test_launch_counts(lib):
    """x's codes for the router, h's codes; no schedule kernel in the masked layout."""
    for wl in (INT8, INT8.with_(masked_cap=128)):
        assert B.moe_layer_launch_count(B.params(wl)) == 9


@pytest.mark.parametrize("change", [dict(I_shared=128), dict(block_m=256), dict(fused_combine=True), dict(H=131072),
                                    dict(I=131072), dict(H=200), dict(dtype=4)])
def test_params_refused(lib, change):
    p = B.params(INT8.with_(**change))
    assert B.moe_workspace_size(p) == 0 and B.moe_workspace_size_norm(p) == 0


def linear(lib, M=4, N=8, K=32, a=ADDR, lda=32, sa=ADDR, w=ADDR, ldw=32, sw=ADDR, bias=None, out=ADDR, ldo=8, kind=0):
    return lib.moe_linear_int8(M, N, K, a, lda, sa, w, ldw, sw, bias, out, ldo, kind, None, None)


@pytest.mark.parametrize("bad,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(K=-16), INVALID), (dict(lda=16), INVALID),
    (dict(ldw=16), INVALID), (dict(ldo=7), INVALID), (dict(kind=3), INVALID), (dict(kind=-1), INVALID),
    (dict(K=24), UNSUPPORTED), (dict(K=131072, lda=131072, ldw=131072), UNSUPPORTED), (dict(lda=40), UNSUPPORTED),
    (dict(ldw=40), UNSUPPORTED), (dict(lda=1 << 40), UNSUPPORTED), (dict(M=2**31 - 1, N=2**31 - 1, ldo=2**31), UNSUPPORTED),
    (dict(M=2**30 + 1), UNSUPPORTED), (dict(N=2**30 + 1, ldo=2**31), UNSUPPORTED), (dict(M=2**30, N=2**30, ldo=2**30), UNSUPPORTED),
    (dict(a=None), INVALID), (dict(sa=None), INVALID), (dict(w=None), INVALID), (dict(sw=None), INVALID),
    (dict(out=None), INVALID), (dict(a=ADDR + 8), INVALID), (dict(w=ADDR + 8), INVALID), (dict(out=ADDR + 1), INVALID),
    (dict(out=ADDR + 2, kind=2), INVALID), (dict(sa=ADDR + 2), INVALID), (dict(sw=ADDR + 1), INVALID),
    (dict(bias=ADDR + 2), INVALID)])
def test_linear_refuses(lib, bad, code):
    assert linear(lib, **bad) == code


def test_linear_of_nothing(lib):
    assert linear(lib, M=0, a=None, sa=None, w=None, sw=None, out=None) == OK


def norm(lib, p, x=ADDR, res=ADDR, w=ADDR, eps=1e-6, res_out=ADDR, out=ADDR, scale=ADDR):
    return lib.moe_add_rms_norm(ctypes.byref(p), x, res, w, eps, res_out, out, scale, None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(w=None), dict(out=None), dict(scale=None), dict(res=None), dict(eps=0.0),
                                 dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-40),
                                 dict(x=ADDR + 8), dict(res=ADDR + 2), dict(w=ADDR + 8), dict(res_out=ADDR + 8),
                                 dict(out=ADDR + 8), dict(scale=ADDR + 2)])
def test_norm_refuses(lib, bad):
    assert norm(lib, B.params(INT8), **bad) == INVALID


def test_norm_checks_its_params_first(lib):
    assert norm(lib, B.params(INT8.with_(H=100))) == UNSUPPORTED
    assert norm(lib, B.params(INT8.with_(dtype=9))) == INVALID
    assert norm(lib, B.params(INT8.with_(T=0)), x=None, res=None, w=None, res_out=None, out=None, scale=None) == OK
    assert norm(lib, B.params(INT8.with_(T=0)), eps=0.0) == INVALID


def test_stages_refuse_missing_scales(lib):
    p = B.params(INT8)
    n = B.moe_workspace_size_norm(p)
    pp = ctypes.byref(p)
    assert lib.moe_route(pp, ADDR, None, ADDR, None, ADDR, ADDR, ADDR, n, None) == INVALID
    assert lib.moe_permute(pp, ADDR, ADDR, None, *[ADDR] * 6, ADDR, n, None) == INVALID
    assert lib.moe_permute(pp, ADDR, ADDR, ADDR, *[ADDR] * 5, None, ADDR, n, None) == INVALID
    ffn = [ADDR] * 11
    for i in (1, 7, 8, 9):  # x_perm_scale and the three weight scales
        bad = list(ffn)
        bad[i] = None
        assert lib.moe_expert_ffn(pp, *bad, ADDR, n, None) == INVALID
    assert lib.moe_shared_expert_ffn(pp, *[ADDR] * 5, ADDR, n, None) == UNSUPPORTED
    layer = [ADDR, None, ADDR, None, ADDR, ADDR, ADDR, ADDR, ADDR, ADDR, None, None, None, ADDR, None, None, None]
    assert lib.moe_layer_forward(pp, *layer, ADDR, n, None) == INVALID
    masked = B.params(INT8.with_(masked_cap=128))
    bad = list(ffn)
    bad[3] = None  # counts
    assert lib.moe_expert_ffn(ctypes.byref(masked), *bad, ADDR, B.moe_workspace_size(masked), None) == INVALID


@pytest.mark.parametrize("at", [0, 2, 5, 7, 8, 9, 10, 11, 12, 16])
def test_norm_layer_refuses_before_any_launch(lib, at):
    """A missing pointer of the layer is found before the norm runs."""
    p = B.params(INT8)
    n = B.moe_workspace_size_norm(p)
    args = [ADDR, ADDR, ADDR, 1e-6, ADDR, ADDR, None, ADDR, ADDR, ADDR, ADDR, ADDR, ADDR, None, None, None, ADDR, None, None, None]
    args[at] = None
    assert lib.moe_norm_layer_forward(ctypes.byref(p), *args, ADDR, n, None) == INVALID


def test_norm_layer_checks_its_workspace(lib):
    p = B.params(INT8)
    args = [ADDR, ADDR, ADDR, 1e-6, ADDR, ADDR, None, *[ADDR] * 6, None, None, None, ADDR, None, None, None]
    assert lib.moe_norm_layer_forward(ctypes.byref(p), *args, ADDR, B.moe_workspace_size_norm(p) - 1, None) == INVALID
    assert lib.moe_norm_layer_forward(ctypes.byref(p), *args, ADDR + 8, B.moe_workspace_size_norm(p), None) == INVALID
    e = B.params(INT8.with_(T=0))
    none = [None, None, None, 1e-6] + [None] * 16
    assert lib.moe_norm_layer_forward(ctypes.byref(e), *none, ADDR, B.moe_workspace_size_norm(e), None) == OK


def test_empty_batch(lib):
    p = B.params(INT8.with_(T=0))
    n, pp = B.moe_workspace_size(p), ctypes.byref(p)
    assert lib.moe_route(pp, None, None, None, None, None, None, ADDR, n, None) == OK
    assert lib.moe_expert_ffn(pp, *([None] * 11), ADDR, n, None) == OK
    assert lib.moe_combine(pp, None, None, None, None, None, None) == OK
    assert lib.moe_layer_forward(pp, *([None] * 17), ADDR, n, None) == OK


# -------------------------------------------------------------------------------- oracle pins
def test_oracle_int8_rows():
    """By hand: 254 / 127 = 2, halves to the even code, a zero row has scale 1."""
    h = np.array([[254.0, -3.0, 5.0, 1.0, -254.0], [0.0] * 5, [127.0, 0.5, 1.5, -2.5, 126.4]])
    want = np.array([[254.0, -4.0, 4.0, 0.0, -254.0], [0.0] * 5, [127.0, 0.0, 2.0, -2.0, 126.0]])
    np.testing.assert_array_equal(o.quantize_rows_int8(h), want)
    np.testing.assert_array_equal(o.store_activation(h, "int8"), want)
    assert o.activation_format(W.DTYPE_INT8) == "int8"


def test_oracle_norm():
    """By hand: rows (3, 4) and (0, 0) with eps 0.5 and 1; and torch's own norm in 64 bits."""
    z, y = o.add_rms_norm([[3.0, 4.0], [0.0, 0.0]], None, [2.0, 1.0], 0.5)
    np.testing.assert_allclose(y, [[6.0 / np.sqrt(13.0), 4.0 / np.sqrt(13.0)], [0.0, 0.0]], rtol=1e-15)
    g = torch.Generator().manual_seed(0)
    x, r = (torch.randn((5, 96), generator=g).bfloat16() for _ in range(2))
    w = torch.randn(96, generator=g).bfloat16()
    z, y = o.add_rms_norm(x.double().numpy(), r.double().numpy(), w.double().numpy(), 1e-5)
    s = (x.float() + r.float()).bfloat16()
    np.testing.assert_array_equal(z, s.double().numpy())
    ref = torch.nn.functional.rms_norm(s.double(), (96,), w.double(), 1e-5)
    np.testing.assert_allclose(y, ref.numpy(), rtol=1e-13)


def test_generator_int8():
    d = inputs.make_inputs(INT8, seed=1)
    assert d["x_q"].dtype == torch.int8 and d["x_q"].abs().amax(dim=1).eq(127).all()
    assert d["w_down_q"].shape == (4, 256, 128) and d["w_down_s"].shape == (4, 256)
    v = torch.tensor([[254.0, -3.0, 5.0], [0.0, 0.0, 0.0]])
    q, s = inputs.quantize_rows_int8(v)
    assert q.tolist() == [[127, -2, 2], [0, 0, 0]] and s.tolist() == [2.0, 1.0]
