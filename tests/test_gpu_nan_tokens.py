"""Tokens of NaN, which moe_add_rms_norm makes of non-finite rows, through routing and the layer."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_08_b200 import binding as B
from mixture_experts_ffn_08_b200 import inputs, workloads as W
from tests import int8_help as I8
from tests import parity as P

pytestmark = pytest.mark.gpu

GROUPS = dict(n_group=4, topk_group=2, group_topn=2)


@pytest.mark.parametrize("E,K,groups", [(4, 2, {}), (32, 8, {}), (40, 3, {}), (256, 8, {}), (300, 8, GROUPS), (256, 8, GROUPS),
                                        (8, 4, GROUPS), (1, 1, {})])
@pytest.mark.parametrize("score_fn", [W.SCORE_SOFTMAX, W.SCORE_SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
def test_topk_of_nan(E, K, groups, score_fn, biased):
    """Rows of NaN get K different ids below E; a sigmoid's single NaN is not chosen; other rows stay."""
    T = 9
    p = B.params(W.Workload("topk", T=T, H=128, I=128, E=E, K=K, score_fn=score_fn, **groups))
    z = torch.randn((T, E), generator=I8.gen(E), device="cuda")
    bias = torch.linspace(-1, 1, E, device="cuda") if biased else None

    def run(logits):
        ids = torch.full((T, K), -5, dtype=torch.int32, device="cuda")
        w = torch.zeros((T, K), device="cuda")
        B.check(B.moe_grouped_topk(p, logits, bias, ids, w))
        return ids.cpu().numpy(), w.cpu().numpy()

    ids, w = run(z)
    bad = z.clone()
    bad[2] = float("nan")
    bad[5] = float("inf")
    bad[7, E // 2] = float("nan")
    ids2, w2 = run(bad)
    for t in range(T):
        assert ((0 <= ids2[t]) & (ids2[t] < E)).all() and len(set(ids2[t])) == K
    rest = [0, 1, 3, 4, 6, 8]
    np.testing.assert_array_equal(ids2[rest], ids[rest])
    np.testing.assert_array_equal(w2[rest], w[rest])
    assert np.isnan(w2[2]).all()
    if score_fn == W.SCORE_SIGMOID and K < E and not groups:
        assert E // 2 not in ids2[7] and np.isfinite(w2[7]).all()


@pytest.mark.parametrize("dtype", [W.DTYPE_BF16, W.DTYPE_FP8, W.DTYPE_INT8])
@pytest.mark.parametrize("E,K,masked", [(4, 2, False), (32, 4, False), (40, 2, False), (64, 8, True)])
def test_layer_of_a_nan_token(dtype, E, K, masked):
    """Its output is NaN, the other tokens' bits are those without it, and no error is reported."""
    wl = W.Workload("norm_layer", T=70, H=256, I=128, E=E, K=K, dtype=dtype, masked_cap=128 if masked else 0)
    d = inputs.make_inputs(wl, seed=9, device="cuda")
    if dtype == W.DTYPE_BF16:
        a = P.device_inputs_ptrs(d, wl)
        tail = tuple(a[n] for n in ("w_r", "bias", "w_gate", "w_up", "w_down", "w_gate_scale", "w_up_scale", "w_down_scale",
                                    "ws_gate", "ws_up", "ws_down"))
    else:
        tail = I8.layer_args(d)[2:]
    x = torch.randn((wl.T, wl.H), generator=I8.gen(9), device="cuda").bfloat16()
    w = torch.ones(wl.H, device="cuda").bfloat16()
    p = B.params(wl)
    ws = torch.empty(B.moe_workspace_size_norm(p), dtype=torch.uint8, device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            x[17, 3] = float("nan")
        B.check(B.moe_clear_device_status(ws))
        out = torch.zeros_like(x)
        ids = torch.full((wl.T, K), -5, dtype=torch.int32, device="cuda")
        B.check(B.moe_norm_layer_forward(p, x, None, w, 1e-6, None, *tail, out, ids, None, None, ws, ws.numel()))
        torch.cuda.synchronize()
        assert B.moe_get_device_status(ws) == 0
        assert ((ids >= 0) & (ids < E)).all()
        outs.append(out)
    rest = torch.arange(wl.T, device="cuda") != 17
    assert torch.equal(outs[0][rest], outs[1][rest])
    assert torch.isnan(outs[1][17]).all()
