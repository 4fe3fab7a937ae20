"""Helpers of the int8 and norm tests: inputs, plain forms in 64 bits, derived bounds."""
from __future__ import annotations

import numpy as np
import torch

from mixture_experts_ffn_08_b200 import binding as B
from mixture_experts_ffn_08_b200 import workloads as W
from oracle import moe_oracle as o
from tests import parity as P

INT8_SMALL = W.Workload("int8_small", T=48, H=256, I=128, E=8, K=2, dtype=W.DTYPE_INT8)

# Half a step of the output type, relative to the value (normal numbers).
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(shape, g):
    """The whole int8 range, -128 too."""
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


def scales(n, g, mid=0.01):
    return mid * torch.exp2(torch.randn(n, generator=g, device="cuda"))


def expert_weights_fn(d):
    def get(e):
        return tuple(o.dequant_rows(d[n + "_q"][e].cpu().numpy(), d[n + "_s"][e].cpu().numpy())
                     for n in ("w_gate", "w_up", "w_down"))
    return get


def ffn_rows(x, wg, wu, wd):
    """(y, bound) in 64 bits of rows x through one int8 expert.

    The kernel's h differs from the exact one by at most DELTA of itself: three roundings of g
    and of u (2^-24 each), which SiLU amplifies by at most 1 + |g|, and the fast exponential (2 +
    1.16 |g| units in the last place) and division (2): below 2e-5 for |g| <= 40, where every
    test stays, and the row's scale with it.  So a code may be the neighbouring one only where
    h / s lies within 2 DELTA of itself from a border, and then y moves by one step times that
    column of W_down.  Beside that there are the scale's own DELTA and the rounding to bf16, half a
    step of what the kernel computed, |y| and what codes moved it by.
    The last term is the reference's own: the kernel's sum over q is an exact integer and may be
    exactly 0, where the I products q s w added in fp64 leave up to I 2^-53 of their sizes' sum."""
    delta = 2e-5
    g, u = x @ wg.T, x @ wu.T
    assert np.abs(g).max(initial=0.0) <= 40
    h = o.silu(g) * u
    s = o.int8_scale(np.abs(h).max(axis=1))[:, None]
    v = h / s
    near = np.abs(np.abs(v - np.trunc(v)) - 0.5) <= 2 * delta * np.abs(v) + 1e-6
    q = np.round(v) * s
    y = q @ wd.T
    own = (np.abs(q) @ np.abs(wd).T) * (q.shape[1] + 4) * 2.0 ** -53
    moved = s * (near @ np.abs(wd).T)
    return y, np.abs(y) * (2.0 ** -8 + 2 * delta) + moved * (1 + 2.0 ** -8) + own + 1e-37


def check_ffn(y, rows_of, x, weights, what=""):
    """rows_of: {expert: row numbers}; x: dequantised rows [rows, H]; y: what the kernel wrote."""
    worst = 0.0
    for e, rows in rows_of.items():
        if len(rows) == 0:
            continue
        ref, tol = ffn_rows(x[rows], *weights(e))
        err = np.abs(y[rows] - ref)
        assert np.isfinite(y[rows]).all(), f"{what}: expert {e}: not finite"
        assert (err <= tol).all(), f"{what}: expert {e}: {np.max(err / tol):.3g} times the bound"
        worst = max(worst, float(np.max(err / tol)))
    return worst


def run_layer(wl, d, ws=None):
    """One int8 moe_layer_forward: out, ids, w, counts and the workspace."""
    p = B.params(wl)
    ws = P.alloc_ws(p) if ws is None else ws
    r = dict(out=torch.empty((wl.T, wl.H), dtype=torch.bfloat16, device="cuda"),
             ids=torch.empty((wl.T, wl.K), dtype=torch.int32, device="cuda"),
             w=torch.empty((wl.T, wl.K), dtype=torch.float32, device="cuda"),
             counts=torch.empty((wl.E,), dtype=torch.int32, device="cuda"), ws=ws)
    B.check(B.moe_layer_forward(p, *layer_args(d), r["out"], r["ids"], r["w"], r["counts"], ws, ws.numel()))
    torch.cuda.synchronize()
    return r


def weight_args(d):
    """The weights and their scales of an int8 workload, in the entry points' order."""
    return (d["w_gate_q"], d["w_up_q"], d["w_down_q"], d["w_gate_s"], d["w_up_s"], d["w_down_s"])


def layer_args(d):
    return (d["x_q"], d["x_scale"], d["w_r"], d["bias"], *weight_args(d), None, None, None)
