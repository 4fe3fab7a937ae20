"""The int8 products' epilogues at every number of rows in a warp's last 32, where some lanes store and
some do not between the column steps.  K and the codes are small enough that fp32 holds every sum."""
import numpy as np
import pytest
import torch

from mixture_experts_ffn_08_b200 import binding as B
from mixture_experts_ffn_08_b200 import inputs
from tests import int8_help as I8
from tests import parity as P
from tests import test_gpu_int8 as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,ldo", [(128, 128), (136, 136), (130, 131), (20000, 20000), (20001, 20003)])
def test_linear_at_every_row_count(N, ldo):
    """One round of tiles (stored from TMEM, or by way of shared memory), and persistent one-SM tiles."""
    K = 64
    g = I8.gen(N)
    a, w = I8.codes((128, K), g), I8.codes((N, K), g)
    one_a, one_w = torch.ones(128, device="cuda"), torch.ones(N, device="cuda")
    ref = (a.double() @ w.double().T).float()
    for M in range(5, 129):
        out = torch.full((M, ldo), 55.0, device="cuda")
        B.check(B.moe_linear_int8(M, N, K, a, K, one_a, w, K, one_w, None, out, ldo, B.MOE_OUT_FP32, None))
        assert torch.equal(out[:, :N], ref[:M]) and (out[:, N:] == 55.0).all(), M


def test_linear_pair_tiles_at_every_row_count():
    N, K = 9600, 64
    g = I8.gen(1)
    a, w = I8.codes((320, K), g), I8.codes((N, K), g)
    one_a, one_w = torch.ones(320, device="cuda"), torch.ones(N, device="cuda")
    ref = (a.double() @ w.double().T).float()
    for M in range(256, 321):
        out = torch.empty((M, N), device="cuda")
        B.check(B.moe_linear_int8(M, N, K, a, K, one_a, w, K, one_w, None, out, N, B.MOE_OUT_FP32, None))
        assert torch.equal(out, ref[:M]), M


# Two rows and so many channels that a warp takes two of them; the last warp has one where N is odd.
TWO_CHANNELS = [(2, 7104, 16), (2, 7105, 528), (2, 7333, 1040), (2, 9999, 8192), (2, 20001, 4112)]


@pytest.mark.parametrize("M,N,K", TWO_CHANNELS)
def test_linear_of_two_rows_and_two_channels(M, N, K):
    for i, dtype in enumerate(G.KIND):
        args, ref, tol = G.linear_case(M, N, K, dtype, bias=i == 1, pad=(16, 32, (0, 1, 8)[i]), seed=N + i)
        G.linear(*args)
        G.check_linear(args, ref, tol)


@pytest.mark.parametrize("more", [0, 256])
@pytest.mark.parametrize("cap", [0, 384])
def test_experts_at_every_row_count(more, cap):
    """Expert e has more + e rows, in one-SM tiles (few rows) and in pair tiles."""
    E = 40
    wl = I8.INT8_SMALL.with_(T=E * more + E * (E - 1) // 2, H=2560 if more else 256, I=1280 if more else 128, E=E, K=1,
                             masked_cap=cap)
    d = inputs.make_inputs(wl, seed=3, device="cuda")
    ids = torch.repeat_interleave(torch.arange(E), more + torch.arange(E)).int().cuda()
    p = B.params(wl)
    ws = P.alloc_ws(p)
    rows = B.moe_max_padded_rows(p)
    counts, offs, rop, por = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E, E + 1, wl.T, rows))
    xp, xps = torch.zeros((rows, wl.H), dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda")
    B.check(B.moe_permute(p, ids, d["x_q"], d["x_scale"], counts, offs, rop, por, xp, xps, ws, ws.numel()))
    y = torch.full((rows, wl.H), 33.0, dtype=torch.bfloat16, device="cuda")
    B.check(B.moe_expert_ffn(p, xp, xps, offs, counts, *I8.weight_args(d), y, ws, ws.numel()))
    torch.cuda.synchronize()
    assert B.moe_get_device_status(ws) == 0
    assert (y[rop.long()] != 33.0).any(dim=1).all()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[rop.long()] = False
    assert (y[rest] == 33.0).all()
    first, n = offs.tolist(), counts.tolist()
    assert n == [more + e for e in range(E)]
    for e in (1, 7, 15, 16, 17, 31, 32, 33, 39):  # (in 64 bits, the others take the same paths)
        r = np.arange(first[e], first[e] + n[e])
        x = P.f64(xp[r[0]:r[-1] + 1]) * P.f64(xps[r[0]:r[-1] + 1])[:, None]
        ref, tol = I8.ffn_rows(x, *I8.expert_weights_fn(d)(e))
        assert (np.abs(P.f64(y[r[0]:r[-1] + 1]) - ref) <= tol).all(), e
