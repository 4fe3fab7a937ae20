"""Which kernel and tile the int8 products take (csrc/i8_choice.h), asked without a GPU: the GPU tests'
shapes reach every variant on 148 SMs, and every choice can be launched on other numbers of SMs too."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

from tests import test_gpu_int8 as G
from tests import test_gpu_int8_rows as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DOT, SPLIT, PERSISTENT = range(3)
PAIR = 0

ASK = """
#include "i8_choice.h"
extern "C" void linear(int M, int N, int K, int sms, int* out) {
  const moe::I8Choice c = moe::i8_linear_choice(M, N, K, sms);
  const int v[] = {c.kernel, c.rows, c.channels, c.bn, c.ks};
  for (int i = 0; i < 5; ++i) out[i] = v[i];
}
extern "C" void experts(long long pairs, int E, int H, int I, int sms, int* out) {
  const moe::I8ExpertTiles t = moe::i8_expert_tiles(pairs, E, H, I, sms);
  out[0] = t.gate_up;
  out[1] = t.down;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    (d / "ask.cpp").write_text(ASK)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror",
                    "-I" + os.path.join(ROOT, "mixture_experts_ffn_08_b200", "csrc"), str(d / "ask.cpp"), "-o", str(d / "ask.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "ask.so"))

    def linear(M, N, K, sms=148):
        out = (ctypes.c_int * 5)()
        lib.linear(M, N, K, sms, out)
        return tuple(out)

    def experts(pairs, E, H, I, sms=148):
        out = (ctypes.c_int * 2)()
        lib.experts(ctypes.c_longlong(pairs), E, H, I, sms, out)
        return tuple(out)

    linear.experts = experts
    return linear


def shapes_of(test):
    """The (M, N, K) that a GPU test is parametrised over."""
    lists = {m.args[0]: m.args[1] for m in test.pytestmark if m.name == "parametrize"}
    if "M,N,K" in lists:
        return list(lists["M,N,K"])
    return [(M, N, K) for M, (N, K) in itertools.product(lists["M"], lists["N,K"])]


def test_the_tiles_list_reaches_every_split_variant(ask):
    got = {c[1:] for c in map(lambda s: ask(*s), G.TILES) if c[0] == SPLIT}
    assert got == {(rows, 0, bn, ks) for rows in (32, 64, 128) for bn in (32, 64, 128) for ks in (1, 2, 4)}


def test_the_gpu_tests_reach_every_other_variant(ask):
    shapes = G.TILES + R.TWO_CHANNELS
    for test in (G.test_linear_sizes, G.test_linear_large, G.test_linear_few_rows):
        shapes = shapes + shapes_of(test)
    got = {ask(*s) for s in shapes}
    assert {(c[1], c[2]) for c in got if c[0] == DOT} == {(1, 1), (2, 1), (2, 2), (3, 1), (4, 1)}
    assert {c[3] for c in got if c[0] == PERSISTENT} == {PAIR, 128, 256}


def test_the_gpu_tests_reach_every_expert_tile(ask):
    lists = {m.args[0]: m.args[1] for m in G.test_expert_ffn.pytestmark if m.name == "parametrize"}
    tiles = [ask.experts(T * K, E, H, I) for T, H, I, E, K, _, _ in lists["T,H,I,E,K,cap,empty"]]
    tiles += [ask.experts(70, 4, H, I) for H, I in ((7168, 2048), (4096, 14336))]  # test_expert_ffn_full_width
    assert {t[0] for t in tiles} == {t[1] for t in tiles} == {PAIR, 64, 128, 256}


@pytest.mark.parametrize("sms", [1, 80, 132, 148, 160, 192])
def test_choices_can_be_launched(ask, sms):
    """One round of split tiles fits the SMs and leaves no part without K; grids stay in their limits."""
    rng = random.Random(sms)
    for _ in range(20000):
        M, N, K = (int(2 ** rng.uniform(0, b)) for b in (15, 18, 12))
        K = 16 * K
        kernel, rows, channels, bn, ks = ask(M, N, K, sms)
        if kernel == DOT:
            assert rows == M <= 4 and channels in ((1, 2) if M == 2 else (1,))
        elif kernel == SPLIT:
            assert rows in (32, 64, 128) and bn in (32, 64, 128) and ks in (1, 2, 4)
            assert rows >= min(M, 128) and (M <= 64 or rows == 128)
            ctas = -(-M // 128) * -(-N // bn) * ks
            assert ctas <= sms and -(-N // bn) <= 65535
            assert ks == 1 or ks * 2 <= -(-K // 128) + 1
        else:
            assert bn in (PAIR, 128, 256) and (bn == PAIR) == (M > 128)
        E = rng.choice([1, 8, 128, 1024])
        assert set(ask.experts(M, E, 128 * (1 + N % 57), 128 * (1 + K % 113), sms)) <= {PAIR, 64, 128, 256}


def test_the_largest_sizes(ask):
    """The limits of moe_linear_int8: no overflow on the way to a choice."""
    assert ask(1, 2 ** 30, 131056) == (DOT, 1, 1, 0, 0)
    assert ask(2 ** 30, 1, 131056)[0] == PERSISTENT and ask(2 ** 30, 1, 131056)[3] == PAIR
    assert ask(4, 2 ** 30, 16)[0] in (DOT, PERSISTENT)
    assert ask(128, 2 ** 30, 131056) in {(PERSISTENT, 0, 0, bn, 1) for bn in (128, 256)}
