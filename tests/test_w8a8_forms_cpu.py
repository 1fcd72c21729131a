"""The sizes that the GPU tests of the int8 products take, against the launch policy: every form of a kernel that it
chooses over a wide range of sizes is run by a test.  Without a GPU.

A form is what a call runs: the decode kernel with or without quantization; else tile, height, whether the contraction
is split, and into how many pieces the last round's tiles are cut.  The policy is taken from its source, since a plan
tells neither the pieces nor the gated backward's first launch."""

import ctypes
import math
import random
import subprocess

import numpy as np
import pytest

import test_gpu_w8a8 as old
import test_gpu_w8a8_forms as new
import w4a16_group_quantized_qmv_amd as w4
from w4a16_group_quantized_qmv_amd import build

CUS = 256
SOURCE = """
#include "w8a8_policy.h"
using namespace w4a16;
extern "C" void form(int op, int64_t E, int64_t T, int64_t R, int64_t N, int64_t K, int cus, int last, int* out) {
    const Product p = product_of(op, Sizes{E, T, R, N, K}, 0, cus, last != 0);
    const bool back = is_backward(op) && last;
    const W8TileShape& s = back ? kW8ColumnTiles[p.tile] : kW8Tiles[p.tile];
    const int v[] = {p.decode, p.quantize, p.tile, p.height, p.split, p.cut, !back && is_gated(op) ? s.bn / 2 : s.bn};
    for (int i = 0; i < 7; ++i) out[i] = v[i];
}
"""
# the launches of experts' calls: operator, whether it is the last launch of it
LAUNCHES = {"linear": (w4.W8A8_EXPERTS_LINEAR, 1), "backward": (w4.W8A8_EXPERTS_LINEAR_BACKWARD, 1), "gate_up": (w4.W8A8_EXPERTS_GATE_UP, 1),
            "gate_up backward, both products": (w4.W8A8_EXPERTS_GATE_UP_BACKWARD, 0),
            "gate_up backward, dx": (w4.W8A8_EXPERTS_GATE_UP_BACKWARD, 1)}


@pytest.fixture(scope="module")
def policy(tmp_path_factory):
    folder = tmp_path_factory.mktemp("policy")
    (folder / "form.hip").write_text(SOURCE)
    subprocess.run([build.hipcc(), f"--offload-arch={build.ARCH}", "--offload-host-only", "-std=c++17", "-O1", "-fPIC", "-shared", "-I",
                    build.INCLUDE, "-I", build.CSRC, str(folder / "form.hip"), "-o", str(folder / "form.so")], check=True)
    ctypes.CDLL(w4.lib_path(), mode=ctypes.RTLD_GLOBAL)             # (the tiles' shapes)
    f = ctypes.CDLL(str(folder / "form.so")).form
    f.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 5 + [ctypes.c_int] * 2 + [ctypes.c_void_p]
    out = (ctypes.c_int * 7)()

    def choose(op, E, T, R, N, K, last=1):
        f(op, E, T, R, N, K, CUS, last, out)
        return tuple(out)
    return choose


def dense(policy, op, M, N, K):
    decode, quantize, tile, height, split, cut, _ = policy(op, 1, M, M, N, K)
    return ("decode", quantize) if decode else (tile, height, "split" if split > 1 else "whole", cut)


def pieces(offsets, height, columns, most):
    """Into how many pieces find_expert_tile cuts what whole rounds over the compute units leave."""
    tiles = sum(-(-int(b - a) // height) for a, b in zip(offsets, offsets[1:]) if b > a) * columns
    rest = tiles % CUS
    if most < 2 or tiles <= CUS or rest == 0:
        return 1
    return 4 if most >= 4 and 4 * rest <= CUS else 2 if 2 * rest <= CUS else 1


def ragged(policy, op, last, E, T, R, N, K, offsets):
    _, _, tile, height, _, most, width = policy(op, E, T, R, N, K, last)
    outputs = K if op in (w4.W8A8_EXPERTS_LINEAR_BACKWARD, w4.W8A8_EXPERTS_GATE_UP_BACKWARD) and last else N
    return tile, pieces(offsets, height, -(-outputs // width), most)


def spread(rng, low, high):
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


@pytest.mark.parametrize("op", ["linear", "backward"])
def test_dense_sizes_reach_what_the_policy_chooses(policy, op):
    rng = random.Random(8)
    op, sizes = {"linear": (w4.W8A8_LINEAR, old.SHAPES + old.FORWARD + new.LINEAR),
                 "backward": (w4.W8A8_LINEAR_BACKWARD, [s for s in old.SHAPES if s[2] < 131056] + old.BACKWARD + new.BACKWARD)}[op]
    tested = {dense(policy, op, *s) for s in sizes}
    for M, N, K in sizes:                                    # the policy here is the library's
        p, form = w4.w8a8_plan(op, M, N, K, 0, CUS), dense(policy, op, M, N, K)
        if form[0] != "decode":
            assert form[:2] == (p["variant"] % 10, p["tile_m"]) and (form[3] > 1) == (p["variant"] >= 10)
    chosen = {}
    for _ in range(20000):
        M, N, K = spread(rng, 1, 10000), spread(rng, 1, 16384), 16 * spread(rng, 1, 1000)
        if M * N * K <= 4e11:
            chosen.setdefault(dense(policy, op, M, N, K), (M, N, K))
    assert len(chosen) >= 14
    assert not set(chosen) - tested, {f: s for f, s in chosen.items() if f not in tested}


@pytest.mark.parametrize("name", list(LAUNCHES))
def test_experts_sizes_reach_what_the_policy_chooses(policy, name):
    op, last = LAUNCHES[name]
    tested = {ragged(policy, op, last, E, T, R, N, K, old.ragged(np.random.default_rng(E * 1000 + R), E, R, kind))
              for E, T, R, N, K, kind in old.EXPERTS + new.EXPERTS}
    rng, chosen = random.Random(9), {}
    for _ in range(2000):
        E, T = spread(rng, 1, 1024), spread(rng, 1, 10000)
        top, N, K = rng.randint(1, min(8, E)), spread(rng, 1, 4096), 16 * spread(rng, 1, 256)
        if E * N * K <= 6e8 and T * top * N * K <= 4e11:
            offsets = old.ragged(np.random.default_rng(T), E, T * top, "random")
            chosen.setdefault(ragged(policy, op, last, E, T, T * top, N, K, offsets), (E, T, top, N, K))
    assert len(chosen) >= 4
    assert not set(chosen) - tested, {f: s for f, s in chosen.items() if f not in tested}


def test_a_whole_block_leaves_the_smallest_tiles(policy):
    """Each launch of a block of the tests runs some tile other than the one for the fewest rows."""
    for name, (op, last) in LAUNCHES.items():
        smallest = policy(op, 4, 3, 6, 32, 64, last)[2]
        blocks = [(E, T, T * top, *((K, F) if op in (w4.W8A8_EXPERTS_LINEAR, w4.W8A8_EXPERTS_LINEAR_BACKWARD) else (F, K)))
                  for E, T, F, K, top in new.BLOCKS]
        assert any(policy(op, *b, last)[2] != smallest for b in blocks), name
