"""The shapes of the experts' GPU tests against the rule that chooses a product's
kernel (csrc/tile_choice.h, compiled here for the host): each kernel, with and
without a tail of K, has a shape that reaches it, and the rule holds its order."""
import ctypes
import os
import subprocess

import pytest

import segmented_rank_gemm_segment_amd as srg
import test_gpu_experts_gemm as gpu

WRAP = """
#include "tile_choice.h"
extern "C" int kernel(int c, int E, int K, int N, int f) { return lora::experts_kernel_of(c, E, K, N, f != 0); }
"""
FEW, MID, LARGE = range(3)


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    d = tmp_path_factory.mktemp("rule")
    (d / "wrap.cpp").write_text(WRAP)
    csrc = os.path.join(os.path.dirname(os.path.abspath(srg.__file__)), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + csrc,
                    str(d / "wrap.cpp"), "-o", str(d / "rule.so")], check=True)
    return ctypes.CDLL(str(d / "rule.so")).kernel


def test_every_kernel_has_a_shape(rule):
    reached = set()
    for n, k, E, _, d_in, d_out, _, _ in gpu.SHAPES:
        reached.add((rule(n * k, E, d_in, d_out, 1), True, d_in % 64 != 0))
        reached.add((rule(n * k, E, d_out, d_in, 0), False, d_out % 64 != 0))
    assert reached == {(k, f, t) for k in (FEW, MID, LARGE) for f in (True, False) for t in (True, False)}


def test_weights_have_both_tiles():
    tiles = {(-(-s[5] // 256)) * (-(-s[4] // 256)) * s[2] > 256 for s in gpu.SHAPES}
    assert tiles == {True, False}


@pytest.mark.parametrize("forward", [0, 1])
def test_order(rule, forward):
    """More rows never go to smaller tiles."""
    for E, K, N in ((1, 4096, 14336), (8, 4096, 4096), (64, 2048, 1536), (256, 1024, 512), (1024, 8, 256)):
        seen = [rule(c, E, K, N, forward) for c in (1, 4, 64, 1000, 16384, 1 << 20, 1 << 30)]
        assert seen == sorted(seen), (E, K, N, seen)
        assert seen[-1] == LARGE
    assert rule(8, 128, 2048, 1536, forward) == FEW
    assert rule(512, 128, 2048, 1536, forward) == MID
