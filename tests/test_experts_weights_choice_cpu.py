"""The shapes of the GPU tests of the weights' gradients against the rule that chooses their
tiles (csrc/tile_choice.h, compiled here for the host): every instance of the kernel is
reached with segments of one stage of 64 rows and of several, with tiles that are full and
some that are not, and with tiles that follow each other in a workgroup."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import segmented_rank_gemm_segment_amd as srg
import test_gpu_experts_gemm as products
import test_gpu_experts_weights as weights
from test_gpu_experts import make_ids

WRAP = """
#include "tile_choice.h"
extern "C" int large(int M, int N, int E) { return lora::experts_weights_large(M, N, E); }
"""


@pytest.fixture(scope="module")
def large(tmp_path_factory):
    d = tmp_path_factory.mktemp("rule")
    (d / "wrap.cpp").write_text(WRAP)
    csrc = os.path.join(os.path.dirname(os.path.abspath(srg.__file__)), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + csrc,
                    str(d / "wrap.cpp"), "-o", str(d / "rule.so")], check=True)
    return ctypes.CDLL(str(d / "rule.so")).large


def test_every_instance_has_its_shapes(large):
    short, long = set(), set()
    for shapes, seed in ((products.SHAPES, 4), (weights.SHAPES, 31)):
        for n, k, E, kind, d_in, d_out, gathered, _ in shapes:
            ids = make_ids(seed, n, k, E, kind)
            rows = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
            big = bool(large(d_out, d_in, E))
            tile, workgroups = (256, 256) if big else (128, 512)
            tiles = E * -(-d_out // tile) * -(-d_in // tile)
            partial = d_out % tile != 0 and d_in % tile != 0 and min(d_out, d_in) > tile
            if partial and np.any((rows > 0) & (rows <= 64)):
                short.add((big, gathered))
            if partial and np.any((rows > 192) & (rows % 64 != 0)) and tiles > workgroups:
                long.add((big, gathered))
    every = {(b, g) for b in (True, False) for g in (True, False)}
    assert short == every and long == every, (short, long)


def test_border(large):
    """256 tiles and less leave the larger ones to a part of the CUs."""
    assert not large(1024, 1024, 16) and large(1024, 1032, 16) and large(256, 256, 257)
    assert not large(8, 8, 256) and large(1 << 22, 1 << 22, 1024)
