"""The shapes of the MXFP4 GPU tests against the rules that choose a kernel
(csrc/tile_choice.h, compiled here for the host): every kernel that a call can
reach has a shape, so a changed border cannot leave one untested."""
import ctypes
import os
import subprocess

import pytest

import segmented_rank_gemm_segment_amd as srg
import test_gpu_mxfp4_kernels as kernels

WRAP = """
#include "tile_choice.h"
extern "C" int weight(int M, int N, int lora) { return lora::mx_weight_kernel_of(M, N, lora != 0); }
extern "C" int both(int M, int N) { return lora::mx_both_kernel_of(M, N); }
extern "C" int experts(int n, int E, int K, int N) { return lora::mx_experts_kernel_of(n, E, K, N); }
extern "C" int tiles8(int N) { return lora::mx_stream8_tiles(N); }
extern "C" int wide(int K, long ldw, long ldx) { return lora::mx_wide_scales(K, ldw, ldx); }
"""
STREAM8, STREAM16, T32, T64, T128, T192, T256, PERSISTENT = range(8)
DIMS = [8, 136, 1024, 2048, 2056, 4096, 4104, 6144, 8192, 8200, 14336, 28672]
ROWS = [1, 8, 9, 16, 17, 32, 33, 64, 100, 256, 300, 512, 700, 1024, 1500, 2048, 2304, 4096, 8192, 16384, 65536]


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    (d / "wrap.cpp").write_text(WRAP)
    csrc = os.path.join(os.path.dirname(os.path.abspath(srg.__file__)), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + csrc,
                    str(d / "wrap.cpp"), "-o", str(d / "rules.so")], check=True)
    L = ctypes.CDLL(str(d / "rules.so"))
    L.wide.argtypes = [ctypes.c_int, ctypes.c_long, ctypes.c_long]
    return L


def weight_key(L, n, d_in, d_out, lora):
    k = L.weight(n, d_out, int(lora))
    if k == STREAM8:
        return k, L.tiles8(d_out)
    if k == PERSISTENT:                      # the scale rows' width, and a tail of K
        return k, bool(L.wide(d_in, (d_in // 32 + 15) // 16 * 16, 0)), d_in % 256 != 0
    return (k,)


@pytest.mark.parametrize("lora", [False, True])
def test_every_weight_kernel_has_a_shape(rules, lora):
    reached = {weight_key(rules, n, d_in, d_out, lora)
               for n in ROWS for d_out in DIMS for d_in in (512, 768, 608)}
    shapes = [s[:3] for s in kernels.LORA_SHAPES] if lora else kernels.WEIGHT_SHAPES
    tested = {weight_key(rules, *s, lora) for s in shapes}
    assert reached <= tested, sorted(reached - tested)
    assert (T192 in {k[0] for k in reached}) == lora and (PERSISTENT in {k[0] for k in reached}) != lora


def test_every_kernel_of_two_mxfp4_operands_has_a_shape(rules):
    def key(n, d_in, d_out, pad):
        k = rules.both(n, d_out)
        ld = (d_in // 32 + 15) // 16 * 16 + pad
        return (k, bool(rules.wide(d_in, ld, ld))) if k == PERSISTENT else (k,)
    reached = {key(n, d_in, d_out, 0) for n in ROWS for d_out in DIMS for d_in in (512, 608)}
    tested = {key(*s, pad) for s in kernels.BOTH_SHAPES for pad in (0, 4)}
    assert reached <= tested and len(reached) == 5, sorted(reached - tested)


def test_every_experts_kernel_has_a_shape(rules):
    def key(n, E, d_in, d_out):
        k = rules.experts(n, E, d_in, d_out)
        if k == PERSISTENT:
            return k, bool(rules.wide(d_in, (d_in // 32 + 15) // 16 * 16, 0)), d_in % 256 != 0
        return (k,)
    tested = {key(n * k, E, d_in, d_out) for n, k, E, d_in, d_out in kernels.EXPERT_SHAPES}
    reached = {key(n * k, E, d_in, d_out) for n in ROWS for k in (1, 8) for E in (1, 8, 64, 1000)
               for d_in in (512, 2048, 4096, 768, 608) for d_out in (136, 2048, 8200)}
    assert reached <= tested and len(reached) == 6, sorted(reached - tested)


def test_base_rows_share_a_k_order(rules):
    """With adapters or without, a batch's kernel adds K up in one order: streamed,
    the four groups of the 32- and 64-row tiles, or that of all others."""
    order = {STREAM8: 8, STREAM16: 16, T32: 4, T64: 4, T128: 1, T192: 1, T256: 1, PERSISTENT: 1}
    for n in range(1, 3000, 7):
        for d_out in DIMS:
            assert order[rules.weight(n, d_out, 0)] == order[rules.weight(n, d_out, 1)], (n, d_out)


ORDER = """
#include "tile_order.h"
using namespace lora;
template <bool SPARE>
static int walk(int grid, int tm, int tn, int heavy, int *count) {
  for (int b = 0; b < grid; ++b) {
    int m = -1, n = -1;
    if (!tile_order<SPARE>(b, tm, tn, heavy, m, n)) continue;
    if (m < 0 || m >= tm || n < 0 || n >= tn) return -1;
    ++count[m * tn + n];
  }
  return 0;
}
extern "C" int dense(int tm, int tn, int heavy, int *count) { return walk<false>(tile_grid(tm, tn), tm, tn, heavy, count); }
extern "C" int layer(int tm, int tn, int rows, int *count) {
  const int g = tile_grid(tm, tn);
  return walk<true>(g > rows ? g : rows, tm, tn, -1, count);
}
extern "C" int experts(int bound, int tm, int tn, int *count) { return walk<true>(expert_grid(bound, tn), tm, tn, -1, count); }
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    d = tmp_path_factory.mktemp("order")
    (d / "wrap.cpp").write_text(ORDER)
    csrc = os.path.join(os.path.dirname(os.path.abspath(srg.__file__)), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + csrc,
                    str(d / "wrap.cpp"), "-o", str(d / "order.so")], check=True)
    return ctypes.CDLL(str(d / "order.so"))


def once(f, tm, tn, *args):
    count = (ctypes.c_int * (tm * tn))()
    assert f(*args, count) == 0
    assert all(c == 1 for c in count), (tm, tn, args, max(count), min(count))


@pytest.mark.parametrize("tn", [1, 4, 7, 8, 9, 24, 32, 129])
def test_every_tile_is_taken_once(order, tn):
    """By the grid of a dense batch; by that of the one-launch layer, which has a
    workgroup a row; and by the experts', which is sized by a bound on the M-tiles."""
    for tm in (1, 2, 8, 31, 32, 33, 45, 130):
        for heavy in (-1, 0, tm - 1):
            once(order.dense, tm, tn, tm, tn, heavy)
        if tm <= 8:
            once(order.layer, tm, tn, tm, tn, 64 * tm)
        for bound in (tm, tm + 1, tm + 20, 4 * tm + 100):
            once(order.experts, tm, tn, bound, tm, tn)
