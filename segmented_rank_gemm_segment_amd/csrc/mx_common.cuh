// What the products with MXFP4 operands share.
#pragma once

#include "lds_dma.cuh"

namespace lora {
namespace {

// 32 x 32 x 64 product of MXFP4 fragments: lane l holds row l % 32 of each
// operand at codes [32 (l / 32), 32 (l / 32) + 32), one block, whose scale is
// byte SEL of its scale word.
template <int SEL>
__device__ __forceinline__ f32x16 mfma_mx(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SEL, (int)sa, SEL,
                                                         (int)sb);
}

// Tile t of the persistent kernels' order: groups of kPersistentGroup M-tiles, each
// sweeping N.
constexpr int kPersistentGroup = 8;
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int &mi, int &ni) {
  const int grp = t / (kPersistentGroup * tiles_n), first = grp * kPersistentGroup;
  const int cnt = min(kPersistentGroup, tiles_m - first);
  const int in = t - grp * kPersistentGroup * tiles_n;
  mi = first + in % cnt;
  ni = in / cnt;
}

}  // namespace
}  // namespace lora
