// Launches of the products with MXFP4 operands (the MFMA tiles of
// gemm_tile.cuh): an MXFP4 weight under bf16 activations, with or without the
// LoRA term, both operands MXFP4, and the experts' product.
#include "mx_mid.cuh"
#include "mx_stream.cuh"
#include "mx_weight.cuh"

namespace lora {
namespace {

template <int BM, int BN, int WM, int WN, int BK, int STAGES, int KG>
hipError_t launch_codes(const GemmArgs &g, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_bf16_kernel<BM, BN, WM, WN, BK, STAGES, KG, 0, false, kMxXW>),
                     dim3(tile_grid((g.M + BM - 1) / BM, (g.N + BN - 1) / BN)),
                     dim3(WM * WN * KG * kWave), 0, stream, g);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int BK, int STAGES, int KG>
hipError_t launch_experts(const GemmArgs &g, int tiles_m, hipStream_t stream) {
  const int tn = (g.N + BN - 1) / BN;
  // the workgroups find the number of tiles themselves: room for any up to tiles_m
  const int split = tiles_m < kHeavyMaxTilesM ? tiles_m : kHeavyMaxTilesM;
  int grid = (tiles_m * tn + 7) / 8 * 8;
  if (8 * ((tn + 7) / 8) * split > grid) grid = 8 * ((tn + 7) / 8) * split;
  hipLaunchKernelGGL(
      (gemm_bf16_kernel<BM, BN, WM, WN, BK, STAGES, KG, 0, false, kMxW, false, true>), dim3(grid),
      dim3(WM * WN * KG * kWave), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_mx(const void *X, int64_t ldx, const void *W, int64_t ldw,
                          const MxScales &mx, void *Y, int64_t ldy, int M, int K, int N,
                          const float *H, const SegView *seg, const PoolView *pool,
                          hipStream_t stream) {
  const bool lora = seg != nullptr;
  if (mx.x && M > LORA_GEMM_SMALL_M && !mid_tiles(M, N))
    return launch_mx_product(X, ldx, W, ldw, mx, Y, ldy, M, K, N, stream);
  if (mx.x && M <= LORA_GEMM_SMALL_M) {
    GemmArgs g = gemm_args(X, ldx, W, ldw * 2, Y, ldy, M, K, N, nullptr, nullptr, nullptr);
    g.mx = mx;
    return launch_mx_mid<true>(g, false, stream);
  }
  if (mx.x) {
    // both operands in units of four codes
    GemmArgs g = gemm_args(X, ldx / 2, W, ldw / 2, Y, ldy, M, K / 4, N, nullptr, nullptr, nullptr);
    g.mx = mx;
    return launch_rows_split(g, false, [&](const GemmArgs &a) {
      if (a.M <= LORA_GEMM_SMALL_M) return launch_codes<LORA_GEMM_SMALL>(a, stream);
      if (mid_tiles(a.M, N)) return launch_codes<LORA_GEMM_MID>(a, stream);
      if (large192_tiles(a.M, N)) return launch_codes<LORA_GEMM_LARGE192>(a, stream);
      return launch_codes<LORA_GEMM_LARGE>(a, stream);
    });
  }
  GemmArgs g = gemm_args(X, ldx, W, ldw * 2, Y, ldy, M, K, N, H, seg, pool);
  g.mx = mx;
  if (M <= kStreamRows) return launch_mx_stream(g, lora, stream);
  if (M <= LORA_GEMM_SMALL_M) return launch_mx_mid<false>(g, lora, stream);
  if (mid_tiles(M, N)) return launch_tile<LORA_GEMM_MID, kMxW>(g, lora, stream);
  if (!lora) return launch_mx_weight<false>(g, stream);
  // With adapters the shared tiles, whose LoRA term goes through LDS: read from
  // memory into each wave's fragments instead it cost 11 us a tile, and the two
  // were level (16943 x 4096 x 14336, 8 slots: 1.69 ms).  Both add up K in the same
  // order, so base-only rows keep the base product's bits.
  if (large192_tiles(M, N)) return launch_tile<LORA_GEMM_LARGE192, kMxW>(g, lora, stream);
  return launch_tile<LORA_GEMM_LARGE, kMxW>(g, lora, stream);
}

hipError_t launch_experts_gemm_mx(const void *X, int64_t ldx, const ExpertView &ex, const void *W,
                                  int64_t ldw, const MxScales &mx, void *Y, int64_t ldy, int K,
                                  int N, hipStream_t stream) {
  GemmArgs g = gemm_args(X, ldx, W, ldw * 2, Y, ldy, 0, K, N, nullptr, nullptr, nullptr);
  g.mx = mx;
  g.ex = ex;
  // at most one part-filled M-tile an expert, and no more tiles than rows
  auto tiles = [&](int bm) {
    const int64_t t = (int64_t)ex.n_choices / bm + ex.n_experts;
    return (int)(t < ex.n_choices ? t : ex.n_choices);
  };
  if (ex.n_choices / ex.n_experts <= 32) return launch_experts_stream(g, tiles(16), stream);
  if (ex.n_choices / ex.n_experts >= 512) return launch_mx_weight<true>(g, stream);
  return launch_experts<LORA_GEMM_MID>(g, tiles(128), stream);
}

}  // namespace lora
