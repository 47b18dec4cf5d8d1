// Launches of the products with MXFP4 operands: an MXFP4 weight under bf16
// activations, with or without the LoRA term, both operands MXFP4, and the
// experts' product.  Which kernel a batch takes is a matter of how many tiles of
// each size it makes for the CUs.
#include <cmath>

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

// Cost of a batch in tiles of 64, 128 and 256 rows and columns: rounds over the
// CUs (64: several workgroups follow each other on a CU, so parts of a round)
// times a round's time, given in microseconds at K 4096.
struct TileCost {
  double t64, t128, t256;
};
TileCost tile_cost(int M, int N, double us64, double us128, double us256) {
  auto tiles = [&](int b) { return (double)(((int64_t)M + b - 1) / b) * (((int64_t)N + b - 1) / b); };
  const double n64 = tiles(64) / kCUs;
  return TileCost{(n64 < 1 ? 1 : n64) * us64, ceil(tiles(128) / kCUs) * us128,
                  ceil(tiles(256) / kCUs) * us256};
}

}  // namespace

hipError_t launch_gemm_mx(const void *X, int64_t ldx, const void *W, int64_t ldw,
                          const MxScales &mx, void *Y, int64_t ldy, int M, int K, int N,
                          const float *H, const SegView *seg, const PoolView *pool,
                          hipStream_t stream) {
  const bool lora = seg != nullptr;
  if (mx.x) {
    const TileCost c = tile_cost(M, N, 6.6, 19.6, 27.5);
    if (c.t64 <= c.t128 && c.t64 <= c.t256) {
      GemmArgs g = gemm_args(X, ldx, W, ldw * 2, Y, ldy, M, K, N, nullptr, nullptr, nullptr);
      g.mx = mx;
      return launch_mx_mid<true>(g, false, stream);
    }
    if (c.t256 <= c.t128) return launch_mx_product(X, ldx, W, ldw, mx, Y, ldy, M, K, N, stream);
    // in units of four codes
    GemmArgs g = gemm_args(X, ldx / 2, W, ldw / 2, Y, ldy, M, K / 4, N, nullptr, nullptr, nullptr);
    g.mx = mx;
    return launch_codes<LORA_GEMM_MID>(g, stream);
  }
  GemmArgs g = gemm_args(X, ldx, W, ldw * 2, Y, ldy, M, K, N, H, seg, pool);
  g.mx = mx;
  if (stream_rows(M, N)) return launch_mx_stream(g, lora, stream);
  // Base-only rows of a batch with adapters have the base product's bits, so both
  // go by the same rule as far as the order of adding up K goes: the 64-tiles', or
  // that of all others.
  const TileCost c = tile_cost(M, N, 12.8, 46.5, 85);
  if (c.t64 <= c.t128 && c.t64 <= c.t256) return launch_mx_mid<false>(g, lora, stream);
  if (!lora)
    return c.t256 <= c.t128 ? launch_mx_weight<false>(g, stream)
                            : launch_tile<LORA_GEMM_MID, kMxW>(g, false, stream);
  // With adapters the shared tiles, whose LoRA term goes through LDS: read from
  // memory into each wave's fragments instead, at the end of the persistent
  // kernel's tiles, it cost 11 us a tile, and the two were level (16943 x 4096 x
  // 14336, 8 slots: 1.69 ms).
  if (c.t128 <= c.t256 * (109. / 85)) return launch_tile<LORA_GEMM_MID, kMxW>(g, true, stream);
  if (large192_tiles(M, N)) return launch_tile<LORA_GEMM_LARGE192, kMxW>(g, true, stream);
  return launch_tile<LORA_GEMM_LARGE, kMxW>(g, true, stream);
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
  // by the mean rows of an expert, in us.  2: 16 experts of 4096 -> 4096 28 in tiles
  // of 8 against 38 in tiles of 16.  Streamed against the 32-row tiles: 3 rows 38
  // against 31, 8 rows 50 against 33, but where K is short, on 64 experts of 2048 ->
  // 1536, 4 rows 29 against 35, 8 rows 37 against 38, 16 rows 52 against 43.  Those
  // against the 256-tiles: 64 rows 89 against 98 and 80 against 97, 96 rows 116
  // against 100 and 105 against 99.
  const int rows = ex.n_choices / ex.n_experts;
  if (rows <= 2) return launch_experts_stream<4, 2>(g, tiles(8), stream);
  if (rows <= 8 && K <= 2048) return launch_experts_stream<4, 1>(g, tiles(16), stream);
  if (rows < 80) return launch_experts_mid(g, tiles(32), stream);
  return launch_mx_weight<true>(g, stream);
}

}  // namespace lora
