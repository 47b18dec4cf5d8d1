// Launches of the products with MXFP4 operands: an MXFP4 weight under bf16
// activations, with or without the LoRA term, both operands MXFP4, and the
// experts' product, on the kernels that tile_choice.h names for the batch.
#include "mx_mid.cuh"
#include "mx_stream.cuh"
#include "mx_weight.cuh"

namespace lora {

hipError_t launch_gemm_mx(const void *X, int64_t ldx, const void *W, int64_t ldw,
                          const MxScales &mx, void *Y, int64_t ldy, int M, int K, int N,
                          const float *H, const SegView *seg, const PoolView *pool,
                          hipStream_t stream) {
  if (mx.x) {
    const MxKernel k = mx_both_kernel_of(M, N);
    if (k == kMxPersistent) return launch_mx_product(X, ldx, W, ldw, mx, Y, ldy, M, K, N, stream);
    if (k == kMxTiles128) {
      // in units of four codes
      GemmArgs g = gemm_args(X, ldx / 2, W, ldw / 2, Y, ldy, M, K / 4, N, nullptr, nullptr, nullptr);
      g.mx = mx;
      return launch_tile_plain<LORA_GEMM_MID, kMxXW>(g, stream);
    }
    GemmArgs g = gemm_args(X, ldx, W, ldw * 2, Y, ldy, M, K, N, nullptr, nullptr, nullptr);
    g.mx = mx;
    return launch_mx_mid<true>(g, k, false, stream);
  }
  const bool lora = seg != nullptr;
  GemmArgs g = gemm_args(X, ldx, W, ldw * 2, Y, ldy, M, K, N, H, seg, pool);
  g.mx = mx;
  const MxKernel k = mx_weight_kernel_of(M, N, lora);
  switch (k) {
    case kMxStream8:
    case kMxStream16: return launch_mx_stream(g, k, lora, stream);
    case kMxTiles32:
    case kMxTiles64: return launch_mx_mid<false>(g, k, lora, stream);
    case kMxTiles128: return launch_tile<LORA_GEMM_MID, kMxW>(g, lora, stream);
    case kMxTiles192: return launch_tile_lora<LORA_GEMM_LARGE192, kMxW>(g, stream);
    case kMxTiles256: return launch_tile_lora<LORA_GEMM_LARGE, kMxW>(g, stream);
    default: return launch_mx_weight<false>(g, stream);
  }
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
  switch (mx_experts_kernel_of(ex.n_choices, ex.n_experts, K, N)) {
    case kMxStream8: return launch_experts_stream<4, 2>(g, tiles(8), stream);
    case kMxStream16: return launch_experts_stream<4, 1>(g, tiles(16), stream);
    case kMxTiles32: return launch_experts_mid(g, tiles(32), stream);
    default: return launch_mx_weight<true>(g, stream);
  }
}

}  // namespace lora
