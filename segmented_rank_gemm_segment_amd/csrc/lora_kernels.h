// Host-side launchers of the HIP kernels (internal to liblora).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lora.h"

namespace lora {

struct SegView {
  int n_rows;
  int max_segments;
  const int32_t *token_indices;
  const int32_t *row_segment;
  const int32_t *seg_off;
  const int32_t *seg_slot;
  const int32_t *seg_rank;
  const float *seg_scale;
  const int32_t *num_segments;
};

constexpr int kMaxProj = 8;

// Stacked projections: output columns [col_off[q], col_off[q + 1]) belong
// to projection q, whose rank rows are [q * rs, q * rs + rank) of a slot
// (rs = r_max / n_proj).  One projection: n_proj = 1, rs = r_max.
struct ProjView {
  int n_proj, rs;
  int col_off[kMaxProj + 1];
};

struct PoolView {
  int n_slots, r_max, d_in, d_out, dtype, policy;
  const void *A;
  const void *Bt;  // [n_slots][rs][d_out]: column j's rank rows are its own projection's
  const void *B;   // optional d_out-major copy of B ([n_slots][d_out][rs]) or null
  const float *dora;   // optional DoRA column factors ([n_slots][d_out]) or null
  ProjView proj;
};

// Projection of output column col (col < col_off[n_proj]).
__host__ __device__ inline int proj_of(const ProjView &pv, int col) {
  int q = 0;
#pragma unroll
  for (int i = 1; i < kMaxProj; ++i) q += (i < pv.n_proj && col >= pv.col_off[i]) ? 1 : 0;
  return q;
}

// E8M0 block scales of MXFP4 operands, one byte per 32 codes: rows of ldx and
// ldw bytes (multiples of 4).  x: scales of X when it holds codes too.
struct MxScales {
  const unsigned char *x;
  int64_t ldx;
  const unsigned char *w;
  int64_t ldw;
};

// The experts' product: sorted rows [off[e], off[e + 1]) are expert e's, whose
// codes and scales start e strides (bytes) after the first expert's.  Sorted
// row p is X row sorted_choice[p] / top_k, or X row p where that is null.
struct ExpertView {
  int n_choices, top_k, n_experts;
  const int32_t *off;
  const int32_t *sorted_choice;
  int64_t w_stride, s_stride;
};

struct BuildArgs {
  const int32_t *row_slot;
  int n, n_slots, r_max;
  const int32_t *slot_rank;
  const float *slot_scale;
  int32_t *token_indices, *row_segment, *seg_off, *seg_slot, *seg_rank;
  float *seg_scale;
  int32_t *num_segments, *status;
};

hipError_t launch_build_segments(const int32_t *row_slot, int n, int n_slots, int r_max,
                                 const int32_t *slot_rank, const float *slot_scale,
                                 int32_t *token_indices, int32_t *row_segment, int32_t *seg_off,
                                 int32_t *seg_slot, int32_t *seg_rank, float *seg_scale,
                                 int32_t *num_segments, int32_t *status, hipStream_t stream);

hipError_t launch_shrink(const void *X, int64_t ldx, const SegView &seg, const PoolView &pool,
                         float *H, hipStream_t stream);

// Segment build and shrink as one launch when every segment is short: block
// 0 builds the metadata while the other blocks compute H slot by slot from
// the per-row slot ids.  Returns hipErrorNotSupported (nothing launched)
// when the batch is outside that case.
hipError_t launch_build_shrink(const BuildArgs &a, const void *X, int64_t ldx,
                               const PoolView &pool, float *H, hipStream_t stream);

hipError_t launch_expand(const float *H, const SegView &seg, const PoolView &pool, void *Y,
                         int64_t ldy, hipStream_t stream);

// dH = dY B of every row's own adapter (adapter_dh.hip).
hipError_t launch_adapter_dh(const void *dY, int64_t lddy, const SegView &seg, const PoolView &pool,
                             float *dH, hipStream_t stream);

// dA[slot] (+)= s dH^T X and dBt[slot] (+)= s H^T dY over each segment's rows (either
// output may be null).
hipError_t launch_adapter_grads(const void *X, int64_t ldx, const float *dH, float *dA,
                                const void *dY, int64_t lddy, const float *H, float *dBt,
                                const SegView &seg, const PoolView &pool, bool accumulate,
                                hipStream_t stream);

// Adapter weights into a slot (one source per projection), then the slot's
// rank and scale alpha / rank.  b_rank_rows: B sources are [rank][ldb]
// (B^T) instead of [d_out_q][ldb].
hipError_t launch_pack_slot(const PoolView &pool, int32_t *slot_rank, float *slot_scale, int slot,
                            int rank, double alpha, const void *const *A_src, const int64_t *lda,
                            const void *const *B_src, const int64_t *ldb, int b_rank_rows,
                            hipStream_t stream);

// slot_scale[a] = alpha[a] / slot_rank[a] (0 for rank <= 0), on the device.
hipError_t launch_set_scales(const int32_t *slot_rank, const double *alpha, float *slot_scale,
                             int n_slots, hipStream_t stream);

// The pool's d_out-major B from its Bt, every slot.
hipError_t launch_write_b(const PoolView &pool, hipStream_t stream);

// DoRA column factors of one slot from its current contents and W.
hipError_t launch_dora_prepare(const PoolView &pool, const int32_t *slot_rank,
                               const float *slot_scale, int slot, const void *W, int64_t ldw,
                               const float *magnitude, hipStream_t stream);

// Y = X W^T (+ fused LoRA when seg/pool/H are given).  With wscale, W holds
// FP8 E4M3 codes (bf16 X and Y) and row j of the weight is wscale[j] times
// its codes.
hipError_t launch_gemm(const void *X, int64_t ldx, const void *W, int64_t ldw, void *Y,
                       int64_t ldy, int M, int K, int N, int dtype, const float *H,
                       const SegView *seg, const PoolView *pool, hipStream_t stream,
                       const float *wscale = nullptr);

// The same with an MXFP4 weight (codes W, ldw bytes a row) and bf16 X
// (mx.x null), or with both operands MXFP4 codes (ldx bytes a row).
hipError_t launch_gemm_mx(const void *X, int64_t ldx, const void *W, int64_t ldw,
                          const MxScales &mx, void *Y, int64_t ldy, int M, int K, int N,
                          const float *H, const SegView *seg, const PoolView *pool,
                          hipStream_t stream);

// Both operands MXFP4, large batches.
hipError_t launch_mx_product(const void *X, int64_t ldx, const void *W, int64_t ldw,
                             const MxScales &mx, void *Y, int64_t ldy, int M, int K, int N,
                             hipStream_t stream);

// Y[p] = X[row of p] W_e^T for every sorted row p of every expert e.
hipError_t launch_experts_gemm_mx(const void *X, int64_t ldx, const ExpertView &ex, const void *W,
                                  int64_t ldw, const MxScales &mx, void *Y, int64_t ldy, int K,
                                  int N, hipStream_t stream);

// The experts' products on bf16 weights [n_experts][N or K][ldw], w_stride elements
// apart: Y[p] = X[row of p] W_e^T (K = d_in, N = d_out), dX[p] = dY[p] W_e (K = d_out,
// N = d_in), and dW_e (+)= sum_p dY[p]^T X[row of p] (M = d_out, N = d_in).
hipError_t launch_experts_gemm(const void *X, int64_t ldx, const ExpertView &ex, const void *W,
                               int64_t ldw, void *Y, int64_t ldy, int K, int N, hipStream_t stream);
hipError_t launch_experts_gemm_rows(const void *dY, int64_t lddy, const ExpertView &ex,
                                    const void *W, int64_t ldw, void *dX, int64_t lddx, int K,
                                    int N, hipStream_t stream);
hipError_t launch_experts_gemm_weights(const void *dY, int64_t lddy, const void *X, int64_t ldx,
                                       const ExpertView &ex, void *dW, int64_t lddw, int dtype,
                                       bool accumulate, int M, int N, hipStream_t stream);

// MXFP4 codes and scales (ldq and lds bytes a row) of rows of d values, and back.
hipError_t launch_mx_quantize(const void *X, int64_t ldx, int n, int d, int dtype, void *q,
                              int64_t ldq, void *s, int64_t lds, hipStream_t stream);
hipError_t launch_mx_dequantize(const void *q, int64_t ldq, const void *s, int64_t lds, int n,
                                int d, int dtype, void *X, int64_t ldx, hipStream_t stream);

// Choices sorted by expert.  Batches past one workgroup's count them per block
// of kExpertBlockChoices: counts holds expert_blocks(n) (n_experts + 1) words.
constexpr int kExpertOneGroupChoices = 8192, kExpertBlockChoices = 4096;
inline int expert_blocks(int n_choices) {
  return (int)(((int64_t)n_choices + kExpertBlockChoices - 1) / kExpertBlockChoices);
}
hipError_t launch_experts_sort(const int32_t *ids, int n_choices, int n_experts, int32_t *offsets,
                               int32_t *sorted, int32_t *position, int32_t *status,
                               int32_t *counts, hipStream_t stream);
hipError_t launch_experts_gather(const void *X, int64_t ldx, const int32_t *position, int n, int k,
                                 int d, int dtype, void *Xs, int64_t lds, hipStream_t stream);
hipError_t launch_experts_combine(const void *Ys, int64_t lds, const float *w,
                                  const int32_t *position, int n, int k, int d, int dtype, void *Y,
                                  int64_t ldy, hipStream_t stream);
hipError_t launch_experts_combine_backward(const void *dY, int64_t ldy, const void *Ys, int64_t lds,
                                           const float *w, const int32_t *position, int n, int k,
                                           int d, int dtype, void *dYs, int64_t ldds, float *dw,
                                           hipStream_t stream);

// AdamW over many tensors (adamw.hip).  On the device: the tensors, and each chunk's
// tensor (a chunk is kAdamwChunk elements of one).
constexpr int kAdamwChunk = 4096, kAdamwBlock = 256;
struct AdamwTensor {
  void *param;
  const void *grad;
  float *master;         // or null
  int64_t numel;
  int64_t start;         // of its moments, in elements: whole blocks
  int64_t first_chunk;
};
constexpr int64_t kAdamwTensorBytes = sizeof(AdamwTensor);
struct AdamwArgs {
  int n_tensors, param_dtype, grad_dtype, bits;
  bool master;
  int64_t n_chunks;
  const AdamwTensor *tensors;
  const int32_t *chunk_tensor;
  void *m, *v;
  float *m_scale, *v_scale;
  int32_t *step;
  const int32_t *active;     // or null
  const float *lr_dev, *grad_scale;   // or null
  double lr, beta1, beta2, weight_decay;
  float eps;
  uint32_t seed;
};
hipError_t launch_adamw(const AdamwArgs &a, hipStream_t stream);
hipError_t launch_adamw_read(const void *m, const void *v, const float *m_scale,
                             const float *v_scale, int64_t total, int dtype, void *m_out,
                             void *v_out, hipStream_t stream);

// Inputs and outputs of the one-launch layer beyond the product's own
// (layer.cuh): the per-row slot ids and the pool's shrink operands, H, the
// sync buffer (or null) and the segment metadata it writes.
struct LayerArgs {
  const int32_t *row_slot;
  const void *A;              // pool A, [n_slots][r_max][d_in] (bf16)
  const int32_t *slot_rank;
  const float *slot_scale;
  int n_slots, rank_bound;    // rank_bound: ranks above it demote a row to base-only
  int d_in, r_max, rs, n_proj;
  float *H;                   // [n][r_max], written and read back
  uint32_t *sync;             // LORA_LAYER_SYNC_BYTES bytes, or null (no hand-off)
  int32_t *token_indices, *row_segment, *seg_off, *seg_slot, *seg_rank;
  float *seg_scale;
  int32_t *num_segments, *status;
};

// The whole layer in one launch (segment metadata, H, Y) for bf16 pools and
// 1 <= M <= 512 rows; hipErrorNotSupported (nothing launched) otherwise.
// With wscale, W holds FP8 E4M3 codes and row j of the weight is wscale[j]
// times its codes.
hipError_t launch_layer(const void *X, int64_t ldx, const void *W, int64_t ldw, void *Y,
                        int64_t ldy, int M, const PoolView &pool, const LayerArgs &lay,
                        hipStream_t stream, const float *wscale = nullptr);

// Device scratch of the allocation-free call lora_linear_fused_static: byte
// offsets of its parts, each 256-byte aligned.  H is float [n][r_max]; the
// segment arrays hold up to LORA_MAX_SLOTS + 1 segments (min(n, n_slots + 1)).
constexpr size_t kScrAlign = 256;
constexpr size_t scr_up(size_t x) { return (x + kScrAlign - 1) / kScrAlign * kScrAlign; }
constexpr size_t kScrH = 0;
constexpr size_t kScrTok = scr_up(kScrH + 4ull * LORA_STATIC_MAX_H);
constexpr size_t kScrRowSeg = scr_up(kScrTok + 4ull * LORA_STATIC_MAX_ROWS);
constexpr size_t kScrSegOff = scr_up(kScrRowSeg + 4ull * LORA_STATIC_MAX_ROWS);
constexpr size_t kScrSegSlot = scr_up(kScrSegOff + 4ull * (LORA_MAX_SLOTS + 2));
constexpr size_t kScrSegRank = scr_up(kScrSegSlot + 4ull * (LORA_MAX_SLOTS + 1));
constexpr size_t kScrSegScale = scr_up(kScrSegRank + 4ull * (LORA_MAX_SLOTS + 1));
constexpr size_t kScrNumSeg = scr_up(kScrSegScale + 4ull * (LORA_MAX_SLOTS + 1));
constexpr size_t kScrStatus = kScrNumSeg + kScrAlign;
constexpr size_t kScratchBytes = kScrStatus + kScrAlign;

// Device address of this device's scratch (looked up once per device).
hipError_t static_scratch(void **out);

}  // namespace lora
