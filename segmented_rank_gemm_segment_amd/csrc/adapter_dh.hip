// dH = dY B_a of a batch's rows, the first step of the adapters' gradients:
//
//   dH[i][k] = sum_j dY[i][j] Bt_a[k][j]      k < r_a, i in a
//
// A work item is 16 RA rows of one segment at most (seg_item) and 16 RB ranks, a
// workgroup's; its eight waves take every eighth piece of the sum's axis.  A lane of the
// matrix instructions holds 16 bytes of one row of either operand, so both come from
// memory as they lie there, without LDS: 64 bytes of each of 16 rows a load, and a piece's
// loads while the products of the one before run.  (32 x 32 instructions take 32 bytes of
// each of 32 rows a load, up to 1.15 times as long.)  The waves' sums are added through
// LDS in a fixed order.  fp32 goes through the fp32 matrix instruction, a lane's 4 values
// in turn.
//
// Bound by how fast a workgroup gets its operands, some 45 GB/s a CU, and pieces twice as
// long change nothing; so by the workgroups that share the work, and then by RA and RB,
// which say how often dY and the rank rows are read.  Measured, in us: 128 segments of 2
// rows, d_out 4096, rank 16, 8.2 (the forward pass's shrink kernels 10.9); 64 of 32, 4096,
// rank 16, 10.8 (23.9); 8 of 64, 4096, rank 64, 10.6 (18.9); 64 of 64, 14336, rank 64, 84
// (388); 8 of 2118, 14336, rank 64, 216 (186, 2.2 TB/s of dY).
#include <algorithm>

#include "lds_dma.cuh"
#include "lora_device.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kWaves = 8;
constexpr int kPiece = 2;                     // loads of a row's 64 bytes

struct DhArgs {
  const void *dY;
  int64_t lddy;
  const void *Bt;
  const int32_t *token_indices, *row_segment, *seg_off, *seg_slot, *seg_rank, *num_segments;
  float *dH;
  int r_max, d, nb, seg_cap;
};

// RA: blocks of 16 rows; RB: blocks of 16 ranks, from rank k0 on.
template <typename T, int RA, int RB>
__device__ __forceinline__ void dh_item(const DhArgs &a, const SegItem &it, int k0, float *part) {
  const int l = threadIdx.x & (kWave - 1), quarter = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  constexpr int STEP = 64 / (int)sizeof(T), SPAN = STEP * kPiece;     // elements of a load, a piece
  const int off = quarter * (STEP / 4);
  const T *ap[RA], *bp[RB];
#pragma unroll
  for (int i = 0; i < RA; ++i)
    ap[i] = static_cast<const T *>(a.dY) +
            (int64_t)a.token_indices[min(it.p0 + i * 16 + (l & 15), it.p1 - 1)] * a.lddy + off;
#pragma unroll
  for (int i = 0; i < RB; ++i)
    bp[i] = static_cast<const T *>(a.Bt) +
            ((int64_t)it.slot * a.r_max + min(k0 + i * 16 + (l & 15), it.r - 1)) * a.d + off;
  struct Piece {
    u32x4 a[RA][kPiece], b[RB][kPiece];
  };
  auto load = [&](Piece &p, int j0) __attribute__((always_inline)) {
    if (j0 + SPAN <= a.d) {
#pragma unroll
      for (int q = 0; q < kPiece; ++q) {
#pragma unroll
        for (int i = 0; i < RA; ++i) p.a[i][q] = *reinterpret_cast<const u32x4 *>(ap[i] + j0 + q * STEP);
#pragma unroll
        for (int i = 0; i < RB; ++i) p.b[i][q] = *reinterpret_cast<const u32x4 *>(bp[i] + j0 + q * STEP);
      }
    } else {
      // past the row's end: its first 16 bytes instead, and zeros of both
#pragma unroll
      for (int q = 0; q < kPiece; ++q) {
        const bool in = j0 + q * STEP + off < a.d;
        const int at = in ? j0 + q * STEP : -off;
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RA; ++i) {
          const u32x4 x = *reinterpret_cast<const u32x4 *>(ap[i] + at);
          p.a[i][q] = in ? x : zero;
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const u32x4 x = *reinterpret_cast<const u32x4 *>(bp[i] + at);
          p.b[i][q] = in ? x : zero;
        }
      }
    }
  };
  f32x4 acc[RA][RB];
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Piece &p) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kPiece; ++q)
#pragma unroll
      for (int i = 0; i < RA; ++i)
#pragma unroll
        for (int j = 0; j < RB; ++j) {
          if constexpr (sizeof(T) == 2) {
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(p.a[i][q]), as_bf16x8(p.b[j][q]),
                                                                acc[i][j], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __uint_as_float(p.a[i][q][e]), __uint_as_float(p.b[j][q][e]), acc[i][j], 0, 0, 0);
          }
        }
  };
  const int pieces = (a.d + SPAN - 1) / SPAN;
  if (w < pieces) {
    Piece cur, nxt;
    load(cur, w * SPAN);
    for (int p = w; p < pieces; p += kWaves) {
      if (p + kWaves < pieces) load(nxt, (p + kWaves) * SPAN);
      compute(cur);
      cur = nxt;
    }
  }
  // register e of block (i, j) at ((i RB + j) 4 + e) of the wave's
  constexpr int N = RA * RB * 4;
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[(w * N + (i * RB + j) * 4 + e) * kWave + l] = acc[i][j][e];
  __syncthreads();
  for (int v = w; v < N; v += kWaves) {
    float x = part[v * kWave + l];
#pragma unroll
    for (int o = 1; o < kWaves; ++o) x += part[(o * N + v) * kWave + l];
    const int block = v / 4, p = it.p0 + block / RB * 16 + quarter * 4 + v % 4;
    const int k = k0 + block % RB * 16 + (l & 15);
    if (p < it.p1 && k < it.r) a.dH[(int64_t)a.token_indices[p] * a.r_max + k] = x;
  }
}

// Items of up to 16 RA rows, workgroups of 16 RB ranks; both halved while that holds the
// item too.
template <typename T, int RA, int RB>
__device__ __forceinline__ void dh_fit(const DhArgs &a, const SegItem &it, int k0, float *part) {
  if constexpr (RA > 1) {
    if (it.p1 - it.p0 <= 8 * RA) return dh_fit<T, RA / 2, RB>(a, it, k0, part);
  }
  if constexpr (RB > 1) {
    if (it.r <= 8 * RB) return dh_fit<T, RA, RB / 2>(a, it, k0, part);
  }
  dh_item<T, RA, RB>(a, it, k0, part);
}
template <typename T, int RA, int RB>
__global__ __launch_bounds__(kWaves *kWave) void adapter_dh_kernel(DhArgs a) {
  __shared__ float part[kWaves * RA * RB * 4 * kWave];
  const SegItem it = seg_item(blockIdx.x, a.nb, 16 * RA, a.seg_cap, a.token_indices, a.row_segment,
                              a.num_segments, a.seg_rank, a.seg_off, a.seg_slot, nullptr);
  const int k0 = blockIdx.y * 16 * RB;
  if (it.ok && k0 < it.r) dh_fit<T, RA, RB>(a, it, k0, part);
}

template <typename T, int RA, int RB>
void launch(DhArgs a, int n, hipStream_t stream) {
  a.nb = (n + 16 * RA - 1) / (16 * RA);
  const dim3 grid(a.nb + a.seg_cap, (a.r_max + 16 * RB - 1) / (16 * RB));
  hipLaunchKernelGGL((adapter_dh_kernel<T, RA, RB>), grid, dim3(kWaves * kWave), 0, stream, a);
}
// 16 x 16 workgroups while they are few, then 32 rows and all ranks, for rank 64 64 rows in
// the longest batches.  16 x 16 against 32 rows, in us, at d_out 4096: rank 16, 2048 rows
// 10.8 and 14.1, 4096 rows 18.9 and 15.7; rank 64, 1024 rows 18.8 and 25.3, 2048 rows 34.5
// and 25.5.  32 against 64 rows: rank 64, 4096 rows 28.3 and 33.4, 16944 rows 76 and 69;
// rank 16, 16944 rows 41 and 46.
constexpr int64_t kSmallWork = 49152, kSmallWorkRank64 = 65536;       // rows x ranks
constexpr int kLargeRows = 16384;
template <typename T>
void launch_tiles(const DhArgs &a, int n, hipStream_t stream) {
  if ((int64_t)n * a.r_max <= (a.r_max > 32 ? kSmallWorkRank64 : kSmallWork)) launch<T, 1, 1>(a, n, stream);
  else if (a.r_max <= 16) launch<T, 2, 1>(a, n, stream);
  else if (a.r_max <= 32) launch<T, 2, 2>(a, n, stream);
  else if (n < kLargeRows) launch<T, 2, 4>(a, n, stream);
  else launch<T, 4, 4>(a, n, stream);
}

}  // namespace

hipError_t launch_adapter_dh(const void *dY, int64_t lddy, const SegView &seg, const PoolView &pool,
                             float *dH, hipStream_t stream) {
  const int n = seg.n_rows, S = std::min(std::min(n, pool.n_slots + 1), seg.max_segments);
  const DhArgs a{dY, lddy, pool.Bt, seg.token_indices, seg.row_segment, seg.seg_off, seg.seg_slot,
                 seg.seg_rank, seg.num_segments, dH, pool.r_max, pool.d_out, 0, S};
  if (pool.dtype == LORA_BF16) launch_tiles<bf16_t>(a, n, stream);
  else launch_tiles<float>(a, n, stream);
  return hipGetLastError();
}

}  // namespace lora
