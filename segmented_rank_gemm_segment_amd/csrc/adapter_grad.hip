// Gradients of the adapters of a batch: for every slot a with rows in it,
//
//   dA_a[k][c]  (+)= s_a sum_{i in a} dH[i][k] X[i][c]         k < r_a
//   dBt_a[k][j] (+)= s_a sum_{i in a} H[i][k] dY[i][j]
//
// two products of the same form, out = s V^T U over the segment's rows, both in one
// launch.  Bound by memory: U is read once and the gradients written once, and what
// is multiplied per byte of U, up to 64 ranks, is below what the matrix cores do
// meanwhile.  Measured: 16,943 rows of 8 slots, 4096 -> 14336, ranks 8 to 64, 157 to 165
// us (625 MB of X and dY, 3.9 TB/s); 2303 rows of 37 slots, 8192 -> 1024, ranks 8 to 32,
// added to what is there, 27 us (42 MB read and twice 27 MB of gradients, 3.6 TB/s).
// A segment's rows stay in the workgroup of their columns, so few long segments leave CUs
// idle: one of 16,943 rows, 4096 -> 4096, rank 16, has 32 workgroups and takes 240 us for the
// 54 of its bytes (8 segments: 45), 256 -> 256 two, 228 us for 3.
//
// Segments of more than kShortRows rows go through the matrix cores.  The reduction runs
// over rows, so both operands want 8 rows of one column in a lane.  A lane loads VEC
// neighbouring columns of 8 rows and transposes them among its own registers (byte
// permutations), so U goes from memory to the matrix cores without LDS.  Column j of every
// lane's VEC is one operand: a wave holds 32 VEC columns, and in its accumulators a lane
// has VEC neighbouring columns of a rank row.  The workgroup's four waves take every
// fourth 16 rows of the same columns, and their sums are added through LDS in a fixed
// order.
//
// V is fp32 and is split into three bf16, each the rounding of what the ones before
// leave, which hold its 24 significant bits; each is multiplied (with two, 16 bits, the
// gradients were 2.4e-6 off where fp32 sums are 3e-7).  fp32 pools go through the fp32
// matrix instruction.
//
// Shorter segments, a decode batch's or many tenants' few rows each, are bound by the
// writes: each thread keeps its columns of all rows in registers and forms one rank row
// after the other (128 segments of two rows, 4096 -> 4096, ranks 8 and 16, 14 us for 45
// MB).  Each of the two launches leaves the other's segments alone, 2 to 4 us where that
// is all of them.
#include "lds_dma.cuh"
#include "lora_device.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kWaves = 4, kRows = 16;       // rows of a step: 8 a lane half
constexpr int kShortRows = 8;

struct GradJob {
  const void *U;
  int64_t ldu;
  const float *V;
  float *out;
  int d, blocks;                            // columns, workgroups along them
};
struct GradArgs {
  GradJob job[2];
  const int32_t *token_indices, *seg_off, *seg_slot, *seg_rank, *num_segments;
  const float *seg_scale;
  int r_max;
  int accumulate;
};

// WORDS 4-byte words of a row.
template <int WORDS> struct Words;
template <> struct Words<4> {
  uint4 w;
  __device__ __forceinline__ void load(const void *p) { w = ldg16(p); }
  __device__ __forceinline__ void clear() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t at(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
};
template <> struct Words<2> {
  uint2 w;
  __device__ __forceinline__ void load(const void *p) { w = *static_cast<const uint2 *>(p); }
  __device__ __forceinline__ void clear() { w = make_uint2(0u, 0u); }
  __device__ __forceinline__ uint32_t at(int i) const { return i == 0 ? w.x : w.y; }
};

// N neighbouring columns of a rank row: p (+)= scale x.
template <int N>
__device__ __forceinline__ void store_row(float *p, const float (&x)[N], float scale, bool add) {
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    float o[4] = {x[j] * scale, x[j + 1] * scale, x[j + 2] * scale, x[j + 3] * scale};
    if (add) {
      float old[4];
      Elem<float>::unpack(ldg16(p + j), old);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += old[e];
    }
    stg16(p + j, Elem<float>::pack(o));
  }
}

// RB: blocks of 32 ranks; VEC: columns of a lane.
template <typename T, int RB, int VEC>
__global__ __launch_bounds__(kWaves *kWave, 2) void adapter_grad_kernel(GradArgs a) {
  constexpr int COLS = 32 * VEC, WORDS = VEC * (int)sizeof(T) / 4;
  constexpr bool BF16 = sizeof(T) == 2;
  // one half of a rank block's accumulators of every wave
  __shared__ float part[kWaves][8][VEC][kWave];
  const int l = threadIdx.x & (kWave - 1), h = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const bool second = (int)blockIdx.x >= a.job[0].blocks;
  const GradJob &J = a.job[second ? 1 : 0];
  const int col = ((int)blockIdx.x - (second ? a.job[0].blocks : 0)) * COLS + (l & 31) * VEC;
  const bool active = col < J.d;
  const T *const U = static_cast<const T *>(J.U) + (active ? col : 0);

  struct Stage {
    Words<WORDS> u[8];
    float v[RB][8];
  };
  auto segment = [&](int seg) __attribute__((always_inline)) {
    const SegMeta meta = load_seg_meta(seg, a.num_segments, a.seg_rank, a.seg_off, a.seg_slot, a.seg_scale);
    if (meta.r <= 0) return;
    const int o0 = meta.o0, o1 = meta.o1, r = meta.r;
    const int steps = (o1 - o0 + kRows - 1) / kRows;
    auto rows_of = [&](int step) __attribute__((always_inline)) {
      return a.token_indices[min(o0 + step * kRows + (l & 15), o1 - 1)];
    };
    auto load = [&](Stage &s, int rows) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int lo = __builtin_amdgcn_readlane(rows, q), hi = __builtin_amdgcn_readlane(rows, q + 8);
        const int row = h ? hi : lo;
        s.u[q].load(U + (int64_t)row * J.ldu);
#pragma unroll
        for (int b = 0; b < RB; ++b)
          s.v[b][q] = J.V[(int64_t)row * a.r_max + min(b * 32 + (l & 31), a.r_max - 1)];
      }
    };
    f32x16 acc[RB][VEC];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[b][j][v] = 0.f;

    auto compute = [&](Stage &s, int step) __attribute__((always_inline)) {
      // ranks past the slot's (H holds anything there), and rows past the segment
      const int left = o1 - (o0 + step * kRows + h * 8);
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (b * 32 + (l & 31) >= r || q >= left) s.v[b][q] = 0.f;
      if ((step + 1) * kRows > o1 - o0) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q >= left) s.u[q].clear();
      }
      if constexpr (BF16) {
        mfma_bf16x8 col8[VEC];
#pragma unroll
        for (int d = 0; d < VEC / 2; ++d) {
          u32x4 even, odd;
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint32_t x = s.u[2 * p].at(d), y = s.u[2 * p + 1].at(d);
            even[p] = __builtin_amdgcn_perm(y, x, 0x05040100u);
            odd[p] = __builtin_amdgcn_perm(y, x, 0x07060302u);
          }
          col8[2 * d] = as_bf16x8(even);
          col8[2 * d + 1] = as_bf16x8(odd);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          if (b * 32 >= r) break;
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            u32x4 x;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              x[p] = pack_bf16x2(s.v[b][2 * p], s.v[b][2 * p + 1]);
              s.v[b][2 * p] -= bf16_lo(x[p]);       // exact: what is left for the next part
              s.v[b][2 * p + 1] -= bf16_hi(x[p]);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j)
              acc[b][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(x), col8[j], acc[b][j], 0, 0, 0);
          }
        }
      } else {
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          if (b * 32 >= r) break;
#pragma unroll
          for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int j = 0; j < VEC; ++j)
              acc[b][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                  s.v[b][q], __uint_as_float(s.u[q].at(j)), acc[b][j], 0, 0, 0);
        }
      }
    };

    if (w < steps) {
      Stage cur, nxt;
      int rows = rows_of(w);
      load(cur, rows);
      rows = rows_of(min(w + kWaves, steps - 1));
      for (int step = w; step < steps; step += kWaves) {
        load(nxt, rows);                            // (the last one reads the last step again)
        rows = rows_of(min(step + 2 * kWaves, steps - 1));
        compute(cur, step);
        cur = nxt;
      }
    }

    float *const out = J.out + (int64_t)meta.slot * a.r_max * J.d + col;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      if (b * 32 >= r) break;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < 8; ++v)
#pragma unroll
          for (int j = 0; j < VEC; ++j) part[w][v][j][l] = acc[b][j][half * 8 + v];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int v = w * 2 + i, k = b * 32 + acc_row(half * 8 + v, l);
          float x[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            x[j] = part[0][v][j][l];
#pragma unroll
            for (int o = 1; o < kWaves; ++o) x[j] += part[o][v][j][l];
          }
          if (k < r && active) store_row(out + (int64_t)k * J.d, x, meta.sc, a.accumulate != 0);
        }
      }
    }
  };

  // Of this workgroup's segments, 64 at a time, the long ones.
  const int S = __builtin_amdgcn_readfirstlane(*a.num_segments);
  for (int s0 = blockIdx.y; s0 < S; s0 += kWave * gridDim.y) {
    const int mine = s0 + l * gridDim.y;
    const int at = min(mine, S - 1);
    const bool is_long = mine < S && a.seg_off[at + 1] - a.seg_off[at] > kShortRows;
    for (uint64_t todo = __ballot(is_long); todo; todo &= todo - 1)
      segment(s0 + (__ffsll((unsigned long long)todo) - 1) * (int)gridDim.y);
  }
}

// One short segment, 256 threads' columns.
template <typename T>
__global__ __launch_bounds__(kWaves *kWave) void adapter_grad_short_kernel(GradArgs a) {
  constexpr int VEC = Elem<T>::kVec, COLS = kWaves * kWave * VEC;
  __shared__ __align__(16) float vs[64][kShortRows];
  const SegMeta meta = load_seg_meta(blockIdx.y, a.num_segments, a.seg_rank, a.seg_off, a.seg_slot, a.seg_scale);
  const int n = meta.o1 - meta.o0, r = meta.r;
  if ((int)blockIdx.y >= meta.S || r <= 0 || n > kShortRows) return;
  const bool second = (int)blockIdx.x >= a.job[0].blocks;
  const GradJob &J = a.job[second ? 1 : 0];
  const int col = ((int)blockIdx.x - (second ? a.job[0].blocks : 0)) * COLS + threadIdx.x * VEC;
  const bool active = col < J.d;
  const T *const U = static_cast<const T *>(J.U) + (active ? col : 0);
  uint4 raw[kShortRows];
#pragma unroll
  for (int i = 0; i < kShortRows; ++i)
    if (i < n) raw[i] = ldg16(U + (int64_t)a.token_indices[meta.o0 + i] * J.ldu);
  for (int i = threadIdx.x; i < r * kShortRows; i += kWaves * kWave) {
    const int k = i / kShortRows, q = i % kShortRows;
    vs[k][q] = q < n ? J.V[(int64_t)a.token_indices[meta.o0 + q] * a.r_max + k] : 0.f;
  }
  float u[kShortRows][VEC];
#pragma unroll
  for (int i = 0; i < kShortRows; ++i) {
    if (i >= n) raw[i] = make_uint4(0u, 0u, 0u, 0u);
    Elem<T>::unpack(raw[i], u[i]);
  }
  __syncthreads();
  if (!active) return;
  float *out = J.out + (int64_t)meta.slot * a.r_max * J.d + col;
  for (int k = 0; k < r; ++k, out += J.d) {
    const f32x4 v0 = *reinterpret_cast<const f32x4 *>(vs[k]), v1 = *reinterpret_cast<const f32x4 *>(vs[k] + 4);
    float x[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      x[j] = v0[0] * u[0][j];
#pragma unroll
      for (int i = 1; i < kShortRows; ++i) x[j] = fmaf(i < 4 ? v0[i] : v1[i - 4], u[i][j], x[j]);
    }
    store_row(out, x, meta.sc, a.accumulate != 0);
  }
}

template <typename T, int RB, int VEC>
void launch_long(GradArgs a, int S, hipStream_t stream) {
  int blocks = 0;
  for (GradJob &j : a.job) blocks += j.blocks = (j.d + 32 * VEC - 1) / (32 * VEC);
  hipLaunchKernelGGL((adapter_grad_kernel<T, RB, VEC>), dim3(blocks, S), dim3(kWaves * kWave), 0, stream, a);
}
template <typename T>
void launch_short(GradArgs a, int S, hipStream_t stream) {
  constexpr int COLS = kWaves * kWave * Elem<T>::kVec;
  int blocks = 0;
  for (GradJob &j : a.job) blocks += j.blocks = (j.d + COLS - 1) / COLS;
  hipLaunchKernelGGL(adapter_grad_short_kernel<T>, dim3(blocks, S), dim3(kWaves * kWave), 0, stream, a);
}

}  // namespace

hipError_t launch_adapter_grads(const void *X, int64_t ldx, const float *dH, float *dA,
                                const void *dY, int64_t lddy, const float *H, float *dBt,
                                const SegView &seg, const PoolView &pool, bool accumulate,
                                hipStream_t stream) {
  GradArgs a{};
  int jobs = 0;
  if (dBt) a.job[jobs++] = GradJob{dY, lddy, H, dBt, pool.d_out, 0};
  if (dA) a.job[jobs++] = GradJob{X, ldx, dH, dA, pool.d_in, 0};
  if (jobs == 0) return hipSuccess;
  a.token_indices = seg.token_indices;
  a.seg_off = seg.seg_off;
  a.seg_slot = seg.seg_slot;
  a.seg_rank = seg.seg_rank;
  a.num_segments = seg.num_segments;
  a.seg_scale = seg.seg_scale;
  a.r_max = pool.r_max;
  a.accumulate = accumulate;
  const int n = seg.n_rows, S = n < pool.n_slots + 1 ? n : pool.n_slots + 1;
  // no more long segments than rows for them
  const int longs = n / (kShortRows + 1) < S ? n / (kShortRows + 1) : S;
  if (pool.dtype == LORA_BF16) {
    launch_short<bf16_t>(a, S, stream);
    if (longs > 0 && pool.r_max <= 32) launch_long<bf16_t, 1, 8>(a, longs, stream);
    else if (longs > 0) launch_long<bf16_t, 2, 4>(a, longs, stream);
  } else {
    launch_short<float>(a, S, stream);
    if (longs > 0 && pool.r_max <= 32) launch_long<float, 1, 4>(a, longs, stream);
    else if (longs > 0) launch_long<float, 2, 4>(a, longs, stream);
  }
  return hipGetLastError();
}

}  // namespace lora
