// Gradients of the adapters of a batch: for every slot a with rows in it,
//
//   dA_a[k][c]  (+)= s_a sum_{i in a} dH[i][k] X[i][c]         k < r_a
//   dBt_a[k][j] (+)= s_a sum_{i in a} H[i][k] dY[i][j]
//
// two products of the same form, out = s V^T U over the segment's rows, in one
// launch.  Bound by memory: U is read once and the gradients written once, and what
// is multiplied per byte of U, up to 64 ranks, is below what the matrix cores do
// meanwhile.
//
// The reduction runs over rows, so both matrix operands want 8 rows of one column in
// a lane.  A lane loads 16 bytes of each of 8 rows: 8 columns of 8 rows, which it
// transposes among its own registers (32 byte permutations), so U goes from memory
// to the matrix cores without LDS.  Column j of every lane's 8 is one operand: a wave
// holds 256 columns, and in its accumulators a lane has 8 neighbouring columns of a
// rank row, stored as 32 bytes.
//
// V is fp32 and is split into three bf16, each the rounding of what the ones before
// leave, which hold its 24 significant bits; each is multiplied (with two, 16 bits, the
// gradients were 2.4e-6 off where fp32 sums are 3e-7).  fp32 pools go through the fp32 matrix instruction.
//
// A segment of up to kRows rows is one step: each wave of the workgroup takes other
// columns.  In a longer one the four waves take every fourth step of the same columns
// and their sums are added through LDS in a fixed order.
#include "lds_dma.cuh"
#include "lora_device.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kWaves = 4, kRows = 16;       // rows of a step: 8 a lane half

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

// RB: blocks of 32 ranks.
template <typename T, int RB>
__global__ __launch_bounds__(kWaves *kWave, RB == 1 ? 2 : 1) void adapter_grad_kernel(GradArgs a) {
  constexpr int VEC = Elem<T>::kVec, COLS = 32 * VEC;
  constexpr bool BF16 = sizeof(T) == 2;
  // one half of a rank block's accumulators of every wave
  __shared__ float part[kWaves][8][VEC][kWave];
  const int l = threadIdx.x & (kWave - 1), h = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int seg = blockIdx.y;
  const SegMeta meta = load_seg_meta(seg, a.num_segments, a.seg_rank, a.seg_off, a.seg_slot, a.seg_scale);
  if (seg >= meta.S || meta.r <= 0) return;
  const int o0 = meta.o0, o1 = meta.o1, r = meta.r;
  const int steps = (o1 - o0 + kRows - 1) / kRows;
  const bool split = steps > 1;
  const bool second = (int)blockIdx.x >= a.job[0].blocks;
  const GradJob &J = a.job[second ? 1 : 0];
  int block = blockIdx.x - (second ? a.job[0].blocks : 0);
  if (!split) {                             // four column blocks in one workgroup
    if (block % kWaves) return;
    block += w;
    if (block >= J.blocks) return;
  }
  const int col = block * COLS + (l & 31) * VEC;
  const bool active = col < J.d;
  const T *const U = static_cast<const T *>(J.U) + (active ? col : 0);

  struct Stage {
    uint4 u[8];
    float v[RB][8];
  };
  auto rows_of = [&](int step) __attribute__((always_inline)) {
    return a.token_indices[min(o0 + step * kRows + (l & 15), o1 - 1)];
  };
  auto load = [&](Stage &s, int rows) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int lo = __builtin_amdgcn_readlane(rows, q), hi = __builtin_amdgcn_readlane(rows, q + 8);
      const int row = h ? hi : lo;
      s.u[q] = ldg16(U + (int64_t)row * J.ldu);
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
        if (q >= left) s.u[q] = make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (BF16) {
      mfma_bf16x8 col8[8];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        u32x4 even, odd;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t x = (&s.u[2 * p].x)[d], y = (&s.u[2 * p + 1].x)[d];
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
            s.v[b][2 * p] -= bf16_lo(x[p]);         // exact: what is left for the next part
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
                s.v[b][q], __uint_as_float((&s.u[q].x)[j]), acc[b][j], 0, 0, 0);
      }
    }
  };

  const int first = split ? w : 0, by = split ? kWaves : 1;
  if (first < steps) {
    Stage cur, nxt;
    int rows = rows_of(first);
    load(cur, rows);
    rows = rows_of(min(first + by, steps - 1));
    for (int step = first; step < steps; step += by) {
      load(nxt, rows);                      // (the last one reads the last step again)
      rows = rows_of(min(step + 2 * by, steps - 1));
      compute(cur, step);
      cur = nxt;
    }
  }

  // rank row k of the wave's columns
  float *const out = J.out + (int64_t)meta.slot * a.r_max * J.d + col;
  auto store = [&](int k, float (&x)[VEC]) __attribute__((always_inline)) {
    if (k >= r || !active) return;
    float *const p = out + (int64_t)k * J.d;
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
      float o[4] = {x[j] * meta.sc, x[j + 1] * meta.sc, x[j + 2] * meta.sc, x[j + 3] * meta.sc};
      if (a.accumulate) {
        float old[4];
        Elem<float>::unpack(ldg16(p + j), old);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += old[e];
      }
      stg16(p + j, Elem<float>::pack(o));
    }
  };
#pragma unroll
  for (int b = 0; b < RB; ++b) {
    if (b * 32 >= r) break;
    if (!split) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        float x[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = acc[b][j][v];
        store(b * 32 + acc_row(v, l), x);
      }
      continue;
    }
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
        const int v = w * 2 + i;
        float x[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          x[j] = part[0][v][j][l];
#pragma unroll
          for (int o = 1; o < kWaves; ++o) x[j] += part[o][v][j][l];
        }
        store(b * 32 + acc_row(half * 8 + v, l), x);
      }
    }
  }
}

template <typename T>
void launch_t(const GradArgs &a, dim3 grid, hipStream_t stream) {
  if (a.r_max <= 32)
    hipLaunchKernelGGL((adapter_grad_kernel<T, 1>), grid, dim3(kWaves * kWave), 0, stream, a);
  else
    hipLaunchKernelGGL((adapter_grad_kernel<T, 2>), grid, dim3(kWaves * kWave), 0, stream, a);
}

}  // namespace

hipError_t launch_adapter_grads(const void *X, int64_t ldx, const float *dH, float *dA,
                                const void *dY, int64_t lddy, const float *H, float *dBt,
                                const SegView &seg, const PoolView &pool, bool accumulate,
                                hipStream_t stream) {
  const int cols = 32 * (pool.dtype == LORA_BF16 ? Elem<bf16_t>::kVec : Elem<float>::kVec);
  GradArgs a{};
  int n = 0, blocks = 0;
  auto add = [&](const void *U, int64_t ldu, const float *V, float *out, int d) {
    if (!out) return;
    a.job[n++] = GradJob{U, ldu, V, out, d, (d + cols - 1) / cols};
    blocks += (d + cols - 1) / cols;
  };
  add(dY, lddy, H, dBt, pool.d_out);
  add(X, ldx, dH, dA, pool.d_in);
  if (n == 0) return hipSuccess;
  a.token_indices = seg.token_indices;
  a.seg_off = seg.seg_off;
  a.seg_slot = seg.seg_slot;
  a.seg_rank = seg.seg_rank;
  a.num_segments = seg.num_segments;
  a.seg_scale = seg.seg_scale;
  a.r_max = pool.r_max;
  a.accumulate = accumulate;
  const int S = seg.n_rows < pool.n_slots + 1 ? seg.n_rows : pool.n_slots + 1;
  const dim3 grid(blocks, S);
  if (pool.dtype == LORA_BF16) launch_t<bf16_t>(a, grid, stream);
  else launch_t<float>(a, grid, stream);
  return hipGetLastError();
}

}  // namespace lora
