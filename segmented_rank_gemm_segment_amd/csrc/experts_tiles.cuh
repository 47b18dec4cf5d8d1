// What the experts' products on bf16 weights share: out[m][n] = sum_k P[m][k] Q[n][k] on
// tiles of a persistent workgroup, operands staged in LDS by direct global -> LDS loads.
//
// An operand whose memory runs along K is staged as rows of 64 k, 128 bytes, and read 16
// bytes (8 of K) a lane; one whose memory runs along m or n is staged as one row for each
// k and read through the LDS transpose read, which hands 16 lanes 4 k of their own columns
// each.  Both give a lane the same 8 k, so they combine.  16-byte chunks are XOR-swizzled
// by the row: neither read has bank conflicts.
#pragma once

#include "lds_dma.cuh"
#include "lora_device.cuh"
#include "lora_kernels.h"
#include "mx_common.cuh"
#include "tile_choice.h"

namespace lora {
namespace {

struct ExpertGemmArgs {
  const bf16_t *P;
  int64_t ldp;
  const bf16_t *Q;
  int64_t ldq;
  void *out;
  int64_t ldo;
  int M, N, K;              // of M (rows) and K the one that is not an expert's rows
  int n_choices, top_k, n_experts;
  const int32_t *off;
  const int32_t *sorted;    // X rows through sorted_choice / top_k, or null
  int64_t w_stride;         // elements from an expert's weight to the next one's
  int accumulate;
  uint32_t div_m;           // choice / top_k = umulhi(2 choice, div_m) >> div_s
  int div_s;
};

// A choice's token.
__device__ __forceinline__ int token_of(const ExpertGemmArgs &g, int choice) {
  return (int)(__umulhi(2u * (uint32_t)choice, g.div_m) >> g.div_s);
}

inline ExpertGemmArgs expert_args(const void *P, int64_t ldp, const void *Q, int64_t ldq, void *out,
                                  int64_t ldo, int M, int N, int K, const ExpertView &ex) {
  ExpertGemmArgs g{static_cast<const bf16_t *>(P), ldp, static_cast<const bf16_t *>(Q), ldq, out, ldo,
                   M, N, K, ex.n_choices, ex.top_k, ex.n_experts, ex.off, ex.sorted_choice,
                   ex.w_stride, 0, 0, 0};
  // 2^(s - 1) < top_k <= 2^s, div_m = ceil(2^(31 + s) / top_k) < 2^32: a choice c, below
  // 2^30, gives c / top_k and less than 2^30 / 2^(31 + s) <= 1 / (2 top_k) more, which
  // reaches no further whole number
  int s = 0;
  while (1 << s < ex.top_k) ++s;
  g.div_s = s;
  g.div_m = (uint32_t)(((1ull << (31 + s)) + ex.top_k - 1) / ex.top_k);
  return g;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ mfma_bf16x8 read_transposed(const unsigned char *p, int second) {
  typedef __attribute__((address_space(3))) s16x4 *lds_t;
  const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p)));
  const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p + second)));
  return as_bf16x8(u32x4{a.x, a.y, b.x, b.y});
}

// What the chunks of an LDS row are XORed with.  Along K: 16 consecutive rows at one chunk
// in 16 bank groups.  Else (rows of B elements): a half wave's transpose read takes 32
// bytes of four rows twice.
template <int B, bool ALONG_K> __device__ __forceinline__ int chunk_xor(int row) {
  return ALONG_K ? (row >> 1) & 7 : B >= 128 ? (row & 3) * 4 : ((row >> 1) & 1) * 4;
}

// Where lane l reads in a stage of B rows or columns: of W waves, wave w's fragment i holds
// 32 (w F + i) and on, its sub-step kk 16 k.  Along K sub-steps are two XORed chunks; else
// a fragment's columns are XORed and sub-steps are 16 rows apart.
template <int B, bool ALONG_K, int W> struct FragmentReader {
  static constexpr int F = B / 32 / W, RB = ALONG_K ? 128 : B * 2;
  static constexpr int ROWS = ALONG_K ? 1 : F, SUBS = ALONG_K ? 4 : 1;
  int at[ROWS], sub[SUBS];
  __device__ __forceinline__ void init(int w, int l) {
    if constexpr (ALONG_K) {
      at[0] = (w * F * 32 + (l & 31)) * RB;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) sub[kk] = ((kk * 2 + (l >> 5)) ^ chunk_xor<B, true>(l & 31)) * 16;
    } else {
      const int t = l & 15, k = (l >> 5) * 8 + (t >> 2);
#pragma unroll
      for (int i = 0; i < F; ++i)
        at[i] = k * RB +
                (((w * F + i) * 4 + ((l >> 4) & 1) * 2 + ((t & 3) >> 1)) ^ chunk_xor<B, false>(k)) * 16 + (t & 1) * 8;
    }
  }
  __device__ __forceinline__ mfma_bf16x8 read(const unsigned char *st, int i, int kk) const {
    if constexpr (ALONG_K)
      return as_bf16x8(*reinterpret_cast<const u32x4 *>(st + at[0] + sub[kk] + i * 32 * RB));
    else
      return read_transposed(st + at[i] + kk * 16 * RB, 4 * RB);
  }
};

// tab[e] = the sum of count(e') over the experts before e, tab[n_experts] over all.
// Called by every thread; scratch: a word of LDS for every wave, free again on return.
constexpr int kExpertTab = (4 * (LORA_MAX_EXPERTS + 1) + 15) / 16 * 16;
template <int T, class Count>
__device__ __forceinline__ void expert_table(int E, int *tab, int *scratch, Count count) {
  const int tid = threadIdx.x, l = tid & (kWave - 1), wid = tid / kWave;
  const int ept = (E + T - 1) / T, e0 = tid * ept, e1 = min(E, e0 + ept);
  int n = 0;
  for (int e = e0; e < e1; ++e) n += count(e);
  int inc = n;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int v = __shfl_up(inc, o);
    inc += l >= o ? v : 0;
  }
  if (l == kWave - 1) scratch[wid] = inc;
  __syncthreads();
  int at = inc - n;
  for (int w = 0; w < wid; ++w) at += scratch[w];
  for (int e = e0; e < e1; ++e) {
    tab[e] = at;
    at += count(e);
  }
  if (e0 < E && e1 == E) tab[E] = at;
  __syncthreads();
}
// The last expert whose entry is at most v (below tab[E]).
__device__ __forceinline__ int expert_find(const int *tab, int E, int v) {
  int lo = 0, hi = E;                               // tab[lo] <= v < tab[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__builtin_amdgcn_readfirstlane(tab[mid]) <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// (wave-uniform values, in scalar registers)
__device__ __forceinline__ int scalar_int(int v) { return __builtin_amdgcn_readfirstlane(v); }
template <class T> __device__ __forceinline__ const unsigned char *scalar_ptr(const T *p) {
  const uint64_t v = (uint64_t)p;
  return reinterpret_cast<const unsigned char *>(((uint64_t)(uint32_t)scalar_int((int)(v >> 32)) << 32) |
                                                 (uint32_t)scalar_int((int)v));
}

// A 32 x 32 fragment's way out: lane l has row l % 32 and, of its columns, [8 v + 4 (l /
// 32), +4) in entries [4 v, 4 v + 4).  It goes by way of 2 KB of LDS, 64 bytes of each row
// at a time, so that four neighbouring lanes write 64 bytes of a row: out + row ldo + col
// for rows below `rows` and columns below `cols` (multiples of 8).  SUM: fp32 `out`, or
// sums of bf16 with what is there (`add`), formed in fp32.
template <bool F32OUT, bool SUM>
__device__ __forceinline__ void store_fragment(unsigned char *lds, const f32x16 &c, int l, void *out,
                                               int64_t ldo, int rows, int cols, bool add) {
  const int wr = (l & 31) * 64, ws = (l >> 2) & 3;              // the lane's row, its chunks' XOR
  const int rr = l >> 2, rc = ((l & 3) ^ (rr >> 2 & 3)) * 16;   // the row and chunk it stores
  if constexpr (!SUM) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      // lower lanes' second quad against upper lanes' first: 8 columns each
      const uint32_t lo0 = pack_bf16x2(c[8 * p], c[8 * p + 1]), lo1 = pack_bf16x2(c[8 * p + 2], c[8 * p + 3]);
      const uint32_t hi0 = pack_bf16x2(c[8 * p + 4], c[8 * p + 5]), hi1 = pack_bf16x2(c[8 * p + 6], c[8 * p + 7]);
      const auto s0 = __builtin_amdgcn_permlane32_swap(lo0, hi0, false, false);
      const auto s1 = __builtin_amdgcn_permlane32_swap(lo1, hi1, false, false);
      *reinterpret_cast<u32x4 *>(lds + wr + (((p * 2 + (l >> 5)) ^ ws) * 16)) = u32x4{s0[0], s1[0], s0[1], s1[1]};
    }
    u32x4 o[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) o[p] = *reinterpret_cast<const u32x4 *>(lds + (rr + p * 16) * 64 + rc);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int row = rr + p * 16, col = (l & 3) * 8;
      if (row < rows && col < cols)
        *reinterpret_cast<u32x4 *>(static_cast<bf16_t *>(out) + row * ldo + col) = o[p];
    }
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p) {                               // 16 columns in fp32
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int a = 8 * p + 4 * v;
        *reinterpret_cast<f32x4 *>(lds + wr + (((v * 2 + (l >> 5)) ^ ws) * 16)) = f32x4{c[a], c[a + 1], c[a + 2], c[a + 3]};
      }
      f32x4 o[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) o[q] = *reinterpret_cast<const f32x4 *>(lds + (rr + q * 16) * 64 + rc);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int row = rr + q * 16, col = p * 16 + (l & 3) * 4;
        if (row >= rows || col >= cols) continue;
        if constexpr (F32OUT) {
          f32x4 *const y = reinterpret_cast<f32x4 *>(static_cast<float *>(out) + row * ldo + col);
          if (add) o[q] += *y;
          *y = o[q];
        } else {
          uint2 *const y = reinterpret_cast<uint2 *>(static_cast<bf16_t *>(out) + row * ldo + col);
          const uint2 old = *y;
          *y = make_uint2(pack_bf16x2(o[q][0] + bf16_lo(old.x), o[q][1] + bf16_hi(old.x)),
                          pack_bf16x2(o[q][2] + bf16_lo(old.y), o[q][3] + bf16_hi(old.y)));
        }
      }
    }
  }
}

}  // namespace
}  // namespace lora
