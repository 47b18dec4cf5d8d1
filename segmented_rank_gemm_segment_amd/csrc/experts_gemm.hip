// The experts' products on bf16 weights, and their gradients: for every expert e with
// sorted rows p in [off[e], off[e + 1]),
//
//   kForward  Y[p]  = X[row(p)] W_e^T                  sums over d_in
//   kRows     dX[p] = dY[p] W_e                        sums over d_out
//   kWeights  dW_e (+)= sum_p dY[p]^T X[row(p)]        sums over the expert's rows
//
// all as out[m][n] = sum_k P[m][k] Q[n][k] on BM x BN tiles, K in stages of 64 in two
// LDS buffers filled by direct global -> LDS loads.  An operand whose memory runs
// along K is staged as rows of 128 bytes and read 16 bytes (8 of K) a lane; one whose
// memory runs along m or n (W in kRows, both in kWeights) is staged as 64 rows, one
// for each k, and read through the LDS transpose read, which hands 16 lanes 4 k of
// their own columns each.  Both orders give a lane the same 8 k, so they combine.
// 16-byte chunks are XOR-swizzled by the row so that neither read has bank conflicts.
//
// Workgroups are persistent and each XCD walks its own part of the tiles: the loads
// of a tile's first stages go out under the products of the one before.
#include <type_traits>

#include "lds_dma.cuh"
#include "lora_device.cuh"
#include "lora_kernels.h"
#include "mx_common.cuh"
#include "tile_choice.h"

namespace lora {
namespace {

enum Form { kForward = 0, kRows = 1, kWeights = 2 };

struct ExpertGemmArgs {
  const bf16_t *P;
  int64_t ldp;
  const bf16_t *Q;
  int64_t ldq;
  void *out;
  int64_t ldo;
  int M, N, K;              // kWeights: M; the others: K; rows or K are the experts'
  int n_choices, top_k, n_experts;
  const int32_t *off;
  const int32_t *sorted;    // X rows through sorted_choice / top_k, or null
  int64_t w_stride;         // elements from an expert's weight to the next one's
  int accumulate;           // kWeights
  uint32_t div_m;           // choice / top_k = umulhi(choice, div_m) >> div_s, top_k > 1
  int div_s;
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ mfma_bf16x8 read_transposed(const unsigned char *p, int second) {
  typedef __attribute__((address_space(3))) s16x4 *lds_t;
  const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p)));
  const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t)(p + second)));
  return as_bf16x8(u32x4{a.x, a.y, b.x, b.y});
}

// One operand of a tile: B rows of m or n, ALONG_K or not; I load instructions a wave.
template <int B, bool ALONG_K, int NW>
struct Operand {
  static constexpr int BYTES = B * 128, I = BYTES / 1024 / NW;
  static constexpr int RB = ALONG_K ? 128 : B * 2;          // bytes of an LDS row
  static constexpr int LPR = RB / 16, RPI = 64 / LPR;       // lanes a row, rows a load
  static_assert(BYTES % (1024 * NW) == 0, "loads");
  // what a row's chunks are XORed with.  Along K: 16 consecutive rows at one chunk in 16
  // bank groups.  Else: a half wave's transpose read takes 32 bytes of four rows twice.
  __device__ static __forceinline__ int swz(int row) {
    return ALONG_K ? (row >> 1) & 7 : B >= 128 ? (row & 3) * 4 : ((row >> 1) & 1) * 4;
  }
  __device__ static __forceinline__ int row(int wid, int i, int l) { return (wid * I + i) * RPI + l / LPR; }
  // elements from the start of its row's memory that the lane loads
  __device__ static __forceinline__ int chunk(int wid, int i, int l) {
    return ((l % LPR) ^ swz(row(wid, i, l))) * 8;
  }
  // Where lane l reads in a stage: of W waves, wave w's fragment i holds rows or columns
  // 32 (w F + i) and on of the operand, its sub-step kk 16 k.  Along K sub-steps are two
  // XORed chunks; else a fragment's columns are XORed and sub-steps are 16 rows apart.
  template <int W> struct Reader {
    static constexpr int F = B / 32 / W;
    static constexpr int ROWS = ALONG_K ? 1 : F, SUBS = ALONG_K ? 4 : 1;
    int at[ROWS], sub[SUBS];
    __device__ __forceinline__ void init(int w, int l) {
      if constexpr (ALONG_K) {
        at[0] = (w * F * 32 + (l & 31)) * RB;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) sub[kk] = ((kk * 2 + (l >> 5)) ^ swz(l & 31)) * 16;
      } else {
        const int t = l & 15, k = (l >> 5) * 8 + (t >> 2);
#pragma unroll
        for (int i = 0; i < F; ++i)
          at[i] = k * RB + (((w * F + i) * 4 + ((l >> 4) & 1) * 2 + ((t & 3) >> 1)) ^ swz(k)) * 16 + (t & 1) * 8;
      }
    }
    __device__ __forceinline__ mfma_bf16x8 read(const unsigned char *st, int i, int kk) const {
      if constexpr (ALONG_K)
        return as_bf16x8(*reinterpret_cast<const u32x4 *>(st + at[0] + sub[kk] + i * 32 * RB));
      else
        return read_transposed(st + at[i] + kk * 16 * RB, 4 * RB);
    }
  };
};

// TAIL: K is no multiple of 64 (kWeights: always).
template <int FORM, int BM, int BN, int WM, int WN, int PER_CU, bool TAIL, bool F32OUT>
__global__ __launch_bounds__(WM *WN *kWave, WM *WN *PER_CU / 4) void experts_gemm_kernel(ExpertGemmArgs g) {
  constexpr int NW = WM * WN, T = NW * kWave;
  constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  using OP = Operand<BM, FORM != kWeights, NW>;
  using OQ = Operand<BN, FORM == kForward, NW>;
  constexpr int STAGE = OP::BYTES + OQ::BYTES;
  constexpr int TAB = (4 * (LORA_MAX_EXPERTS + 1) + 15) / 16 * 16;
  constexpr int SMEM = 2 * STAGE + TAB + NW * 2048;
  static_assert(SMEM * PER_CU <= 160 * 1024, "LDS");
  static_assert(FORM == kWeights || !F32OUT, "rows are bf16");
  __shared__ __align__(16) unsigned char smem[SMEM];
  int *const tab = reinterpret_cast<int *>(smem + 2 * STAGE);

  const int tid = threadIdx.x, l = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int E = g.n_experts, N = g.N;
  const int tiles_n = (N + BN - 1) / BN;

  // tab[e]: M-tiles (kWeights: stages, two more for a tile's own cost) of the experts
  // before e, tab[E] of all
  {
    const int ept = (E + T - 1) / T, e0 = tid * ept, e1 = min(E, e0 + ept);
    auto count = [&](int e) __attribute__((always_inline)) {
      const int rows = g.off[e + 1] - g.off[e];
      return FORM == kWeights ? (rows + 63) / 64 + 2 : (rows + BM - 1) / BM;
    };
    int n = 0;
    for (int e = e0; e < e1; ++e) n += count(e);
    int *const s = reinterpret_cast<int *>(smem);
    int inc = n;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(inc, o);
      inc += l >= o ? v : 0;
    }
    if (l == kWave - 1) s[wid] = inc;
    __syncthreads();
    int at = inc - n;
    for (int w = 0; w < wid; ++w) at += s[w];
    for (int e = e0; e < e1; ++e) {
      tab[e] = at;
      at += count(e);
    }
    if (e0 < E && e1 == E) tab[E] = at;
    __syncthreads();
  }
  // the last expert whose entry is at most v
  auto find = [&](int v) __attribute__((always_inline)) {
    int lo = 0, hi = E;                             // tab[lo] <= v < tab[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__builtin_amdgcn_readfirstlane(tab[mid]) <= v)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };

  // This XCD's tiles: an eighth of the order (kWeights: of its cost; an expert's tiles
  // cost alike).
  const int xcd = blockIdx.x & 7, stride = gridDim.x / 8;
  const int all = __builtin_amdgcn_readfirstlane(tab[E]);
  const int tiles_w = FORM == kWeights ? (g.M + BM - 1) / BM * tiles_n : 0;   // an expert's
  auto begin_of = [&](int x) __attribute__((always_inline)) -> int {
    if constexpr (FORM != kWeights) {
      const int tiles = all * tiles_n;
      return min(tiles, x * ((tiles + 7) / 8));
    } else {
      if (x == 8) return E * tiles_w;
      const int64_t at = (int64_t)all * x / 8;
      const int e = find((int)at);
      const int c0 = __builtin_amdgcn_readfirstlane(tab[e]), c1 = __builtin_amdgcn_readfirstlane(tab[e + 1]);
      return e * tiles_w + (int)((at - c0) * tiles_w / (c1 - c0));
    }
  };
  const int t_end = __builtin_amdgcn_readfirstlane(begin_of(xcd + 1));
  int t = __builtin_amdgcn_readfirstlane(begin_of(xcd)) + blockIdx.x / 8;
  if (t >= t_end) return;

  struct Tile {
    int m0, n0, e, r0, r1;                          // r0, r1: the expert's rows
    int m_end, k_end, stages;
  };
  // (wave-uniform: scalar registers)
  auto uniform = [](int v) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(v); };
  auto tile_of = [&](int t) __attribute__((always_inline)) {
    Tile x;
    int mi, ni;
    if constexpr (FORM == kWeights) {
      x.e = uniform(t / tiles_w);
      tile_at(t - x.e * tiles_w, tiles_w / tiles_n, tiles_n, mi, ni);
    } else {
      x.e = find(uniform(t / tiles_n));
      const int first = uniform(tab[x.e]);
      tile_at(t - first * tiles_n, uniform(tab[x.e + 1]) - first, tiles_n, mi, ni);
    }
    mi = uniform(mi);
    x.r0 = uniform(g.off[x.e]);
    x.r1 = uniform(g.off[x.e + 1]);
    x.n0 = uniform(ni) * BN;
    if constexpr (FORM == kWeights) {
      x.m0 = mi * BM;
      x.m_end = g.M;
      x.k_end = x.r1 - x.r0;
      x.stages = max(1, (x.k_end + 63) / 64);       // (no rows: a stage of zeros)
    } else {
      x.m0 = x.r0 + mi * BM;
      x.m_end = x.r1;
      x.k_end = g.K;
      x.stages = (g.K + 63) / 64;
    }
    return x;
  };

  // This wave's loads: 32-bit byte offsets of the lanes from a scalar base (leading
  // dimensions are below 2^22), but for rows that lie anywhere.  Whatever lies past an
  // end is read from a valid place instead: rows and columns past it are not stored, k
  // past it are zeroed in LDS before use.
  const uint32_t sbase = lds_offset(smem);
  const uint32_t p_dst = __builtin_amdgcn_readfirstlane(sbase + wid * OP::I * 1024);
  const uint32_t q_dst = __builtin_amdgcn_readfirstlane(sbase + OP::BYTES + wid * OQ::I * 1024);
  const bool gathered = g.sorted != nullptr;
  auto token_of = [&](int choice) __attribute__((always_inline)) {
    return g.top_k == 1 ? choice : (int)(__umulhi((uint32_t)choice, g.div_m) >> g.div_s);
  };
  Tile li;                                          // the tile being loaded
  int k_i = 0, b_i = 0, t_i = t;                    // its next stage, the buffer for it
  // at the next stage, and how much further the one after is
  const unsigned char *pbase = nullptr, *qbase = nullptr;
  const int64_t pstep = FORM == kWeights ? 128 * g.ldp : 128;
  const int64_t qstep = FORM == kForward ? 128 : FORM == kRows ? 128 * g.ldq : 0;
  auto scalar = [](const bf16_t *p) __attribute__((always_inline)) {
    const uint64_t v = (uint64_t)p;
    return reinterpret_cast<const unsigned char *>(
        ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
        (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
  };
  const unsigned char *prow[FORM == kForward ? OP::I : 1];
  uint32_t poff[FORM == kForward ? 1 : OP::I], qoff[FORM == kWeights ? 1 : OQ::I];
  int qrow[FORM == kWeights ? OQ::I : 1];           // the next stage's rows, or their choices
  auto fetch_rows = [&]() __attribute__((always_inline)) {
    if constexpr (FORM == kWeights)
#pragma unroll
      for (int i = 0; i < OQ::I; ++i) {
        const int k = k_i * 64 + OQ::row(wid, i, l);
        qrow[i] = k >= li.k_end ? 0 : gathered ? g.sorted[li.r0 + k] : li.r0 + k;
      }
  };
  auto aim = [&](int t) __attribute__((always_inline)) {
    li = tile_of(t);
    // (the lane by way of the asm: what depends on it alone would otherwise be computed
    // ahead of the loop and held in registers that the products need)
    int ln = l;
    asm volatile("" : "+v"(ln));
    const bf16_t *const w = g.Q + li.e * g.w_stride;
    if constexpr (FORM == kWeights) {
      // (an expert without rows reads the start of the output, which is there even where
      // a batch without tokens has no rows at all)
      const bf16_t *const o = static_cast<const bf16_t *>(g.out);
      pbase = scalar(li.k_end > 0 ? g.P + (int64_t)li.r0 * g.ldp + li.m0 : o);
      qbase = scalar(li.k_end > 0 ? g.Q + li.n0 : o);
    } else if constexpr (FORM == kRows) {
      pbase = scalar(g.P + (int64_t)li.m0 * g.ldp);
      qbase = scalar(w + li.n0);
    } else {
      qbase = scalar(w + (int64_t)li.n0 * g.ldq);
    }
#pragma unroll
    for (int i = 0; i < OP::I; ++i) {
      const int c = OP::chunk(wid, i, ln), r = OP::row(wid, i, ln);
      if constexpr (FORM == kWeights) {
        poff[i] = ((uint32_t)r * (uint32_t)g.ldp + (uint32_t)(li.m0 + c < g.M && li.k_end > 0 ? c : 0)) * 2u;
      } else if constexpr (FORM == kRows) {
        poff[i] = ((uint32_t)min(r, li.m_end - 1 - li.m0) * (uint32_t)g.ldp + (uint32_t)c) * 2u;
      } else {
        const int p = min(li.m0 + r, li.m_end - 1);
        prow[i] = reinterpret_cast<const unsigned char *>(g.P) + ((int64_t)(gathered ? token_of(g.sorted[p]) : p) * g.ldp + c) * 2;
      }
    }
    if constexpr (FORM != kWeights)
#pragma unroll
      for (int i = 0; i < OQ::I; ++i) {
        const int c = OQ::chunk(wid, i, ln), r = OQ::row(wid, i, ln);
        if constexpr (FORM == kForward)
          qoff[i] = ((uint32_t)min(r, N - 1 - li.n0) * (uint32_t)g.ldq + (uint32_t)c) * 2u;
        else
          qoff[i] = ((uint32_t)r * (uint32_t)g.ldq + (uint32_t)(li.n0 + c < N ? c : 0)) * 2u;
      }
    fetch_rows();
  };
  auto issue_p = [&](int i) __attribute__((always_inline)) {
    const uint32_t dst = __builtin_amdgcn_readfirstlane(p_dst + b_i * STAGE);
    const int k = k_i * 64 + (FORM == kWeights ? OP::row(wid, i, l) : OP::chunk(wid, i, l));
    const bool past = TAIL && k >= li.k_end;
    if constexpr (FORM == kForward) {
      dma16(dst, i * 1024, prow[i] + k_i * 128 - (past ? OP::chunk(wid, i, l) * 2 : 0));
    } else if constexpr (FORM == kRows) {
      dma16_s(dst, i * 1024, poff[i] - (past ? OP::chunk(wid, i, l) * 2u : 0u), pbase);
    } else {
      dma16_s(dst, i * 1024, poff[i] - (past ? (uint32_t)OP::row(wid, i, l) * (uint32_t)g.ldp * 2u : 0u),
              scalar(reinterpret_cast<const bf16_t *>(pbase)));
    }
  };
  auto issue_q = [&](int i) __attribute__((always_inline)) {
    const uint32_t dst = __builtin_amdgcn_readfirstlane(q_dst + b_i * STAGE);
    if constexpr (FORM == kForward) {
      const int c = OQ::chunk(wid, i, l);
      dma16_s(dst, i * 1024, qoff[i] - (TAIL && k_i * 64 + c >= li.k_end ? c * 2u : 0u),
              qbase);
    } else if constexpr (FORM == kRows) {
      const int r = OQ::row(wid, i, l);
      dma16_s(dst, i * 1024, qoff[i] - (TAIL && k_i * 64 + r >= li.k_end ? (uint32_t)r * (uint32_t)g.ldq * 2u : 0u),
              qbase);
    } else {
      const int c = OQ::chunk(wid, i, l);
      const int row = gathered ? token_of(qrow[i]) : qrow[i];
      dma16(dst, i * 1024, qbase + ((int64_t)row * g.ldq + (li.n0 + c < N && li.k_end > 0 ? c : 0)) * 2);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    b_i ^= 1;
    pbase += pstep;
    qbase += qstep;
    if (++k_i == li.stages) {
      k_i = 0;
      // past the last tile the loads go round on that one, unread
      if (t_i + stride < t_end) t_i += stride;
      aim(t_i);
    } else {
      fetch_rows();
    }
  };
  // stage k of tile x in buffer b: what this wave loaded past K to zero
  auto zero_tail = [&](const Tile &x, int k, int b) {
    const u32x4 z = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < OP::I; ++i) {
      const int at = k * 64 + (FORM == kWeights ? OP::row(wid, i, l) : OP::chunk(wid, i, l));
      if (at >= x.k_end)
        *reinterpret_cast<u32x4 *>(smem + b * STAGE + (wid * OP::I + i) * 1024 + l * 16) = z;
    }
#pragma unroll
    for (int i = 0; i < OQ::I; ++i) {
      const int at = k * 64 + (FORM == kForward ? OQ::chunk(wid, i, l) : OQ::row(wid, i, l));
      if (at >= x.k_end)
        *reinterpret_cast<u32x4 *>(smem + b * STAGE + OP::BYTES + (wid * OQ::I + i) * 1024 + l * 16) = z;
    }
  };
  auto issue = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < OP::I; ++i) issue_p(i);
#pragma unroll
    for (int i = 0; i < OQ::I; ++i) issue_q(i);
    advance();
  };

  typename OP::template Reader<WM> pr;
  typename OQ::template Reader<WN> qr;
  pr.init(wm, l);
  qr.init(wn, l);

  f32x16 acc[FN][FM];
  mfma_bf16x8 pf[2][FM], qf[2][FN];
  auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
  };
  auto read = [&](int to, int q, const unsigned char *st, int kk) __attribute__((always_inline)) {
    if (q < FN)
      qf[to][q] = qr.read(st + OP::BYTES, q, kk);
    else
      pf[to][q - FN] = pr.read(st, q - FN, kk);
  };
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(acc[j][i]));
    if constexpr (FORM == kWeights)
#pragma unroll
      for (int i = 0; i < OQ::I; ++i) asm volatile("" : "+v"(qrow[i]));
  };

  aim(t);
  issue();
  Tile x = tile_of(t);                              // the tile being computed
  int b = 0;
  vm_wait<0>();                                     // the first stage has landed
  if (TAIL && x.k_end < 64) zero_tail(x, 0, 0);
  lgkm_barrier();
  issue();
#pragma unroll
  for (int q = 0; q < FM + FN; ++q) read(0, q, smem, 0);
  zero_acc();
  constexpr int NM = FM * FN, NR = FM + FN, NL = OP::I + OQ::I;
  // Sub-step kk's products with the reads of the next one's fragments from st, and the
  // loads of the next stage but one where LOAD.
  auto sub_step = [&](auto load, int kk, const unsigned char *st) __attribute__((always_inline)) {
    constexpr bool LOAD = decltype(load)::value;
    constexpr int STEPS = NM > NR ? (NM > NL || !LOAD ? NM : NL) : (NR > NL || !LOAD ? NR : NL);
#pragma unroll
    for (int q = 0; q < STEPS; ++q) {
      if (q < NM)
        acc[q / FM][q % FM] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            qf[kk & 1][q / FM], pf[kk & 1][q % FM], acc[q / FM][q % FM], 0, 0, 0);
      if (q < NR) read((kk + 1) & 1, q, st, (kk + 1) & 3);
      if constexpr (LOAD) {
        if (q < OP::I) issue_p(q);
        else if (q < NL) issue_q(q - OP::I);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int kt = 0;
  while (true) {
    const unsigned char *st = smem + b * STAGE;
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) sub_step(std::false_type{}, kk, st);
    const bool last = kt + 1 == x.stages;
    const Tile done = x;
    if (last && t + stride < t_end) x = tile_of(t + stride);
    kt = last ? 0 : kt + 1;                         // the next stage, of x
    pin();
    vm_wait<0>();                                   // it has landed
    if (TAIL && (kt + 1) * 64 > x.k_end) zero_tail(x, kt, b ^ 1);
    pin();
    lgkm_barrier();                                 // it is there, and this one has been read
    sub_step(std::true_type{}, 3, smem + (b ^ 1) * STAGE);
    pin();
    advance();
    b ^= 1;
    if (!last) continue;

    // Lane l has row l % 32 of a fragment and, of its 32 columns, [8 v + 4 (l / 32), +4) in
    // accumulator entries [4 v, 4 v + 4).  The fragments leave by way of 2 KB of LDS a
    // wave, 64 bytes of 32 rows at a time, so that four lanes write 64 bytes of a row
    // (16 bytes of a row a lane: 64 x 1024 rows, 2048 -> 1536 in 378 us where it is now
    // OUTUS; without any stores it would be 330).
    unsigned char *const out = smem + 2 * STAGE + TAB + wid * 2048;
    const int wr = (l & 31) * 64, ws = (l >> 2) & 3;          // the lane's row, its chunks' XOR
    const int rr = l >> 2, rc = ((l & 3) ^ (rr >> 2 & 3)) * 16;   // the row and chunk it stores
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const f32x16 c = acc[j][i];
        const int col0 = done.n0 + (wn * FN + j) * 32;
        const int row0 = done.m0 + (wm * FM + i) * 32;
        const int64_t at = FORM == kWeights ? done.e * g.w_stride : 0;
        if (!F32OUT && !(FORM == kWeights && g.accumulate)) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            // lower lanes' second quad against upper lanes' first: 8 columns each
            const uint32_t lo0 = pack_bf16x2(c[8 * p], c[8 * p + 1]), lo1 = pack_bf16x2(c[8 * p + 2], c[8 * p + 3]);
            const uint32_t hi0 = pack_bf16x2(c[8 * p + 4], c[8 * p + 5]), hi1 = pack_bf16x2(c[8 * p + 6], c[8 * p + 7]);
            const auto s0 = __builtin_amdgcn_permlane32_swap(lo0, hi0, false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(lo1, hi1, false, false);
            *reinterpret_cast<u32x4 *>(out + wr + (((p * 2 + (l >> 5)) ^ ws) * 16)) = u32x4{s0[0], s1[0], s0[1], s1[1]};
          }
          u32x4 o[2];
#pragma unroll
          for (int p = 0; p < 2; ++p)
            o[p] = *reinterpret_cast<const u32x4 *>(out + (rr + p * 16) * 64 + rc);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const int row = row0 + rr + p * 16, col = col0 + (l & 3) * 8;
            if (row < done.m_end && col < N)                  // N % 8 == 0: all 8 columns or none
              *reinterpret_cast<u32x4 *>(static_cast<bf16_t *>(g.out) + at + (int64_t)row * g.ldo + col) = o[p];
          }
        } else {
#pragma unroll
          for (int p = 0; p < 2; ++p) {                       // 16 columns in fp32
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const int a = 8 * p + 4 * v;
              *reinterpret_cast<f32x4 *>(out + wr + (((v * 2 + (l >> 5)) ^ ws) * 16)) = f32x4{c[a], c[a + 1], c[a + 2], c[a + 3]};
            }
            f32x4 o[2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
              o[q] = *reinterpret_cast<const f32x4 *>(out + (rr + q * 16) * 64 + rc);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int row = row0 + rr + q * 16, col = col0 + p * 16 + (l & 3) * 4;
              if (row >= done.m_end || col >= N) continue;
              if constexpr (F32OUT) {
                f32x4 *const y = reinterpret_cast<f32x4 *>(static_cast<float *>(g.out) + at + (int64_t)row * g.ldo + col);
                if (g.accumulate) o[q] += *y;
                *y = o[q];
              } else {
                uint2 *const y = reinterpret_cast<uint2 *>(static_cast<bf16_t *>(g.out) + at + (int64_t)row * g.ldo + col);
                const uint2 old = *y;
                *y = make_uint2(pack_bf16x2(o[q][0] + bf16_lo(old.x), o[q][1] + bf16_hi(old.x)),
                                pack_bf16x2(o[q][2] + bf16_lo(old.y), o[q][3] + bf16_hi(old.y)));
              }
            }
          }
        }
      }
    }
    t += stride;
    if (t >= t_end) break;
    zero_acc();
    pin();                                          // (zeros in these registers: 81 were spilled without)
  }
  vm_wait<0>();                                     // no load outlives the workgroup's LDS
}

template <int FORM, int BM, int BN, int WM, int WN, int PER_CU, bool F32OUT>
void launch_tiles(const ExpertGemmArgs &g, hipStream_t stream) {
  const dim3 grid(kCUs * PER_CU), block(WM * WN * kWave);
  if constexpr (FORM != kWeights) {
    if (g.K % 64 == 0) {
      hipLaunchKernelGGL((experts_gemm_kernel<FORM, BM, BN, WM, WN, PER_CU, false, F32OUT>), grid, block, 0,
                         stream, g);
      return;
    }
  }
  hipLaunchKernelGGL((experts_gemm_kernel<FORM, BM, BN, WM, WN, PER_CU, true, F32OUT>), grid, block, 0,
                     stream, g);
}

ExpertGemmArgs args_of(const void *P, int64_t ldp, const void *Q, int64_t ldq, void *out, int64_t ldo,
                       int M, int N, int K, const ExpertView &ex) {
  ExpertGemmArgs g{static_cast<const bf16_t *>(P), ldp, static_cast<const bf16_t *>(Q), ldq, out, ldo,
                   M, N, K, ex.n_choices, ex.top_k, ex.n_experts, ex.off, ex.sorted_choice,
                   ex.w_stride, 0, 0, 0};
  // 2^s < top_k <= 2^(s + 1): div_m = ceil(2^(32 + s) / top_k) is off by less than top_k,
  // which a choice (below 2^30) takes to less than 2^(31 + s): below one in the quotient
  int s = 0;
  while (2 << s < ex.top_k) ++s;
  g.div_s = s;
  if (ex.top_k > 1) g.div_m = (uint32_t)(((1ull << (32 + s)) + ex.top_k - 1) / ex.top_k);
  return g;
}

// Mean rows of an expert from which the 256 x 256 tiles are taken.
constexpr int kLargeRows = 64;

}  // namespace

hipError_t launch_experts_gemm(const void *X, int64_t ldx, const ExpertView &ex, const void *W,
                               int64_t ldw, void *Y, int64_t ldy, int K, int N, hipStream_t stream) {
  const ExpertGemmArgs g = args_of(X, ldx, W, ldw, Y, ldy, 0, N, K, ex);
  if (ex.n_choices / ex.n_experts < kLargeRows)
    launch_tiles<kForward, 32, 128, 1, 4, 3, false>(g, stream);
  else
    launch_tiles<kForward, 256, 256, 2, 4, 1, false>(g, stream);
  return hipGetLastError();
}

hipError_t launch_experts_gemm_rows(const void *dY, int64_t lddy, const ExpertView &ex,
                                    const void *W, int64_t ldw, void *dX, int64_t lddx, int K,
                                    int N, hipStream_t stream) {
  const ExpertGemmArgs g = args_of(dY, lddy, W, ldw, dX, lddx, 0, N, K, ex);
  if (ex.n_choices / ex.n_experts < kLargeRows)
    launch_tiles<kRows, 32, 128, 1, 4, 3, false>(g, stream);
  else
    launch_tiles<kRows, 256, 256, 2, 4, 1, false>(g, stream);
  return hipGetLastError();
}

hipError_t launch_experts_gemm_weights(const void *dY, int64_t lddy, const void *X, int64_t ldx,
                                       const ExpertView &ex, void *dW, int64_t lddw, int dtype,
                                       bool accumulate, int M, int N, hipStream_t stream) {
  ExpertGemmArgs g = args_of(dY, lddy, X, ldx, dW, lddw, M, N, 0, ex);
  g.accumulate = accumulate;
  if (dtype == LORA_F32)
    launch_tiles<kWeights, 256, 256, 2, 4, 1, true>(g, stream);
  else
    launch_tiles<kWeights, 256, 256, 2, 4, 1, false>(g, stream);
  return hipGetLastError();
}

}  // namespace lora
