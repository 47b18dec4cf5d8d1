// Y = X dq(W)^T, bf16 X and an MXFP4 weight, large batches, and the experts'
// products of long segments: 256 x 256 tiles, bound by the bf16 matrix rate.
//
// The tile's W is a quarter of its X in bytes but has as many rows, so W's codes
// are loaded 256 of K at a time (rows of whole 128-byte cache lines; 128 at a time,
// 2048 x 8192 x 8192 took 221 us against 214) and its scales 512 where alignment
// allows, while X comes in stages of 64.  Three rings of two in LDS, all filled by direct
// global -> LDS loads.  A wave has 128 rows of X and 64 of W; per stage it reads
// each W block once, widens its 32 codes in four steps of 8 to bf16 under the
// block's scale (exact), and lane half h takes K positions [32 h, +32) of the stage
// of both operands.  Waits for all loads (a wave has one stage's in flight, and no
// wait depends on their order), one barrier per stage, loads spread over the
// products, persistent workgroups and stores from registers as in the product of
// two MXFP4 operands.
//
// 16943 x 4096 x 14336: 1.64 to 1.82 ms over the passes of a trace (the clock falls from
// one to the next, to 1.7 GHz; the matrix pipe is busy in 64% of the clocks), 1.1 to 1.2
// PFLOP/s, and 1.45 ms for 16384 rows in a graph, 1.33 PFLOP/s; 8192^3: 0.83 to 0.94 ms
// (a library's bf16 product reaches 1.36 and 1.17 PFLOP/s on these shapes).  8190 x 8
// choices on 64 experts of 2048 -> 1536: 389 to 413 us, 1.0 PFLOP/s.  On the first,
// when it took 1611 us, loads issued a quarter of a stage later took 1664, and three
// stages of X, loaded by the workgroup's halves in turn, 1644.
#pragma once

#include "gemm_tile.cuh"

namespace lora {
namespace {

// WIDE: a load of the scales takes four words a row (K 512).  TAIL: K is no
// multiple of 256.
template <bool GROUPED, bool WIDE, bool TAIL>
__global__ __launch_bounds__(512) void mx_weight_kernel(GemmArgs g) {
  constexpr int BM = 256, BN = 256, WN = 4, TM = 128, TN = 64, FM = 4, FN = 2;
  constexpr int XST = BM * 128, XN = 2;             // X: bytes of a stage, stages
  constexpr int WST = BN * 128, WNB = 2;            // W: bytes of 256 of K, pieces
  constexpr int SROW = WIDE ? 16 : 4, SST = BN * SROW, SNB = 2;
  constexpr int WOFF = XN * XST, SOFF = WOFF + WNB * WST, TOFF = SOFF + SNB * SST;
  constexpr int TAB = GROUPED ? 4 * (LORA_MAX_EXPERTS + 1) : 0;
  static_assert(TOFF + TAB <= 160 * 1024 && !(WIDE && TAIL), "LDS");
  __shared__ __align__(16) unsigned char smem[TOFF + TAB];

  const int tid = threadIdx.x, l = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wid / WN, wn = wid % WN, h = l >> 5;
  const int N = g.N, K = g.K;
  int *const first = reinterpret_cast<int *>(smem + TOFF);   // GROUPED: experts' first M-tiles
  int tiles_m = (g.M + BM - 1) / BM;
  if constexpr (GROUPED) {
    const ExpertTiles et = expert_tiles<BM, 512>(g.ex, reinterpret_cast<int *>(smem));
    tiles_m = et.total;
    const int E = g.ex.n_experts, ept = (E + 511) / 512;
    int at = et.first;
    for (int e = tid * ept; e < min(E, (tid + 1) * ept); ++e) {
      first[e] = at;
      at += (g.ex.off[e + 1] - g.ex.off[e] + BM - 1) / BM;
    }
    if (tid == 0) first[E] = tiles_m;
    __syncthreads();
  }
  const int tiles_n = (N + BN - 1) / BN, tiles = tiles_m * tiles_n;
  const int KT = (K + 63) / 64;

  // XCD x owns the x-th eighth of the tile order
  const int per = (tiles + 7) / 8, xcd = blockIdx.x & 7, stride = gridDim.x / 8;
  const int t_end = min(tiles, (xcd + 1) * per);
  int t = xcd * per + blockIdx.x / 8;
  if (t >= t_end) return;

  // M-tile mi: its rows [m0, m1) and its expert
  auto m_tile = [&](int mi, int &m0, int &m1, int &e) __attribute__((always_inline)) {
    m0 = mi * BM;
    m1 = g.M;
    e = 0;
    if constexpr (GROUPED) {
      int lo = 0, hi = g.ex.n_experts;              // first[lo] <= mi < first[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (__builtin_amdgcn_readfirstlane(first[mid]) <= mi)
          lo = mid;
        else
          hi = mid;
      }
      e = lo;
      const int o = __builtin_amdgcn_readfirstlane(g.ex.off[e]);
      m0 = o + (mi - __builtin_amdgcn_readfirstlane(first[e])) * BM;
      m1 = __builtin_amdgcn_readfirstlane(g.ex.off[e + 1]);
    }
  };

  // This wave's loads.  X: 4 a stage, codes: 4 a piece of four stages, 8 rows of
  // 128 bytes each.  Scales: 64 rows, waves w and w + 4 the same.
  const uint32_t sbase = lds_offset(smem);
  // Rows as 32-bit offsets from the tile's first (leading dimensions are below
  // 2^22 elements); the experts' X rows lie anywhere and take an address each.
  const unsigned char *xrow[GROUPED ? 4 : 1], *xbase = nullptr, *wbase = nullptr, *sbase_g = nullptr;
  uint32_t xoff[4], woff[4], soff;
  auto xchunk = [&](int i) { return (l & 7) ^ ((((wid * 4 + i) * 8 + l / 8) >> 1) & 7); };
  auto wchunk = [&](int i) { return (l & 7) ^ ((((wid * 4 + i) * 8 + l / 8) >> 1) & 7); };
  auto aim = [&](int tile) __attribute__((always_inline)) {
    int mi, ni, m0, m1, e;
    tile_at(tile, tiles_m, tiles_n, mi, ni);
    m_tile(mi, m0, m1, e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = min(m0 + (wid * 4 + i) * 8 + l / 8, m1 - 1);
      if constexpr (GROUPED) {
        const int row = g.ex.sorted_choice ? g.ex.sorted_choice[p] / g.ex.top_k : p;
        xrow[i] = reinterpret_cast<const unsigned char *>(g.X + (int64_t)row * g.ldx) + xchunk(i) * 16;
      } else {
        xoff[i] = (uint32_t)(p - m0) * (uint32_t)(g.ldx * 2) + xchunk(i) * 16;
      }
    }
    if constexpr (!GROUPED) xbase = reinterpret_cast<const unsigned char *>(g.X + (int64_t)m0 * g.ldx);
    const int n0 = ni * BN;
    const int64_t ldw = g.ldw / 2;                  // bytes
    wbase = reinterpret_cast<const unsigned char *>(g.W) + (GROUPED ? e * g.ex.w_stride : 0) + n0 * ldw;
    sbase_g = g.mx.w + (GROUPED ? e * g.ex.s_stride : 0) + n0 * g.mx.ldw;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      woff[i] = (uint32_t)(min((wid * 4 + i) * 8 + l / 8, N - 1 - n0) * (int)ldw) + wchunk(i) * 16;
    soff = (uint32_t)(min((wid & 3) * 64 + l, N - 1 - n0) * (int)g.mx.ldw);
  };
  // The next stage to issue: stage k_issue of tile t_issue; the buffers of its X,
  // its piece of codes and its scales.
  int k_issue = 0, xb = 0, wb = 0, sb_i = 0;
  int t_issue = t;
  constexpr int SPER = WIDE ? 8 : 2;                // stages per load of scales
  auto issue_x = [&](int i) __attribute__((always_inline)) {
    // a chunk past K reads the stage's first chunk and is zeroed before use
    const int c = xchunk(i);
    const int back = TAIL && k_issue * 64 + c * 8 >= K ? c * 16 : 0;
    const uint32_t dst = __builtin_amdgcn_readfirstlane(sbase + xb * XST + wid * 4 * 1024);
    if constexpr (GROUPED)
      dma16(dst, i * 1024, xrow[i] + (int64_t)k_issue * 128 - back);
    else
      dma16_s(dst, i * 1024, xoff[i] - back, xbase + (int64_t)k_issue * 128);
  };
  auto issue_w = [&](int i) __attribute__((always_inline)) {
    const int c = wchunk(i), p = k_issue / 4;
    const uint32_t back = TAIL && p * 256 + c * 32 >= K ? c * 16 : 0;
    dma16_s_unless(__builtin_amdgcn_readfirstlane(k_issue % 4),
                   __builtin_amdgcn_readfirstlane(sbase + wb * WST + wid * 4 * 1024), WOFF + i * 1024,
                   woff[i] - back, wbase + (int64_t)p * 128);
  };
  auto issue_s = [&]() __attribute__((always_inline)) {
    const uint32_t dst =
        __builtin_amdgcn_readfirstlane(sbase + sb_i * SST + (wid & 3) * 64 * SROW);
    const uint32_t skip = __builtin_amdgcn_readfirstlane(k_issue % SPER);
    if constexpr (WIDE)
      dma16_s_unless(skip, dst, SOFF, soff, sbase_g + (int64_t)(k_issue / 8) * 16);
    else
      dma4_s_unless(skip, dst, SOFF, soff, sbase_g + (int64_t)(k_issue / 2) * 4);
  };
  // past a stage's loads (its X, and with the first of their stages codes and scales)
  auto advance = [&]() __attribute__((always_inline)) {
    xb = xb + 1 == XN ? 0 : xb + 1;
    if (k_issue % SPER == 0) sb_i = sb_i + 1 == SNB ? 0 : sb_i + 1;
    if ((k_issue & 3) == 3 || k_issue + 1 == KT) wb = wb + 1 == WNB ? 0 : wb + 1;
    if (++k_issue == KT) {
      k_issue = 0;
      // past the last tile the rings go round on that one, unread
      if (t_issue + stride < t_end) aim(t_issue += stride);
    }
  };
  // X stage k in buffer b and, where they start with it, its piece of codes in
  // buffer w and its scales in s: what lies past K to zero, scales there to 1 (a
  // NaN would spoil the zeros)
  auto zero_tail = [&](int k, int b, int w, int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k * 64 + xchunk(i) * 8 >= K)
        *reinterpret_cast<u32x4 *>(smem + b * XST + (wid * 4 + i) * 1024 + l * 16) = u32x4{0, 0, 0, 0};
    if (k % 4 == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k * 64 + wchunk(i) * 32 >= K)
          *reinterpret_cast<u32x4 *>(smem + WOFF + w * WST + (wid * 4 + i) * 1024 + l * 16) = u32x4{0, 0, 0, 0};
    const int left = K / 32 - k * 2;                // blocks of the scale word inside K
    if (k % 2 == 0 && left < 4) {
      uint32_t *p = reinterpret_cast<uint32_t *>(smem + SOFF + s * SST + ((wid & 3) * 64 + l) * 4);
      const uint32_t keep = ~0u >> (32 - 8 * left);
      *p = (*p & keep) | (0x7f7f7f7fu & ~keep);
    }
  };

  aim(t);
  auto issue = [&]() __attribute__((always_inline)) {
    issue_s();
#pragma unroll
    for (int i = 0; i < 4; ++i) issue_w(i);
#pragma unroll
    for (int i = 0; i < 4; ++i) issue_x(i);
    advance();
  };
  issue();

  // fragment offsets
  const int xo = (wm * TM + (l & 31)) * 128, wo = WOFF + (wn * TN + (l & 31)) * 128;
  const int so = SOFF + (wn * TN + (l & 31)) * SROW;
  int xc[4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) xc[kk] = ((h * 4 + kk) ^ ((l >> 1) & 7)) * 16;

  f32x16 acc[FN][FM];
  u32x4 wq[FN], wr[FN];                             // the stage's blocks, the next stage's
  uint32_t sr[FN];
  float ws[FN];
  mfma_bf16x8 xf[2][FM], wf[2][FN];
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(acc[j][i]));
  };
  auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
  };
  auto read_x = [&](int to, int i, const unsigned char *st, int kk) __attribute__((always_inline)) {
    xf[to][i] = as_bf16x8(*reinterpret_cast<const u32x4 *>(st + xo + i * 32 * 128 + xc[kk]));
  };
  auto read_w = [&](int j, int k, int w, int s) __attribute__((always_inline)) {
    wr[j] = *reinterpret_cast<const u32x4 *>(smem + wo + w * WST + j * 32 * 128 + (((k & 3) * 2 + h) ^ ((l >> 1) & 7)) * 16);
    sr[j] = *reinterpret_cast<const uint32_t *>(smem + so + s * SST + j * 32 * SROW + (WIDE ? k / 2 % 4 * 4 : 0));
  };
  // block of this lane's half in a scale word at stage k
  auto take_w = [&](int k) __attribute__((always_inline)) {
    const int sh = ((k & 1) * 2 + h) * 8;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      wq[j] = wr[j];
      ws[j] = __uint_as_float((sr[j] >> sh & 0xffu) << 23);
    }
  };
  auto widen = [&](int to, int j, int kk) __attribute__((always_inline)) {
    wf[to][j] = fp4x8_to_bf16x8(wq[j][kk], ws[j]);
  };

  // consumer side of the rings: stage kt in X buffer cx; the next stage's piece
  // and scales in rw, rs
  int kt = 0, cx = 0, rw = 0, rs = 0;
  vm_wait<0>();                                     // the first stage has landed
  if (TAIL && KT <= 4) zero_tail(0, 0, 0, 0);
  lgkm_barrier();
  issue();
#pragma unroll
  for (int j = 0; j < FN; ++j) read_w(j, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < FM; ++i) read_x(0, i, smem, 0);
  take_w(0);
#pragma unroll
  for (int j = 0; j < FN; ++j) widen(0, j, 0);
  zero_acc();
  while (true) {
    const unsigned char *st = smem + cx * XST;
    const int nx = cx + 1 == XN ? 0 : cx + 1;
    const bool last = kt + 1 == KT;
    const int kn = last ? 0 : kt + 1;               // the next stage
    // its piece and scales: the following ones where it starts any
    const bool np = last || kn % 4 == 0, ns = last || kn % SPER == 0;
    rw = np ? (rw + 1 == WNB ? 0 : rw + 1) : rw;
    rs = ns ? (rs + 1 == SNB ? 0 : rs + 1) : rs;
#pragma unroll
    for (int kk = 0; kk < 3; ++kk)
#pragma unroll
      for (int q = 0; q < FN * FM; ++q) {
        acc[q / FM][q % FM] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            wf[kk & 1][q / FM], xf[kk & 1][q % FM], acc[q / FM][q % FM], 0, 0, 0);
        if (q < FM) read_x((kk + 1) & 1, q, st, kk + 1);
        if (q == 4 || q == 5) widen((kk + 1) & 1, q - 4, kk + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    pin();
    vm_wait<0>();                                   // the next stage has landed
    if (TAIL && kn >= KT - 4) zero_tail(kn, nx, rw, rs);
    lgkm_barrier();                                 // the next stage is there, this one has been read
#pragma unroll
    for (int j = 0; j < FN; ++j) read_w(j, kn, rw, rs);
    issue_s();
#pragma unroll
    for (int q = 0; q < FN * FM; ++q) {
      acc[q / FM][q % FM] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          wf[1][q / FM], xf[1][q % FM], acc[q / FM][q % FM], 0, 0, 0);
      if (q < FM) read_x(0, q, smem + nx * XST, 0);
      if (q & 1)
        issue_x(q / 2);
      else
        issue_w(q / 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    pin();
    advance();
    take_w(kn);
#pragma unroll
    for (int j = 0; j < FN; ++j) widen(0, j, 0);
    cx = nx;
    if (!last) {
      ++kt;
      continue;
    }
    kt = 0;
    // the tile's rows: lane l has row wm TM + 32 i + l % 32 and, of each 32
    // columns, [8 v + 4 (l / 32), +4) in accumulator entries [4 v, 4 v + 4)
    int mi, ni, m0, m1, e;
    tile_at(t, tiles_m, tiles_n, mi, ni);
    m_tile(mi, m0, m1, e);
    const int n0 = ni * BN + wn * TN + h * 8;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = m0 + wm * TM + i * 32 + (l & 31);
      bf16_t *y = g.Y + (int64_t)row * g.ldy;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const f32x16 c = acc[j][i];
          const uint32_t lo0 = pack_bf16x2(c[8 * p], c[8 * p + 1]), lo1 = pack_bf16x2(c[8 * p + 2], c[8 * p + 3]);
          const uint32_t hi0 = pack_bf16x2(c[8 * p + 4], c[8 * p + 5]), hi1 = pack_bf16x2(c[8 * p + 6], c[8 * p + 7]);
          // lower lanes' second quad against upper lanes' first: 8 columns each
          const auto s0 = __builtin_amdgcn_permlane32_swap(lo0, hi0, false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(lo1, hi1, false, false);
          const int col = n0 + j * 32 + p * 16;
          if (row < m1 && col < N)                  // N % 8 == 0: all 8 columns or none
            stg16(y + col, make_uint4(s0[0], s1[0], s0[1], s1[1]));
        }
    }
    t += stride;
    if (t >= t_end) break;
    zero_acc();
  }
  vm_wait<0>();                                     // no load outlives the workgroup's LDS
}

template <bool GROUPED>
hipError_t launch_mx_weight(const GemmArgs &g, hipStream_t stream) {
  const dim3 grid(kCUs), block(512);
  if (mx_wide_scales(g.K, g.mx.ldw))
    hipLaunchKernelGGL((mx_weight_kernel<GROUPED, true, false>), grid, block, 0, stream, g);
  else if (g.K % 256 == 0)
    hipLaunchKernelGGL((mx_weight_kernel<GROUPED, false, false>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((mx_weight_kernel<GROUPED, false, true>), grid, block, 0, stream, g);
  return hipGetLastError();
}

}  // namespace
}  // namespace lora
