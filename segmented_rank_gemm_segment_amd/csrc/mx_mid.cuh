// Products with an MXFP4 weight for batches between the streamed and the large
// ones (decode batches): tiles of 64 x 64, enough of them for every CU at a few
// hundred rows, or of 32 x 64 where those leave CUs idle and for the experts, under
// bf16 X (with the LoRA term) or MXFP4 X.
//
// A tile has little arithmetic for its bytes: at 256 x 4096 x 4096 each of the 256
// workgroups asks L2 for 0.67 MB (64 rows of X and of W) for 34 MFLOP, the matrix pipe
// is busy in under a quarter of the time, and the kernel is bound by loads and their
// latency.  K advances in stages of 512 bytes of X row (256 values) or
// 256 (512 codes): every load instruction covers whole 128-byte lines, and three
// stages fill the LDS (half of it with 32 rows: two workgroups share a CU).  Four
// K groups of two waves take a quarter of a stage each (a wave all of its rows and
// 32 columns), so a stage costs one barrier for 512 bytes of K (stages are loaded
// by waves 0-3 and 4-7 in turn, so a wave waits for all of its loads, one stage's,
// and no wait depends on the order in which they complete); their sums meet in
// LDS, where each thread then finishes 8 columns of one row with its LoRA term, in
// fp32, and one rounding.
//
// 256 x 4096 x 4096: 12.7 us on weights that stay in the caches behind L2, 15.1 to
// 17.6 from memory (16.6 on the tiles of the bf16 product, 12.9 here, when both were
// timed alike); with a rank-16 adapter a row 18.0 to 18.6 (22.8 against 18.9): 30 MB of
// B rows, 11 MB of them past L2; loading them ahead of the last stages, or of all,
// measured no faster.  Both operands MXFP4: 7.7 us; 333 x 8192 x 1024 8.5 us, from
// memory 9.8 to 10.0.  One row's B rows are read again by every row that shares its
// adapter: 400 x 4096 x 14336 takes 107 us with 128 adapters of rank 16 and 120 with 8
// of up to rank 64 that hold runs of rows.
#pragma once

#include "gemm_tile.cuh"

namespace lora {
namespace {

template <int BM, bool XMX, bool LORA, bool DORA, bool GROUPED = false>
__global__ __launch_bounds__(512) void mx_mid_kernel(GemmArgs g) {
  constexpr int BN = 64, KG = 4, NST = 3, FM = BM / 32;
  constexpr int KS = XMX ? 512 : 256;               // K of a stage
  constexpr int XR = XMX ? 256 : 512, WR = KS / 2;  // bytes of an X and a W row in it
  constexpr int XI = BM * XR / 1024 / 4, WI = BN * WR / 1024 / 4;   // an owner's loads
  constexpr int WPR = KS / 128;                     // scale words per row
  constexpr int SR = XMX ? BM + BN : BN;            // rows with scales (X rows first)
  constexpr int WOFF = BM * XR, SOFF = WOFF + BN * WR, STAGE = SOFF + SR * WPR * 4;
  constexpr int SL = SR * WPR / 64, SI = (SL + 3) / 4;   // scales: of a stage, of an owner
  constexpr int RS = BN + 4;
  static_assert(SR * WPR % 64 == 0 && 64 % WPR == 0, "scale loads");
  static_assert(NST == 3 && NST * STAGE <= 160 * 1024 && KG * BM * RS * 4 <= NST * STAGE, "LDS");
  __shared__ __align__(16) unsigned char smem[NST * STAGE];

  const int tid = threadIdx.x, l = tid & (kWave - 1), h = l >> 5;
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int kg = wid / 2, wn = wid % 2;
  const int grp = wid / 4, w4 = wid % 4;            // owner of the stages k with k % 2 == grp
  const int N = g.N, K = g.K;
  int M = g.M, tiles_m = (M + BM - 1) / BM, mi = 0, ni = 0;
  ExpertTiles et{};
  if constexpr (GROUPED) {
    et = expert_tiles<BM, 512>(g.ex, reinterpret_cast<int *>(smem));
    tiles_m = et.total;
  }
  if (!tile_order<GROUPED>(blockIdx.x, tiles_m, (N + BN - 1) / BN, -1, mi, ni)) return;
  int m0 = mi * BM;
  const int n0 = ni * BN;
  // the experts' product: rows [m0, M) are the tile's expert's, W its weight
  const unsigned char *W = reinterpret_cast<const unsigned char *>(g.W), *SW = g.mx.w;
  if constexpr (GROUPED) {
    int e;
    expert_of_tile<BM, 512>(g.ex, et, mi, reinterpret_cast<int *>(smem), e, m0, M);
    W += (int64_t)e * g.ex.w_stride;
    SW += (int64_t)e * g.ex.s_stride;
  }

  // row of this thread's outputs
  const int e_row = min(tid / 8, BM - 1), e_c8 = tid % 8 * 8;
  int e_seg = 0;
  if constexpr (LORA) e_seg = g.row_segment[min(m0 + e_row, M - 1)];

  // Loads, rows past the ends clamped to the last: 32-bit offsets from the
  // tile's first rows (leading dimensions are below 2^22 elements); the experts'
  // X rows lie anywhere and take an address each.
  const uint32_t sbase = lds_offset(smem);
  const int64_t ldxb = XMX ? g.ldx : g.ldx * 2, ldwb = g.ldw / 2;
  const unsigned char *const xb =
      reinterpret_cast<const unsigned char *>(g.X) + (GROUPED ? 0 : (int64_t)m0 * ldxb);
  const unsigned char *const wb = W + (int64_t)n0 * ldwb;
  constexpr int XCH = XR / 16, WCH = WR / 16;       // 16-byte chunks per row
  // physical chunk of logical chunk c in row r: 16 rows' reads of one chunk hit 16
  // bank groups
  auto xsw = [](int c, int r) { return c ^ (r & 15); };
  auto wsw = [](int c, int r) { return WCH >= 16 ? c ^ (r & 15) : c ^ ((r >> 1) & 7); };
  uint32_t xoff[XI], woff[WI];
  const unsigned char *xrow[GROUPED ? XI : 1];
  int xc[XI], wc[WI];                               // logical chunks
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int r = ((w4 * XI + i) * 64 + l) / XCH;
    xc[i] = xsw(l % XCH, r);
    if constexpr (GROUPED) {
      const int p = min(m0 + r, M - 1);
      xrow[i] = xb + (g.ex.sorted_choice ? g.ex.sorted_choice[p] / g.ex.top_k : p) * ldxb;
      xoff[i] = xc[i] * 16;
    } else {
      xoff[i] = (uint32_t)min(r, M - 1 - m0) * (uint32_t)ldxb + xc[i] * 16;
    }
  }
#pragma unroll
  for (int i = 0; i < WI; ++i) {
    const int r = ((w4 * WI + i) * 64 + l) / WCH;
    wc[i] = wsw(l % WCH, r);
    woff[i] = (uint32_t)min(r, N - 1 - n0) * (uint32_t)ldwb + wc[i] * 16;
  }
  // scales: load i has words [64 si(i), +64) of the stage's (where there are fewer
  // loads than owners, several owners load the same)
  auto si = [&](int i) { return SL < 4 ? w4 % SL : min(w4 * SI + i, SL - 1); };
  const int sword = l % WPR;
  const unsigned char *sp[SI];
#pragma unroll
  for (int i = 0; i < SI; ++i) {
    const int srow = (si(i) * 64 + l) / WPR;
    sp[i] = XMX && srow < BM ? g.mx.x + (int64_t)min(m0 + srow, M - 1) * g.mx.ldx
                             : SW + (int64_t)min(n0 + srow - (SR - BN), N - 1) * g.mx.ldw;
  }
  const int blocks = K / 32;
  constexpr int XE = XMX ? 32 : 8;                  // K of an X chunk
  auto issue = [&](int k, int buf) __attribute__((always_inline)) {
    // chunks past K read the stage's first chunk and are zeroed before use
    const uint32_t st = sbase + buf * STAGE;
    const int k0 = k * KS;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const uint32_t dst = __builtin_amdgcn_readfirstlane(st + w4 * XI * 1024);
      const uint32_t off = xoff[i] - (k0 + xc[i] * XE >= K ? xc[i] * 16 : 0);
      if constexpr (GROUPED)
        dma16(dst, i * 1024, xrow[i] + (int64_t)k * XR + off);
      else
        dma16_s(dst, i * 1024, off, xb + (int64_t)k * XR);
    }
#pragma unroll
    for (int i = 0; i < WI; ++i)
      dma16_s(__builtin_amdgcn_readfirstlane(st + w4 * WI * 1024), WOFF + i * 1024,
              woff[i] - (k0 + wc[i] * 32 >= K ? wc[i] * 16 : 0), wb + (int64_t)k * WR);
#pragma unroll
    for (int i = 0; i < SI; ++i)
      dma4(__builtin_amdgcn_readfirstlane(st + si(i) * 256), SOFF, sp[i] + min(k * WPR + sword, (blocks - 1) / 4) * 4);
  };
  const int KT = (K + KS - 1) / KS;
  auto zero_tail = [&](int buf) {
    unsigned char *st = smem + buf * STAGE;
    const int k0 = (KT - 1) * KS;
#pragma unroll
    for (int i = 0; i < XI; ++i)
      if (k0 + xc[i] * XE >= K)
        *reinterpret_cast<u32x4 *>(st + (w4 * XI + i) * 1024 + l * 16) = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < WI; ++i)
      if (k0 + wc[i] * 32 >= K)
        *reinterpret_cast<u32x4 *>(st + WOFF + (w4 * WI + i) * 1024 + l * 16) = u32x4{0, 0, 0, 0};
    // scales of blocks past K to 1: a NaN would spoil the zeros
    const int left = blocks - 4 * ((KT - 1) * WPR + sword);
    if (left < 4) {
      const uint32_t keep = left <= 0 ? 0u : ~0u >> (32 - 8 * left);
#pragma unroll
      for (int i = 0; i < SI; ++i) {
        uint32_t *p = reinterpret_cast<uint32_t *>(st + SOFF + si(i) * 256 + l * 4);
        *p = (*p & keep) | (0x7f7f7f7fu & ~keep);
      }
    }
  };
#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (s == grp && s < KT) issue(s, s);

  f32x16 acc[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[i][v] = 0.f;
  int e_r = 0, e_slot = 0;
  float e_sc = 0.f;
  const int wrow = wn * 32 + (l & 31);
  int buf = 0;
  auto land = [&](int kt) __attribute__((always_inline)) {
    const bool own = (kt & 1) == grp;
    if (own) {                                      // stage kt has landed
      vm_wait<0>();
      if (kt + 1 == KT && K % KS != 0) zero_tail(buf);
    }
    lgkm_barrier();                                 // it is there, stage kt - 1 has been read
    if (own && kt + NST - 1 < KT) issue(kt + NST - 1, buf == 0 ? NST - 1 : buf - 1);
  };
  auto multiply = [&]() __attribute__((always_inline)) {
    const unsigned char *st = smem + buf * STAGE;
    if constexpr (XMX) {
      u32x4 x[2][FM], w[2];
      uint32_t sx[FM];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int c = kg * 4 + s * 2 + h;
        w[s] = *reinterpret_cast<const u32x4 *>(st + WOFF + wrow * WR + wsw(c, wrow) * 16);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          x[s][i] = *reinterpret_cast<const u32x4 *>(st + (i * 32 + (l & 31)) * XR + xsw(c, l & 31) * 16);
      }
      const uint32_t sw = *reinterpret_cast<const uint32_t *>(st + SOFF + ((BM + wrow) * WPR + kg) * 4) >> (8 * h);
#pragma unroll
      for (int i = 0; i < FM; ++i)
        sx[i] = *reinterpret_cast<const uint32_t *>(st + SOFF + ((i * 32 + (l & 31)) * WPR + kg) * 4) >> (8 * h);
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[i] = mfma_mx<0>(x[0][i], w[0], acc[i], sx[i], sw);
#pragma unroll
      for (int i = 0; i < FM; ++i) acc[i] = mfma_mx<2>(x[1][i], w[1], acc[i], sx[i], sw);
    } else {
      const int cw = kg * 2 + h;                    // this half's block of 32 codes
      const u32x4 q = *reinterpret_cast<const u32x4 *>(st + WOFF + wrow * WR + wsw(cw, wrow) * 16);
      const uint32_t s = *reinterpret_cast<const uint32_t *>(st + SOFF + (wrow * WPR + kg / 2) * 4);
      const float sc = __uint_as_float((s >> (((kg & 1) * 2 + h) * 8) & 0xffu) << 23);
      mfma_bf16x8 x[4][FM];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < FM; ++i)
          x[kk][i] = as_bf16x8(*reinterpret_cast<const u32x4 *>(
              st + (i * 32 + (l & 31)) * XR + xsw(kg * 8 + h * 4 + kk, l & 31) * 16));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const mfma_bf16x8 w = fp4x8_to_bf16x8(q[kk], sc);
#pragma unroll
        for (int i = 0; i < FM; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[kk][i], w, acc[i], 0, 0, 0);
      }
    }
    buf = buf + 1 == NST ? 0 : buf + 1;
  };
  land(0);
  if constexpr (LORA) {
    e_r = g.seg_rank[e_seg];
    e_slot = g.seg_slot[e_seg];
    e_sc = g.seg_scale[e_seg];
  }
  for (int kt = 1; kt < KT; ++kt) {
    multiply();
    land(kt);
  }
  multiply();

  lgkm_barrier();                                   // the ring has been read
  float *red = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v)
      red[(kg * BM + i * 32 + acc_row(v, l)) * RS + wn * 32 + (l & 31)] = acc[i][v];
  lgkm_barrier();
  float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < KG; ++q) {
    const f32x4 p0 = *reinterpret_cast<const f32x4 *>(red + (q * BM + e_row) * RS + e_c8);
    const f32x4 p1 = *reinterpret_cast<const f32x4 *>(red + (q * BM + e_row) * RS + e_c8 + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o[e] += p0[e];
      o[4 + e] += p1[e];
    }
  }
  const int row = m0 + e_row, col = n0 + e_c8;
  if (tid / 8 < BM && row < M && col < N) {         // N % 8 == 0: all 8 columns or none
    if constexpr (LORA) {
      if (e_r > 0) lora_row8<DORA>(g, row, col, e_slot, e_r, e_sc, o);
    }
    stg16(g.Y + (int64_t)row * g.ldy + col, Elem<bf16_t>::pack(o));
  }
}

template <int BM, bool XMX>
hipError_t launch_mx_mid_rows(const GemmArgs &g, bool lora, hipStream_t stream) {
  const dim3 grid(tile_grid((g.M + BM - 1) / BM, (g.N + 63) / 64)), block(512);
  if constexpr (!XMX) {
    if (lora && g.dora) {
      hipLaunchKernelGGL((mx_mid_kernel<BM, false, true, true>), grid, block, 0, stream, g);
      return hipGetLastError();
    }
    if (lora) {
      hipLaunchKernelGGL((mx_mid_kernel<BM, false, true, false>), grid, block, 0, stream, g);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((mx_mid_kernel<BM, XMX, false, false>), grid, block, 0, stream, g);
  return hipGetLastError();
}
template <bool XMX>
hipError_t launch_mx_mid(const GemmArgs &g, MxKernel k, bool lora, hipStream_t stream) {
  return k == kMxTiles32 ? launch_mx_mid_rows<32, XMX>(g, lora, stream)
                         : launch_mx_mid_rows<64, XMX>(g, lora, stream);
}

inline hipError_t launch_experts_mid(const GemmArgs &g, int tiles_m, hipStream_t stream) {
  hipLaunchKernelGGL((mx_mid_kernel<32, false, false, false, true>),
                     dim3(expert_grid(tiles_m, (g.N + 63) / 64)), dim3(512), 0, stream, g);
  return hipGetLastError();
}

}  // namespace
}  // namespace lora
