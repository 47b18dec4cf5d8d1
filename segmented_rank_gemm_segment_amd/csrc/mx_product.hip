// Y = dq(Xq) dq(Wq)^T, both operands MXFP4, large batches: codes and scales go
// to v_mfma_scale_f32_32x32x64_f8f6f4 as they are.
//
// At 8.6 PFLOP/s (the rate of a loop of these MFMAs on registers alone) a
// 256 x 256 tile takes 2.4 thousand cycles for 256 codes of K and needs 68 KB of
// operands for them, so the kernel lives from keeping the loads ahead:
// * two buffers of 256 codes of K, whose row pieces are whole 128-byte cache lines
//   (64-byte pieces and four buffers: 609 us against 523), filled by direct
//   global -> LDS loads, 16-byte chunks XOR-swizzled so 16 lanes' reads hit 16 bank
//   groups; the scales go into buffers of their own, four words a row at once
//   where alignment allows (with a word a row they cost as many cache lookups as
//   the codes);
// * a wave waits for all of its loads (vmcnt(0)) and then issues the next stage's,
//   so it never has more than one stage in flight and no wait depends on the order
//   in which loads complete.  One barrier per stage publishes the next stage and
//   frees this one's buffer, three quarters into its products, so the loads have
//   three quarters of a stage's products to land in;
// * one load to a product: issued together behind the barrier they fill the load
//   queue and hold the products up;
// * workgroups are persistent, one per CU, and the ring runs on from one tile
//   into the next: the next tile's first stages are on their way while this
//   tile's last products and its stores run.
// W is the MFMA's row operand and X its column operand, so a lane ends up with
// one row of Y and runs of columns; two lanes swap halves (v_permlane32_swap)
// and each stores 16 bytes, without LDS, which the ring keeps.
// 16943 x 4096 x 14336: 490 to 530 us, 3.8 to 4.1 PFLOP/s; 8192^3: 264 to 270 us, 4.1 PFLOP/s;
// 2048 x 8192 x 8192: 70 us.  Of the first's clocks (1.75 to 1.87 GHz under this load) the matrix
// pipe is busy in 52%, LDS with the fragments' reads in 29%, a sixth of it bank
// conflicts; 0.91 GB comes from past L2, 1.8 TB/s.  With loads and stores left out the
// products take 283 us, the stores alone 100: no one of these fills the time, and the
// counters do not show what the rest waits for.
#include "lora_device.cuh"
#include "lora_kernels.h"
#include "mx_common.cuh"
#include "tile_choice.h"

namespace lora {
namespace {

struct MxGemmArgs {
  const unsigned char *X, *SX, *W, *SW;   // codes and scales
  int64_t ldx, ldsx, ldw, ldsw;           // bytes a row
  bf16_t *Y;
  int64_t ldy;
  int M, K, N;
};

// WIDE: a load of the scales takes four words a row and serves two stages.
template <int BM, int BN, int WM, int WN, bool WIDE>
__global__ __launch_bounds__(WM *WN *kWave) void mx_product_kernel(MxGemmArgs g) {
  constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  constexpr int R = BM + BN, RW = R / NW, STAGE = R * 128;   // RW: rows that a wave loads
  constexpr int CI = RW / 8;                        // its loads of codes in a stage
  // scales: WIDE rows of four words, for two stages; otherwise one word of every
  // row after the other
  constexpr int SPER = WIDE ? 2 : 1, SSTAGE = WIDE ? R * 16 : R * 8;
  constexpr int SOFF = 2 * STAGE;
  static_assert(RW == kWave && BM % RW == 0 && CI == FM * FN, "a load to a product");
  static_assert(SOFF + 2 * SSTAGE <= 160 * 1024, "LDS");
  __shared__ __align__(16) unsigned char smem[SOFF + 2 * SSTAGE];

  const int tid = threadIdx.x, l = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  const int KT = (g.K + 255) / 256, last_word = (g.K / 32 - 1) / 4;
  const bool ktail = g.K % 256 != 0;

  // XCD x (workgroups x, x + 8, ...) owns the x-th eighth of the tile order and
  // its workgroups take that in turn.
  const int per = (tiles + 7) / 8, xcd = blockIdx.x & 7, stride = gridDim.x / 8;
  const int t_end = min(tiles, (xcd + 1) * per);
  int t_issue = xcd * per + blockIdx.x / 8;
  if (t_issue >= t_end) return;

  // This wave's loads: rows [RW wid, +RW) of X's and W's.  Load i has rows 8 i + l / 8
  // of them at physical chunk l % 8, logical chunk `chunk(i)`; rows past the end
  // read the last one.
  const uint32_t sbase = lds_offset(smem);
  constexpr int XW = BM / RW;                       // waves of X
  const bool isx = wid < XW;
  const int wrow0 = (isx ? wid : wid - XW) * RW;
  const unsigned char *const op = isx ? g.X : g.W, *const sop = isx ? g.SX : g.SW;
  const int64_t ldo = isx ? g.ldx : g.ldw, ldso = isx ? g.ldsx : g.ldsw;
  auto chunk = [&](int i) { return (l & 7) ^ ((i & 1) * 4 + l / 16); };
  const unsigned char *base = nullptr, *bases = nullptr;
  uint32_t off[CI], offs;
  auto aim = [&](int t) __attribute__((always_inline)) {
    int mi, ni;
    tile_at(t, tiles_m, tiles_n, mi, ni);
    const int first = isx ? mi * BM : ni * BN;
    base = op + (int64_t)first * ldo;
    bases = sop + (int64_t)first * ldso;
    const int last = (isx ? g.M : g.N) - 1 - first;
#pragma unroll
    for (int i = 0; i < CI; ++i)
      off[i] = (uint32_t)min(wrow0 + i * 8 + l / 8, last) * (uint32_t)ldo + chunk(i) * 16;
    offs = (uint32_t)min(wrow0 + l, last) * (uint32_t)ldso;
  };
  // The next stage to issue: stage k_issue of tile t_issue, into buffer b_issue,
  // its scales into buffer s_issue where a load of them is due.
  int k_issue = 0, b_issue = 0, s_issue = 0;
  auto issue_codes = [&](int i) __attribute__((always_inline)) {
    // a chunk past K reads the stage's first chunk (in bounds: it starts
    // before K) and is zeroed before use
    const uint32_t back =
        !WIDE && ktail && k_issue == KT - 1 && k_issue * 256 + chunk(i) * 32 >= g.K ? chunk(i) * 16 : 0;
    dma16_s(__builtin_amdgcn_readfirstlane(sbase + b_issue * STAGE + wid * CI * 1024), i * 1024, off[i] - back,
            base + (int64_t)k_issue * 128);
  };
  auto issue_scales = [&]() __attribute__((always_inline)) {
    const uint32_t dst = sbase + s_issue * SSTAGE;
    if constexpr (WIDE) {
      // (a branch inside the asm: see the loop)
      dma16_s_unless(__builtin_amdgcn_readfirstlane(k_issue % SPER),
                     __builtin_amdgcn_readfirstlane(dst + wid * 64 * 16), SOFF, offs, bases + (int64_t)k_issue * 8);
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w)
        dma4_s(__builtin_amdgcn_readfirstlane(dst + wid * 64 * 4), SOFF + w * R * 4, offs,
               bases + (int64_t)min(k_issue * 2 + w, last_word) * 4);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    b_issue ^= 1;
    if (k_issue % SPER == SPER - 1) s_issue ^= 1;   // (WIDE: KT is even)
    if (++k_issue == KT) {
      k_issue = 0;
      // past the last tile the ring goes round on that one, unread
      if (t_issue + stride < t_end) aim(t_issue += stride);
    }
  };
  // the wave's rows of the stage in buf reach past K: their chunks there to zero,
  // their scales to 1 (a NaN would spoil them; WIDE rows have no tail)
  auto zero_tail = [&](int buf) {
#pragma unroll
    for (int i = 0; i < CI; ++i)
      if ((KT - 1) * 256 + chunk(i) * 32 >= g.K)
        *reinterpret_cast<u32x4 *>(smem + buf * STAGE + (wid * CI + i) * 1024 + l * 16) = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int left = g.K / 32 - (KT - 1) * 8 - w * 4;   // blocks of the word inside K
      if (left >= 4) continue;
      uint32_t *p = reinterpret_cast<uint32_t *>(smem + SOFF + buf * SSTAGE + w * R * 4 + (wid * 64 + l) * 4);
      const uint32_t keep = left <= 0 ? 0u : ~0u >> (32 - 8 * left);
      *p = (*p & keep) | (0x7f7f7f7fu & ~keep);
    }
  };

  int t = t_issue;
  aim(t);
  issue_scales();
#pragma unroll
  for (int i = 0; i < CI; ++i) issue_codes(i);
  advance();

  // fragment offsets in a stage
  const int arow = (BM + wn * TN + (l & 31)) * 128, brow = (wm * TM + (l & 31)) * 128;
  int co[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) co[s] = ((2 * s + (l >> 5)) ^ ((l >> 1) & 7)) * 16;
  const int asc = SOFF + (BM + wn * TN + (l & 31)) * (WIDE ? 16 : 4);
  const int bsc = SOFF + (wm * TM + (l & 31)) * (WIDE ? 16 : 4);
  const int sh = (l >> 5) * 8;

  f32x16 acc[FN][FM];
  u32x4 a[2][FN], b[2][FM];
  uint32_t sa[2][FN], sb[2][FM];                    // the stage's scale words
  uint32_t ra[2][FN], rb[2][FM];                    // the next stage's
  auto zero_acc = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][i][v] = 0.f;
  };
  // the products so far, here and not where their sums are next looked at
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(acc[j][i]));
  };
  // fragment q of quarter s of the stage at st
  auto read1 = [&](int q, const unsigned char *st, int s) __attribute__((always_inline)) {
    if (q < FN)
      a[s & 1][q] = *reinterpret_cast<const u32x4 *>(st + arow + q * 32 * 128 + co[s]);
    else
      b[s & 1][q - FN] = *reinterpret_cast<const u32x4 *>(st + brow + (q - FN) * 32 * 128 + co[s]);
  };
  // the next stage's scale words, in order
  int s_read = 0, w_read = 0;
  auto read_scales = [&]() __attribute__((always_inline)) {
    const unsigned char *st = smem + s_read * SSTAGE + w_read * 8;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
        ra[w][j] = *reinterpret_cast<const uint32_t *>(
            st + asc + (WIDE ? j * 32 * 16 + w * 4 : j * 32 * 4 + w * R * 4));
#pragma unroll
      for (int i = 0; i < FM; ++i)
        rb[w][i] = *reinterpret_cast<const uint32_t *>(
            st + bsc + (WIDE ? i * 32 * 16 + w * 4 : i * 32 * 4 + w * R * 4));
    }
    w_read = WIDE ? w_read ^ 1 : 0;
    s_read = w_read ? s_read : s_read ^ 1;
  };

  int buf = 0, kt = 0;
  vm_wait<0>();
  if (!WIDE && ktail && KT == 1) zero_tail(0);
  lgkm_barrier();
  issue_scales();
#pragma unroll
  for (int i = 0; i < CI; ++i) issue_codes(i);
  advance();
  read_scales();
#pragma unroll
  for (int q = 0; q < FN + FM; ++q) read1(q, smem, 0);
  zero_acc();
  // A stage in four quarters of 64 codes; while one is multiplied, the next one's
  // fragments are read.  Before the last quarter the next stage has landed and
  // this one's buffer has been read: the loads of the stage after the next go into
  // it, one to a product, with three quarters left to land in.  Nothing that the
  // compiler sees branches among the products and the sums are pinned after each
  // quarter: it would otherwise move the products behind the next branch.
  while (true) {
    const unsigned char *st = smem + buf * STAGE, *nst = smem + (buf ^ 1) * STAGE;
    // byte 2 s of a shifted word: quarter s's block of this half of the wave
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int j = 0; j < FN; ++j) sa[w][j] = ra[w][j] >> sh;
#pragma unroll
      for (int i = 0; i < FM; ++i) sb[w][i] = rb[w][i] >> sh;
    }
#pragma unroll
    for (int s = 0; s < 3; ++s)
#pragma unroll
      for (int q = 0; q < FN * FM; ++q) {
        f32x16 &c = acc[q / FM][q % FM];
        if (s & 1)
          c = mfma_mx<2>(a[1][q / FM], b[1][q % FM], c, sa[0][q / FM], sb[0][q % FM]);
        else
          c = mfma_mx<0>(a[0][q / FM], b[0][q % FM], c, sa[s / 2][q / FM], sb[s / 2][q % FM]);
        if (q < FN + FM) read1(q, st, s + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
    pin();
    const bool last_stage = kt + 1 == KT;
    vm_wait<0>();                                   // the next stage has landed
    if (!WIDE && ktail && (last_stage ? KT == 1 : kt + 2 == KT)) zero_tail(buf ^ 1);
    lgkm_barrier();                                 // it is there, this one has been read
    read_scales();                                  // (after the last stage: of a settled buffer)
    issue_scales();
#pragma unroll
    for (int q = 0; q < FN * FM; ++q) {
      acc[q / FM][q % FM] = mfma_mx<2>(a[1][q / FM], b[1][q % FM], acc[q / FM][q % FM], sa[1][q / FM], sb[1][q % FM]);
      if (q < FN + FM) read1(q, nst, 0);
      issue_codes(q);
      __builtin_amdgcn_sched_barrier(0);
    }
    pin();
    advance();
    buf ^= 1;
    if (!last_stage) {
      ++kt;
      continue;
    }
    // the tile's rows: lane l has row wm TM + 32 i + l % 32 and, of each 32
    // columns, [8 v + 4 (l / 32), +4) in accumulator entries [4 v, 4 v + 4)
    int mi, ni;
    tile_at(t, tiles_m, tiles_n, mi, ni);
    const int n0 = ni * BN + wn * TN + (l >> 5) * 8;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = mi * BM + wm * TM + i * 32 + (l & 31);
      bf16_t *y = g.Y + (int64_t)row * g.ldy;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const f32x16 c = acc[j][i];
          uint32_t lo0 = pack_bf16x2(c[8 * p], c[8 * p + 1]), lo1 = pack_bf16x2(c[8 * p + 2], c[8 * p + 3]);
          uint32_t hi0 = pack_bf16x2(c[8 * p + 4], c[8 * p + 5]), hi1 = pack_bf16x2(c[8 * p + 6], c[8 * p + 7]);
          // lower lanes' second quad against upper lanes' first: 8 columns each
          const auto s0 = __builtin_amdgcn_permlane32_swap(lo0, hi0, false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(lo1, hi1, false, false);
          const int col = n0 + j * 32 + p * 16;
          if (row < g.M && col < g.N)               // N % 8 == 0: all 8 columns or none
            stg16(y + col, make_uint4(s0[0], s1[0], s0[1], s1[1]));
        }
    }
    t += stride;
    if (t >= t_end) break;
    kt = 0;
    zero_acc();
  }
  vm_wait<0>();                                     // no load outlives the workgroup's LDS
}

}  // namespace

hipError_t launch_mx_product(const void *X, int64_t ldx, const void *W, int64_t ldw,
                             const MxScales &mx, void *Y, int64_t ldy, int M, int K, int N,
                             hipStream_t stream) {
  const MxGemmArgs g{(const unsigned char *)X, mx.x, (const unsigned char *)W, mx.w,
                     ldx, mx.ldx, ldw, mx.ldw, (bf16_t *)Y, ldy, M, K, N};
  if (mx_wide_scales(K, mx.ldw, mx.ldx))
    hipLaunchKernelGGL((mx_product_kernel<256, 256, 4, 2, true>), dim3(kCUs), dim3(512), 0, stream, g);
  else
    hipLaunchKernelGGL((mx_product_kernel<256, 256, 4, 2, false>), dim3(kCUs), dim3(512), 0, stream, g);
  return hipGetLastError();
}

}  // namespace lora
