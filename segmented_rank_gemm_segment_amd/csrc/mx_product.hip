// Y = dq(Xq) dq(Wq)^T, both operands MXFP4, large batches: codes and scales go
// to v_mfma_scale_f32_32x32x64_f8f6f4 as they are.
//
// At 8.6 PFLOP/s (the rate of a loop of these MFMAs on registers alone) a
// 256 x 256 tile takes 1.2 thousand cycles for 128 codes of K and needs 34 KB of
// operands for them, so the kernel lives from keeping the loads ahead:
// * a ring of four buffers of 128 codes of K (64-byte rows, 16-byte chunks
//   XOR-swizzled so 16 lanes' reads hit 16 bank groups), filled by direct
//   global -> LDS loads three stages ahead; scales go into a ring of their own,
//   four words a row at once where alignment allows (a word a row costs as many
//   cache lookups as 64 bytes of codes: 671 us against 601);
// * waves 0-3 load the even stages and waves 4-7 the odd ones, so a wave never has
//   more than one stage in flight and waits for all of its loads (vmcnt(0)): no
//   wait depends on the order in which loads complete (two waves to a buffer,
//   with 16 loads each, were 6% slower).  One barrier per stage publishes the
//   next and frees a buffer;
// * loads spread over the products: issued together behind the barrier they fill
//   the load queue and hold the products up, and a stage's 8 over 8 products
//   measured 616 us against 603 over 16.  A wave whose turn it is not branches
//   over each inside the asm: branches that the compiler sees among the products
//   make it spill or move them;
// * workgroups are persistent, one per CU, and the ring runs on from one tile
//   into the next: the next tile's first stages are on their way while this
//   tile's last products and its stores run.
// W is the MFMA's row operand and X its column operand, so a lane ends up with
// one row of Y and runs of columns; two lanes swap halves (v_permlane32_swap)
// and each stores 16 bytes, without LDS, which the ring keeps.
// 16943 x 4096 x 14336: 603-613 us, 3.3 PFLOP/s; 8192^3: 305-312 us, 3.6 PFLOP/s.
// The clock falls as the matrix pipe gets busier (1.97 GHz at 40%, 1.84 at 48%).
// The loads alone take 305 us (64-byte row pieces use half of each 128-byte
// line), the products alone 283, the stores 100.
#include "lds_dma.cuh"
#include "lora_device.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

struct MxGemmArgs {
  const unsigned char *X, *SX, *W, *SW;   // codes and scales
  int64_t ldx, ldsx, ldw, ldsw;           // bytes a row
  bf16_t *Y;
  int64_t ldy;
  int M, K, N;
};

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kProductCUs = 256;
constexpr int kProductGroup = 8;   // M-tiles per group of the tile order

// SEL: the scale words' byte of this product's block (lds_dma.cuh's fragment
// layout: lane l holds row l % 32, codes [32 (l / 32), +32) of 64).
template <int SEL>
__device__ __forceinline__ f32x16 mfma_mx4(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SEL, (int)sa, SEL,
                                                         (int)sb);
}

// Tile t of the order: groups of kProductGroup M-tiles, each sweeping N.
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int &mi, int &ni) {
  const int grp = t / (kProductGroup * tiles_n), first = grp * kProductGroup;
  const int cnt = min(kProductGroup, tiles_m - first);
  const int in = t - grp * kProductGroup * tiles_n;
  mi = first + in % cnt;
  ni = in / cnt;
}

// WIDE: a load of the scales takes four words a row and serves four stages.
template <int BM, int BN, int WM, int WN, bool WIDE>
__global__ __launch_bounds__(WM *WN *kWave) void mx_product_kernel(MxGemmArgs g) {
  constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  constexpr int R = BM + BN;
  constexpr int STAGES = 4, STAGE = R * 64;
  constexpr int CI = R / 16 / 4, SI = R / 64 / 4;   // an owner's loads of codes and of scales
  constexpr int C0 = CI / 2;   // loads of codes under a stage's second half step, the rest under a first
  // scales: loaded every SPER stages into one of SBUFS buffers, SROW bytes a row
  constexpr int SPER = WIDE ? 4 : 1, SROW = 4 * SPER, SBUFS = WIDE ? 2 : STAGES, SSTAGE = R * SROW;
  static_assert(BM == BN && NW == 8 && CI == FM * FN, "owners, and loads to the products");
  static_assert(STAGES * STAGE + SBUFS * SSTAGE <= 160 * 1024, "LDS");
  __shared__ __align__(16) unsigned char smem[STAGES * STAGE + SBUFS * SSTAGE];

  const int tid = threadIdx.x, l = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int tiles_m = (g.M + BM - 1) / BM, tiles_n = (g.N + BN - 1) / BN;
  const int tiles = tiles_m * tiles_n;
  const int KT = (g.K + 127) / 128;
  const bool ktail = g.K % 128 != 0;

  // XCD x (workgroups x, x + 8, ...) owns the x-th eighth of the tile order and
  // its workgroups take that in turn.
  const int per = (tiles + 7) / 8, xcd = blockIdx.x & 7, stride = gridDim.x / 8;
  const int t_end = min(tiles, (xcd + 1) * per);
  int t_issue = xcd * per + blockIdx.x / 8;
  if (t_issue >= t_end) return;

  // This wave's loads, of every second stage: rows of one operand.  Load i has
  // rows [16 (CI w4 + i), +16) of the stage's (X's first), row l / 4 at physical
  // chunk l % 4, logical chunk `chunk`; rows past the end read the last one.
  const uint32_t sbase = lds_offset(smem);
  const int grp = wid / 4, w4 = wid % 4;
  const bool isx = w4 < 2;
  const unsigned char *const op = isx ? g.X : g.W, *const sop = isx ? g.SX : g.SW;
  const int64_t ldo = isx ? g.ldx : g.ldw, ldso = isx ? g.ldsx : g.ldsw;
  const int chunk = (l & 3) ^ ((l >> 4) & 3);
  const unsigned char *base = nullptr, *bases = nullptr;
  uint32_t off[CI], offs[SI];
  auto aim = [&](int t) __attribute__((always_inline)) {
    int mi, ni;
    tile_at(t, tiles_m, tiles_n, mi, ni);
    const int first = isx ? mi * BM : ni * BN;
    const int last = (isx ? g.M : g.N) - 1 - first;
#pragma unroll
    for (int i = 0; i < CI; ++i)
      off[i] = (uint32_t)min((w4 % 2 * CI + i) * 16 + l / 4, last) * (uint32_t)ldo + chunk * 16;
#pragma unroll
    for (int i = 0; i < SI; ++i) offs[i] = (uint32_t)min((w4 % 2 * SI + i) * 64 + l, last) * (uint32_t)ldso;
    base = op + (int64_t)first * ldo;
    bases = sop + (int64_t)first * ldso;
  };
  // The next stage to issue: stage k_issue of tile t_issue, into buffer b_issue,
  // its scales into buffer s_issue where a load of them is due.
  int k_issue = 0, b_issue = 0, s_issue = 0;
  auto issue_codes = [&](uint32_t skip, int i) __attribute__((always_inline)) {
    // a chunk past K reads the stage's first chunk (in bounds: it starts
    // before K) and is zeroed before use
    const uint32_t back =
        !WIDE && ktail && k_issue == KT - 1 && k_issue * 128 + chunk * 32 >= g.K ? chunk * 16 : 0;
    dma16_s_unless(skip, __builtin_amdgcn_readfirstlane(sbase + b_issue * STAGE + (w4 * CI + i) * 1024),
                   off[i] - back, base + (int64_t)k_issue * 64);
  };
  auto issue_scales = [&](uint32_t skip) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      const uint32_t dst = __builtin_amdgcn_readfirstlane(sbase + STAGES * STAGE + s_issue * SSTAGE +
                                                          (w4 * SI + i) * 64 * SROW);
      if constexpr (WIDE)
        dma16_s_unless(skip, dst, offs[i], bases + (int64_t)k_issue * 4);
      else
        dma4_s_unless(skip, dst, offs[i], bases + (int64_t)k_issue * 4);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    b_issue = b_issue + 1 == STAGES ? 0 : b_issue + 1;
    if (k_issue % SPER == 0) s_issue = s_issue + 1 == SBUFS ? 0 : s_issue + 1;
    if (++k_issue == KT) {
      k_issue = 0;
      // past the last tile the ring goes round on that one, unread
      if (t_issue + stride < t_end) aim(t_issue += stride);
    }
  };
  // the owner's stage in buf reaches past K: its chunks there to zero, their
  // scales to 1 (a NaN would spoil them; WIDE rows have no tail)
  auto zero_tail = [&](int buf) {
    unsigned char *st = smem + buf * STAGE;
#pragma unroll
    for (int i = 0; i < CI; ++i)
      if ((KT - 1) * 128 + chunk * 32 >= g.K)
        *reinterpret_cast<u32x4 *>(st + (w4 * CI + i) * 1024 + l * 16) = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      uint32_t *p = reinterpret_cast<uint32_t *>(smem + STAGES * STAGE + buf * SSTAGE +
                                                 (w4 * SI + i) * 256 + l * 4);
      const uint32_t keep = ~0u >> (32 - 8 * (g.K / 32 - (KT - 1) * 4));   // 1..3 blocks
      *p = (*p & keep) | (0x7f7f7f7fu & ~keep);
    }
  };

  int t = t_issue;
  aim(t);
  for (int s = 0; s < 2; ++s) {
    const uint32_t skip = __builtin_amdgcn_readfirstlane(s ^ grp);
    issue_scales(skip | k_issue % SPER);
#pragma unroll
    for (int i = 0; i < CI; ++i) issue_codes(skip, i);
    advance();
  }

  // fragment offsets in a stage
  const int arow = (BM + wn * TN + (l & 31)) * 64, brow = (wm * TM + (l & 31)) * 64;
  int co[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) co[s] = ((2 * s + (l >> 5)) ^ ((l >> 2) & 3)) * 16;
  const int asc = STAGES * STAGE + (BM + wn * TN + (l & 31)) * SROW;
  const int bsc = STAGES * STAGE + (wm * TM + (l & 31)) * SROW;
  const int sh = (l >> 5) * 8;

  f32x16 acc[FN][FM];
  u32x4 a[2][FN], b[2][FM];
  uint32_t sa[FN], sb[FM], ra[FN], rb[FM];          // the stage's scales, the next one's words
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
  // fragment q of half step s of the stage at st
  auto read1 = [&](int q, const unsigned char *st, int s) __attribute__((always_inline)) {
    if (q < FN)
      a[s][q] = *reinterpret_cast<const u32x4 *>(st + arow + q * 32 * 64 + co[s]);
    else
      b[s][q - FN] = *reinterpret_cast<const u32x4 *>(st + brow + (q - FN) * 32 * 64 + co[s]);
  };
  // the next stage's scale words, in order
  int s_read = 0, w_read = 0;
  auto read_scales = [&]() __attribute__((always_inline)) {
    const unsigned char *st = smem + s_read * SSTAGE + w_read * 4;
#pragma unroll
    for (int j = 0; j < FN; ++j)
      ra[j] = *reinterpret_cast<const uint32_t *>(st + asc + j * 32 * SROW);
#pragma unroll
    for (int i = 0; i < FM; ++i)
      rb[i] = *reinterpret_cast<const uint32_t *>(st + bsc + i * 32 * SROW);
    const bool next = ++w_read == SPER;
    w_read = next ? 0 : w_read;
    s_read = next ? (s_read + 1 == SBUFS ? 0 : s_read + 1) : s_read;
  };

  int buf = 0, kt = 0, turn = 0;                    // turn: the owner of stage kt
  if (grp == 0) {
    vm_wait<0>();
    if (ktail && KT == 1) zero_tail(0);
  }
  issue_scales(grp | k_issue % SPER);               // stage 2's first loads
#pragma unroll
  for (int i = 0; i < C0; ++i) issue_codes(grp, i);
  lgkm_barrier();
  read_scales();
#pragma unroll
  for (int q = 0; q < FN + FM; ++q) read1(q, smem, 0);
  zero_acc();
  // A stage in two half steps of 64 codes.  While the first is multiplied, the
  // second's fragments are read; then stage kt + 1 has landed and its first
  // fragments are read while the second half step is multiplied.  Under the first
  // half step go the rest of stage kt + 2's loads, under the second the first of
  // stage kt + 3's, by the waves that have just waited for stage kt + 1 (into a
  // buffer that was last read during stage kt - 1).  The sums are pinned after
  // each half step: the compiler would otherwise move the products behind the
  // next branch.
  while (true) {
    const unsigned char *st = smem + buf * STAGE;
    const int nbuf = buf + 1 == STAGES ? 0 : buf + 1;
    const uint32_t skip = __builtin_amdgcn_readfirstlane(turn ^ grp);
    // byte 2 s of a shifted word: half step s's block of this half of the wave
#pragma unroll
    for (int j = 0; j < FN; ++j) sa[j] = ra[j] >> sh;
#pragma unroll
    for (int i = 0; i < FM; ++i) sb[i] = rb[i] >> sh;
#pragma unroll
    for (int q = 0; q < FN * FM; ++q) {
      acc[q / FM][q % FM] = mfma_mx4<0>(a[0][q / FM], b[0][q % FM], acc[q / FM][q % FM], sa[q / FM], sb[q % FM]);
      if (q < FN + FM) read1(q, st, 1);
      if (q % 2 == 0) issue_codes(skip, C0 + q / 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    pin();
    const bool last_stage = kt + 1 == KT;
    advance();
    if (skip) {                                     // the next stage's owners: it has landed
      vm_wait<0>();
      if (!WIDE && ktail && (last_stage ? KT == 1 : kt + 2 == KT)) zero_tail(nbuf);
    }
    lgkm_barrier();                                 // stage kt + 1 is there, stage kt has been read
    read_scales();                                  // (after the last stage: of a settled buffer)
    issue_scales((skip ^ 1) | k_issue % SPER);
#pragma unroll
    for (int q = 0; q < FN * FM; ++q) {
      acc[q / FM][q % FM] = mfma_mx4<2>(a[1][q / FM], b[1][q % FM], acc[q / FM][q % FM], sa[q / FM], sb[q % FM]);
      if (q < FN + FM) read1(q, smem + nbuf * STAGE, 0);
      if (q % 2 == 0) issue_codes(skip ^ 1, q / 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    pin();
    buf = nbuf;
    turn ^= 1;
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
  // four scale words at a time where every row's are whole and aligned to that
  if (K % 512 == 0 && mx.ldx % 16 == 0 && mx.ldw % 16 == 0)
    hipLaunchKernelGGL((mx_product_kernel<256, 256, 4, 2, true>), dim3(kProductCUs), dim3(512), 0, stream, g);
  else
    hipLaunchKernelGGL((mx_product_kernel<256, 256, 4, 2, false>), dim3(kProductCUs), dim3(512), 0, stream, g);
  return hipGetLastError();
}

}  // namespace lora
