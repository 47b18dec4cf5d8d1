// The experts' products on bf16 weights that write rows: for every sorted row p of
// expert e,
//
//   kForward  Y[p]  = X[row(p)] W_e^T                  sums over d_in
//   kRows     dX[p] = dY[p] W_e                        sums over d_out
//
// on BM x BN tiles (rows x outputs), K in stages of 64 in two LDS buffers.  W's memory
// runs along K in the one and along the outputs in the other (experts_tiles.cuh).
//
// Workgroups are persistent; each XCD walks its own eighth of the tiles, an expert's M-tiles
// in groups that sweep N, and the loads of a tile's first stages go out under the products
// of the one before.  Per stage a wave waits for all of its loads (it has one stage's in
// flight, so no wait depends on their order) and the workgroup passes one barrier, before
// the last sub-step's products, under which the stage after the next is loaded.
//
// Long segments, 256 x 256 tiles: a stage is 64 KB a CU, 128 flops a byte.  16384 rows, 4096
// -> 14336 in 1435 us (1.34 PFLOP/s; a library's product reaches 1.36 there): its loads
// alone take 1140 and its products alone, whose power brings the clock down to about 1.5
// GHz, 1230.  64 experts of 1024 rows, 2048 -> 1536: 368 us (1.12 PFLOP/s); the loads alone
// 326 (10 TB/s from the L2s), the products 280, and 330 without the stores of 200 MB.
// L2 prefetch of the following stage, a line a lane, took 15% more time; branches that
// leave out fragments past an expert's last row took more than they saved.  (Issue priority
// past the barrier: 2%.)
// Short segments: 128 x 128 tiles, two workgroups a CU, or the kernel for few rows below
// (tile_choice.h), bound by W's bytes.  64 x 8 choices on 128 experts of 2048 -> 1536 in 144
// to 156 us, 5.2 to 5.6 TB/s; one token's 8 choices, 50 MB, in 13.6, 3.7 TB/s.
#include <type_traits>

#include "experts_tiles.cuh"

namespace lora {
namespace {

enum Form { kForward = 0, kRows = 1 };

// One operand's loads: I instructions of 1 KB a wave and stage, RPI LDS rows each.
template <int B, bool ALONG_K, int NW> struct StageLoads {
  static constexpr int BYTES = B * 128, I = BYTES / 1024 / NW;
  static constexpr int LPR = (ALONG_K ? 128 : B * 2) / 16, RPI = 64 / LPR;   // lanes a row
  static_assert(BYTES % (1024 * NW) == 0, "loads");
  __device__ static __forceinline__ int row(int wid, int i, int l) { return (wid * I + i) * RPI + l / LPR; }
  // elements from the start of its row's memory that the lane loads
  __device__ static __forceinline__ int chunk(int wid, int i, int l) {
    return ((l % LPR) ^ chunk_xor<B, ALONG_K>(row(wid, i, l))) * 8;
  }
};

// TAIL: K is no multiple of 64.
template <int FORM, int BM, int BN, int WM, int WN, int PER_CU, bool TAIL>
__global__ __launch_bounds__(WM *WN *kWave, WM *WN *PER_CU / 4) void experts_gemm_kernel(ExpertGemmArgs g) {
  constexpr int NW = WM * WN, T = NW * kWave;
  constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  using OP = StageLoads<BM, true, NW>;
  using OQ = StageLoads<BN, FORM == kForward, NW>;
  constexpr int STAGE = OP::BYTES + OQ::BYTES;
  constexpr int SMEM = 2 * STAGE + kExpertTab + NW * 2048;
  static_assert(SMEM * PER_CU <= 160 * 1024, "LDS");
  __shared__ __align__(16) unsigned char smem[SMEM];
  int *const tab = reinterpret_cast<int *>(smem + 2 * STAGE);

  const int tid = threadIdx.x, l = tid & (kWave - 1);
  const int wid = scalar_int(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int E = g.n_experts, N = g.N;
  const int tiles_n = (N + BN - 1) / BN;

  // tab[e]: M-tiles of the experts before e
  expert_table<T>(E, tab, reinterpret_cast<int *>(smem),
                  [&](int e) { return (g.off[e + 1] - g.off[e] + BM - 1) / BM; });
  // XCD x owns the x-th eighth of the tiles
  const int tiles = scalar_int(tab[E]) * tiles_n;
  const int per = (tiles + 7) / 8, xcd = blockIdx.x & 7, stride = gridDim.x / 8;
  const int t_end = min(tiles, (xcd + 1) * per);
  int t = xcd * per + blockIdx.x / 8;
  if (t >= t_end) return;

  struct Tile {
    int m0, m_end, n0, e;
  };
  auto tile_of = [&](int t) __attribute__((always_inline)) {
    Tile x;
    int mi, ni;
    x.e = expert_find(tab, E, scalar_int(t / tiles_n));
    const int first = scalar_int(tab[x.e]);
    tile_at(t - first * tiles_n, scalar_int(tab[x.e + 1]) - first, tiles_n, mi, ni);
    x.m0 = scalar_int(g.off[x.e]) + scalar_int(mi) * BM;
    x.m_end = scalar_int(g.off[x.e + 1]);
    x.n0 = scalar_int(ni) * BN;
    return x;
  };

  // This wave's loads: 32-bit byte offsets of the lanes from a scalar base (leading
  // dimensions are below 2^22), but for X's rows, which lie anywhere.  Whatever lies past an
  // end is read from a valid place instead: rows and columns past it are not stored, k past
  // it are zeroed in LDS before use.
  const int stages = (g.K + 63) / 64;
  const uint32_t sbase = lds_offset(smem);
  const uint32_t p_dst = scalar_int(sbase + wid * OP::I * 1024);
  const uint32_t q_dst = scalar_int(sbase + OP::BYTES + wid * OQ::I * 1024);
  int k_i = 0, b_i = 0, t_i = t;                    // the next stage to load, its buffer, its tile
  const unsigned char *pbase = nullptr, *qbase = nullptr;   // at that stage
  const int64_t qstep = FORM == kForward ? 128 : 128 * g.ldq;
  const unsigned char *prow[FORM == kForward ? OP::I : 1];
  uint32_t poff[FORM == kForward ? 1 : OP::I], qoff[OQ::I];
  auto aim = [&](int t) __attribute__((always_inline)) {
    const Tile x = tile_of(t);
    // (the lane by way of the asm: what depends on it alone would otherwise be computed
    // ahead of the loop and held in registers that the products need)
    int ln = l;
    asm volatile("" : "+v"(ln));
    const bf16_t *const w = g.Q + x.e * g.w_stride;
    if constexpr (FORM == kRows) pbase = scalar_ptr(g.P + (int64_t)x.m0 * g.ldp);
    qbase = scalar_ptr(FORM == kForward ? w + (int64_t)x.n0 * g.ldq : w + x.n0);
#pragma unroll
    for (int i = 0; i < OP::I; ++i) {
      const int c = OP::chunk(wid, i, ln), r = min(OP::row(wid, i, ln), x.m_end - 1 - x.m0);
      if constexpr (FORM == kRows) {
        poff[i] = ((uint32_t)r * (uint32_t)g.ldp + (uint32_t)c) * 2u;
      } else {
        const int p = x.m0 + r;
        const int row = g.sorted ? token_of(g, g.sorted[p]) : p;
        prow[i] = reinterpret_cast<const unsigned char *>(g.P + (int64_t)row * g.ldp + c);
      }
    }
#pragma unroll
    for (int i = 0; i < OQ::I; ++i) {
      const int c = OQ::chunk(wid, i, ln), r = OQ::row(wid, i, ln);
      if constexpr (FORM == kForward)
        qoff[i] = ((uint32_t)min(r, N - 1 - x.n0) * (uint32_t)g.ldq + (uint32_t)c) * 2u;
      else
        qoff[i] = ((uint32_t)r * (uint32_t)g.ldq + (uint32_t)(x.n0 + c < N ? c : 0)) * 2u;
    }
  };
  auto issue_p = [&](int i) __attribute__((always_inline)) {
    const uint32_t dst = scalar_int(p_dst + b_i * STAGE);
    const int c = OP::chunk(wid, i, l);
    const uint32_t back = TAIL && k_i * 64 + c >= g.K ? c * 2u : 0u;     // to the stage's first k
    if constexpr (FORM == kForward)
      dma16(dst, i * 1024, prow[i] + k_i * 128 - back);
    else
      dma16_s(dst, i * 1024, poff[i] - back, pbase);
  };
  auto issue_q = [&](int i) __attribute__((always_inline)) {
    const uint32_t dst = scalar_int(q_dst + b_i * STAGE);
    if constexpr (FORM == kForward) {
      const int c = OQ::chunk(wid, i, l);
      dma16_s(dst, i * 1024, qoff[i] - (TAIL && k_i * 64 + c >= g.K ? c * 2u : 0u), qbase);
    } else {
      const int r = OQ::row(wid, i, l);
      dma16_s(dst, i * 1024, qoff[i] - (TAIL && k_i * 64 + r >= g.K ? (uint32_t)r * (uint32_t)g.ldq * 2u : 0u), qbase);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    b_i ^= 1;
    if constexpr (FORM == kRows) pbase += 128;
    qbase += qstep;
    if (++k_i == stages) {
      k_i = 0;
      // past the last tile the loads go round on that one, unread
      if (t_i + stride < t_end) t_i += stride;
      aim(t_i);
    }
  };
  // stage k in buffer b: what this wave loaded past K to zero
  auto zero_tail = [&](int k, int b) {
    const u32x4 z = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < OP::I; ++i)
      if (k * 64 + OP::chunk(wid, i, l) >= g.K)
        *reinterpret_cast<u32x4 *>(smem + b * STAGE + (wid * OP::I + i) * 1024 + l * 16) = z;
#pragma unroll
    for (int i = 0; i < OQ::I; ++i)
      if (k * 64 + (FORM == kForward ? OQ::chunk(wid, i, l) : OQ::row(wid, i, l)) >= g.K)
        *reinterpret_cast<u32x4 *>(smem + b * STAGE + OP::BYTES + (wid * OQ::I + i) * 1024 + l * 16) = z;
  };

  FragmentReader<BM, true, WM> pr;
  FragmentReader<BN, FORM == kForward, WN> qr;
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
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(acc[j][i]));
  };
  auto read = [&](int to, int q, const unsigned char *st, int kk) __attribute__((always_inline)) {
    if (q < FN)
      qf[to][q] = qr.read(st + OP::BYTES, q, kk);
    else
      pf[to][q - FN] = pr.read(st, q - FN, kk);
  };
  // Sub-step kk's products with the reads of the next one's fragments from st, and the
  // loads of the next stage but one where LOAD.
  constexpr int NM = FM * FN, NR = FM + FN, NL = OP::I + OQ::I;
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
  auto issue = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < OP::I; ++i) issue_p(i);
#pragma unroll
    for (int i = 0; i < OQ::I; ++i) issue_q(i);
    advance();
  };

  aim(t);
  issue();
  vm_wait<0>();                                     // the first stage has landed
  if (TAIL && stages == 1) zero_tail(0, 0);
  lgkm_barrier();
  issue();
#pragma unroll
  for (int q = 0; q < NR; ++q) read(0, q, smem, 0);
  zero_acc();
  Tile nx = tile_of(t);
  int kt = 0, b = 0;
  while (true) {
    const unsigned char *st = smem + b * STAGE;
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) sub_step(std::false_type{}, kk, st);
    const bool last = kt + 1 == stages;
    const Tile x = nx;
    if (last && t + stride < t_end) nx = tile_of(t + stride);
    kt = last ? 0 : kt + 1;                         // the next stage
    pin();
    vm_wait<0>();                                   // it has landed
    if (TAIL && kt + 1 == stages) zero_tail(kt, b ^ 1);
    lgkm_barrier();                                 // it is there, and this one has been read
    __builtin_amdgcn_s_setprio(1);
    sub_step(std::true_type{}, 3, smem + (b ^ 1) * STAGE);
    __builtin_amdgcn_s_setprio(0);
    pin();
    advance();
    b ^= 1;
    if (!last) continue;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = x.m0 + (wm * FM + i) * 32, col = x.n0 + (wn * FN + j) * 32;
        store_fragment<false, false>(smem + 2 * STAGE + kExpertTab + wid * 2048, acc[j][i], l,
                                     static_cast<bf16_t *>(g.out) + (int64_t)row * g.ldo + col, g.ldo,
                                     x.m_end - row, N - col, false);
      }
    t += stride;
    if (t >= t_end) break;
    zero_acc();
    pin();                                          // (zeros in these registers: 81 were spilled without)
  }
  vm_wait<0>();                                     // no load outlives the workgroup's LDS
}

// A batch of few rows has few tiles, and a CU that streams a tile's W by itself waits for
// memory most of the time: 32 x BN tiles whose K goes round over the workgroup's waves in
// stages of 64, each wave with two buffers of its own.  A wave waits for all of its loads,
// sends out its next stage's and multiplies the one that has landed; the waves' sums are
// added through LDS in their order.
constexpr int kFewWaves = 4;
template <int FORM, int BN, int PER_CU, bool TAIL>
__global__ __launch_bounds__(kFewWaves *kWave, PER_CU) void experts_few_kernel(ExpertGemmArgs g) {
  constexpr int BM = 32, FN = BN / 32, T = kFewWaves * kWave;
  using OP = StageLoads<BM, true, 1>;
  using OQ = StageLoads<BN, FORM == kForward, 1>;
  constexpr int STAGE = OP::BYTES + OQ::BYTES;
  constexpr int RING = kFewWaves * 2 * STAGE;
  static_assert((RING + kExpertTab) * PER_CU <= 160 * 1024, "LDS");
  static_assert(kFewWaves * FN * 16 * kWave * 4 + kFewWaves * 2048 <= RING && FN <= kFewWaves, "sums");
  __shared__ __align__(16) unsigned char smem[RING + kExpertTab];
  int *const tab = reinterpret_cast<int *>(smem + RING);
  const int l = threadIdx.x & (kWave - 1), w = scalar_int(threadIdx.x / kWave);
  const int E = g.n_experts, N = g.N, K = g.K;
  const int tiles_n = (N + BN - 1) / BN, stages = (K + 63) / 64;
  expert_table<T>(E, tab, reinterpret_cast<int *>(smem),
                  [&](int e) { return (g.off[e + 1] - g.off[e] + BM - 1) / BM; });
  const int tiles = scalar_int(tab[E]) * tiles_n;
  unsigned char *const mine = smem + w * 2 * STAGE;
  const uint32_t dst = scalar_int(lds_offset(mine));
  FragmentReader<BM, true, 1> pr;
  FragmentReader<BN, FORM == kForward, 1> qr;
  pr.init(0, l);
  qr.init(0, l);

  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int e = expert_find(tab, E, scalar_int(t / tiles_n));
    const int first = scalar_int(tab[e]) * tiles_n;
    const int m0 = scalar_int(g.off[e]) + scalar_int((t - first) / tiles_n) * BM;
    const int n0 = scalar_int((t - first) % tiles_n) * BN, m_end = scalar_int(g.off[e + 1]);
    // where past an end something valid is read instead, as in the larger tiles
    const bf16_t *const we = g.Q + e * g.w_stride;
    const unsigned char *const qbase = scalar_ptr(FORM == kForward ? we + (int64_t)n0 * g.ldq : we + n0);
    const unsigned char *prow[OP::I];
    uint32_t qoff[OQ::I];
#pragma unroll
    for (int i = 0; i < OP::I; ++i) {
      const int p = min(m0 + OP::row(0, i, l), m_end - 1);
      const int row = FORM == kForward && g.sorted ? token_of(g, g.sorted[p]) : p;
      prow[i] = reinterpret_cast<const unsigned char *>(g.P + (int64_t)row * g.ldp + OP::chunk(0, i, l));
    }
#pragma unroll
    for (int i = 0; i < OQ::I; ++i) {
      const int c = OQ::chunk(0, i, l), r = OQ::row(0, i, l);
      if constexpr (FORM == kForward)
        qoff[i] = ((uint32_t)min(r, N - 1 - n0) * (uint32_t)g.ldq + (uint32_t)c) * 2u;
      else
        qoff[i] = ((uint32_t)r * (uint32_t)g.ldq + (uint32_t)(n0 + c < N ? c : 0)) * 2u;
    }
    auto issue = [&](int s, int b) __attribute__((always_inline)) {
      const uint32_t d = scalar_int(dst + b * STAGE);
      const unsigned char *const q = scalar_ptr(qbase + (int64_t)s * (FORM == kForward ? 128 : 128 * g.ldq));
#pragma unroll
      for (int i = 0; i < OP::I; ++i) {
        const int c = OP::chunk(0, i, l);
        dma16(d, i * 1024, prow[i] + (TAIL && s * 64 + c >= K ? s * 128 - c * 2 : s * 128));
      }
#pragma unroll
      for (int i = 0; i < OQ::I; ++i) {
        const int c = OQ::chunk(0, i, l), r = OQ::row(0, i, l);
        const uint32_t back = !TAIL                ? 0u
                              : FORM == kForward   ? (s * 64 + c >= K ? c * 2u : 0u)
                              : s * 64 + r >= K    ? (uint32_t)r * (uint32_t)g.ldq * 2u
                                                   : 0u;
        dma16_s(d, OP::BYTES + i * 1024, qoff[i] - back, q);
      }
    };
    f32x16 acc[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[j][v] = 0.f;
    int b = 0;
    if (w < stages) issue(w, 0);
    for (int s = w; s < stages; s += kFewWaves) {
      vm_wait<0>();                                 // stage s has landed
      unsigned char *const st = mine + b * STAGE;
      if (TAIL && s + 1 == stages) {
        const u32x4 z = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < OP::I; ++i)
          if (s * 64 + OP::chunk(0, i, l) >= K) *reinterpret_cast<u32x4 *>(st + i * 1024 + l * 16) = z;
#pragma unroll
        for (int i = 0; i < OQ::I; ++i)
          if (s * 64 + (FORM == kForward ? OQ::chunk(0, i, l) : OQ::row(0, i, l)) >= K)
            *reinterpret_cast<u32x4 *>(st + OP::BYTES + i * 1024 + l * 16) = z;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the other buffer has been read
      if (s + kFewWaves < stages) issue(s + kFewWaves, b ^ 1);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const mfma_bf16x8 p = pr.read(st, 0, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qr.read(st + OP::BYTES, j, kk), p, acc[j], 0, 0, 0);
      }
      b ^= 1;
    }
    __syncthreads();                                // the rings are free
    f32x4 *const sums = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sums[((w * FN + j) * 4 + v) * kWave + l] = f32x4{acc[j][4 * v], acc[j][4 * v + 1], acc[j][4 * v + 2], acc[j][4 * v + 3]};
    __syncthreads();
    if (w < FN) {
      f32x16 c;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        f32x4 x = sums[(w * 4 + v) * kWave + l];
#pragma unroll
        for (int o = 1; o < kFewWaves; ++o) x += sums[((o * FN + w) * 4 + v) * kWave + l];
#pragma unroll
        for (int q = 0; q < 4; ++q) c[4 * v + q] = x[q];
      }
      store_fragment<false, false>(smem + kFewWaves * FN * 16 * kWave * 4 + w * 2048, c, l,
                                   static_cast<bf16_t *>(g.out) + (int64_t)m0 * g.ldo + n0 + w * 32, g.ldo,
                                   m_end - m0, N - n0 - w * 32, false);
    }
    __syncthreads();                                // and again
  }
}

template <int FORM, int BN, int PER_CU> void launch_few(const ExpertGemmArgs &g, hipStream_t stream) {
  const dim3 grid(kCUs * PER_CU), block(kFewWaves * kWave);
  if (g.K % 64 == 0)
    hipLaunchKernelGGL((experts_few_kernel<FORM, BN, PER_CU, false>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((experts_few_kernel<FORM, BN, PER_CU, true>), grid, block, 0, stream, g);
}

template <int FORM, int BM, int BN, int WM, int WN, int PER_CU>
void launch_tiles(const ExpertGemmArgs &g, hipStream_t stream) {
  const dim3 grid(kCUs * PER_CU), block(WM * WN * kWave);
  if (g.K % 64 == 0)
    hipLaunchKernelGGL((experts_gemm_kernel<FORM, BM, BN, WM, WN, PER_CU, false>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((experts_gemm_kernel<FORM, BM, BN, WM, WN, PER_CU, true>), grid, block, 0, stream, g);
}

template <int FORM> hipError_t launch_rows(const ExpertGemmArgs &g, hipStream_t stream) {
  switch (experts_kernel_of(g.n_choices, g.n_experts, g.K, g.N, FORM == kForward)) {
    case kExpertsFew: launch_few<FORM, 64, 1>(g, stream); break;
    case kExpertsMid: launch_tiles<FORM, 128, 128, 2, 2, 2>(g, stream); break;
    default: launch_tiles<FORM, 256, 256, 2, 4, 1>(g, stream);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_gemm(const void *X, int64_t ldx, const ExpertView &ex, const void *W,
                               int64_t ldw, void *Y, int64_t ldy, int K, int N, hipStream_t stream) {
  return launch_rows<kForward>(expert_args(X, ldx, W, ldw, Y, ldy, 0, N, K, ex), stream);
}

hipError_t launch_experts_gemm_rows(const void *dY, int64_t lddy, const ExpertView &ex,
                                    const void *W, int64_t ldw, void *dX, int64_t lddx, int K,
                                    int N, hipStream_t stream) {
  return launch_rows<kRows>(expert_args(dY, lddy, W, ldw, dX, lddx, 0, N, K, ex), stream);
}

}  // namespace lora
