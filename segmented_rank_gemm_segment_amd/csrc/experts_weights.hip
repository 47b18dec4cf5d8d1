// The gradients of the experts' weights: for every expert e with sorted rows p,
//
//   dW_e[j][c] (+)= sum_p dY[p][j] X[row(p)][c]
//
// on 256 x 256 tiles (j x c) of a persistent workgroup, the expert's rows being K, in stages
// of 64 and two LDS buffers.  Both operands' memory runs along the outputs: a row of dY and
// one of X are a k each, staged and read by the LDS transpose read (experts_tiles.cuh).
//
// Waits and barriers as in the products that write rows (experts_gemm.hip).  A stage's loads
// have other rows than the last one's, so their addresses take more arithmetic; it stands
// between the products of the first sub-steps (16384 rows, 14336 x 4096, 1904 us with it
// among the last sub-step's loads, 2030 after them, 1720 so).  Loads by two owner waves of a
// ring of four stages of 32, each in one go, took 3300: the others wait for the owners.
//
// An expert's tiles cost its stages and kTileCost more; each XCD takes an eighth of the
// cost, and its CUs an expert's tiles together, which share the operands in its L2.  (Every
// CU the same number of each expert's tiles, longest first, and what is left back and forth
// between the CUs, so that all end together: 5% more time, as the CUs share what binds them.)
//
// Bound by the loads (1380 of the 1720 us alone) and the products (1340 alone, at the clock
// that their power leaves), 1.12 PFLOP/s; an expert's few stages add the waits at tiles'
// ends: 64 experts of 1024 rows, 2048 -> 1536, in 414 us in sorted order, 445 with X's rows
// gathered, 515 with uneven experts.  Few rows:
// the stores, 128 experts of 1 row, 175 us of 156 at a copy's rate.  Experts without rows
// have a stage of zeros and their stores, and with `accumulate` are read and written back: 26
// choices on 212 experts of 1024 x 1024, added, 260 us.  An expert's rows are not shared: two
// experts of 8190 rows, 256 x 256, have 8 workgroups and take 98 us.
#include <type_traits>

#include "experts_tiles.cuh"

namespace lora {
namespace {

constexpr int kKS = 64, kRing = 2;          // k of a stage, buffers
constexpr int kTileCost = 2;                // of a tile's start and stores, in stages

// GATHER: X's rows by way of sorted_choice.
template <int BM, int BN, int WM, int WN, int PER_CU, bool F32OUT, bool GATHER>
__global__ __launch_bounds__(WM *WN *kWave, WM *WN *PER_CU / 4) void experts_weights_kernel(ExpertGemmArgs g) {
  constexpr int NW = WM * WN, T = NW * kWave;
  constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
  constexpr int PB = BM * kKS * 2, QB = BN * kKS * 2, STAGE = PB + QB;
  constexpr int I = PB / 1024 / NW;         // a wave's loads of an operand and stage
  constexpr int LPR = BM * 2 / 16, RPI = 64 / LPR;          // lanes a row, rows a load
  constexpr int NC = 4 / RPI;               // loads of a wave that differ in their chunks
  static_assert(BM == BN && RPI <= 4, "the operands' loads are alike");
  constexpr int SMEM = kRing * STAGE + kExpertTab + NW * 2048;
  static_assert(SMEM * PER_CU <= 160 * 1024, "LDS");
  __shared__ __align__(16) unsigned char smem[SMEM];
  int *const tab = reinterpret_cast<int *>(smem + kRing * STAGE);

  const int tid = threadIdx.x, l = tid & (kWave - 1), h = l / LPR;    // the lane's row of a load
  const int wid = scalar_int(tid / kWave);
  const int wm = wid / WN, wn = wid % WN;
  const int E = g.n_experts, M = g.M, N = g.N;
  const int tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN, tiles_e = tiles_m * tiles_n;

  // tab[e]: cost of a tile of every expert before e
  auto stages_of = [](int rows) { return max(1, (rows + kKS - 1) / kKS); };   // (no rows: one of zeros)
  expert_table<T>(E, tab, reinterpret_cast<int *>(smem),
                  [&](int e) { return stages_of(g.off[e + 1] - g.off[e]) + kTileCost; });
  const int xcd = blockIdx.x & 7, stride = gridDim.x / 8;
  const int all = scalar_int(tab[E]);
  auto begin_of = [&](int x) __attribute__((always_inline)) -> int {
    if (x == 8) return E * tiles_e;
    const int64_t at = (int64_t)all * x / 8;
    const int e = expert_find(tab, E, scalar_int((int)at));
    const int c0 = scalar_int(tab[e]), c1 = scalar_int(tab[e + 1]);
    return scalar_int(e * tiles_e + (int)((at - c0) * tiles_e / (c1 - c0)));
  };
  const int t_end = begin_of(xcd + 1);
  int t = begin_of(xcd) + blockIdx.x / 8;
  if (t >= t_end) return;

  struct Tile {
    int m0, n0, e, r0, rows, stages;
  };
  auto tile_of = [&](int t) __attribute__((always_inline)) {
    Tile x;
    int mi, ni;
    x.e = scalar_int(t / tiles_e);
    tile_at(t - x.e * tiles_e, tiles_m, tiles_n, mi, ni);
    x.m0 = scalar_int(mi) * BM;
    x.n0 = scalar_int(ni) * BN;
    x.r0 = scalar_int(g.off[x.e]);
    x.rows = scalar_int(g.off[x.e + 1]) - x.r0;
    x.stages = stages_of(x.rows);
    return x;
  };

  // This wave's loads, I instructions of RPI rows for each operand and stage.  Rows past the
  // last one are zeroed in LDS before use and read from a valid row here; an expert without
  // rows reads the start of the output, which is there even where a batch without tokens has
  // no rows at all.  Columns past the last one are not stored.
  const uint32_t sbase = lds_offset(smem);
  const uint32_t dst = scalar_int(sbase + wid * I * 1024);
  auto local_row = [&](int i, int h) __attribute__((always_inline)) { return (wid * I + i) * RPI + h; };
  Tile li;                                          // the tile being loaded
  int k_i = 0, b_i = 0, t_i = t;                    // its next stage, the buffer for it
  int f_r0, f_left;                                 // the stage after that one: first row, rows from there
  const unsigned char *pbase = nullptr, *qbase = nullptr;
  const uint32_t ldp2 = (uint32_t)(g.ldp * 2), ldq2 = (uint32_t)(g.ldq * 2);
  const int64_t pstep = kKS * 2 * g.ldp;
  const uint32_t hoff = h * ldp2;
  uint32_t pc[NC], qc[NC];                          // bytes of the lane's chunk of a load
  // Addresses are made, and the following stage's rows looked up, between the products of
  // the first two sub-steps: a wave that does it elsewhere keeps the matrix cores waiting.
  uint32_t poff[I];
  const unsigned char *qaddr[I];
  int qrow[I];                                      // the next stage's rows, or their choices
  auto ready_one = [&](int i) __attribute__((always_inline)) {
    const int left = li.rows - k_i * kKS;
    poff[i] = (local_row(i, h) < left ? hoff + (uint32_t)(wid * I + i) * RPI * ldp2 : 0u) + pc[i % NC];
    const int row = GATHER ? token_of(g, qrow[i]) : qrow[i];
    qaddr[i] = qbase + (uint64_t)(uint32_t)row * ldq2 + qc[i % NC];
  };
  auto fetch_one = [&](int i) __attribute__((always_inline)) {
    const bool in = local_row(i, h) < f_left;
    qrow[i] = in ? f_r0 + local_row(i, h) : 0;
    if constexpr (GATHER) {
      const int choice = g.sorted[qrow[i]];
      qrow[i] = in ? choice : 0;
    }
  };
  auto aim = [&](int t) __attribute__((always_inline)) {
    li = tile_of(t);
    int ln = l;                                     // (not computed ahead of the loop)
    asm volatile("" : "+v"(ln));
    const bool none = li.rows == 0;
    const bf16_t *const o = static_cast<const bf16_t *>(g.out);
    pbase = scalar_ptr(none ? o : g.P + (int64_t)li.r0 * g.ldp + li.m0);
    qbase = scalar_ptr(none ? o : g.Q + li.n0);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = ((ln % LPR) ^ chunk_xor<BM, false>(local_row(i, ln / LPR))) * 8;
      pc[i] = !none && li.m0 + c < M ? c * 2u : 0u;
      qc[i] = !none && li.n0 + c < N ? c * 2u : 0u;
    }
  };
  // the stage that follows the next one
  auto look = [&]() __attribute__((always_inline)) {
    if (k_i + 1 < li.stages) {
      f_r0 = li.r0 + (k_i + 1) * kKS;
      f_left = li.rows - (k_i + 1) * kKS;
    } else {
      const Tile n = t_i + stride < t_end ? tile_of(t_i + stride) : li;
      f_r0 = n.r0;
      f_left = n.rows;
    }
  };
  auto issue_one = [&](int q) __attribute__((always_inline)) {
    const uint32_t d = scalar_int(dst + b_i * STAGE);
    if (q < I)
      dma16_s(d, q * 1024, poff[q], scalar_ptr(pbase));
    else
      dma16(d, PB + (q - I) * 1024, qaddr[q - I]);
  };
  // The choices are there before loads are issued: the compiler's wait for them, at their
  // use, would count the loads and wait for those.
  auto settle = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < I; ++i) asm volatile("" : "+v"(qrow[i]));
  };
  // past a stage's loads
  auto advance = [&]() __attribute__((always_inline)) {
    b_i ^= 1;
    pbase += pstep;
    if (++k_i == li.stages) {
      k_i = 0;
      // past the last tile the loads go round on that one, unread
      if (t_i + stride < t_end) t_i += stride;
      aim(t_i);
    }
    look();
  };
  // a stage of `left` rows in buffer b: what this wave loaded past them to zero
  auto zero_tail = [&](int left, int b) {
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (local_row(i, h) >= left) {
        unsigned char *const p = smem + b * STAGE + (wid * I + i) * 1024 + l * 16;
        *reinterpret_cast<u32x4 *>(p) = u32x4{0, 0, 0, 0};
        *reinterpret_cast<u32x4 *>(p + PB) = u32x4{0, 0, 0, 0};
      }
  };

  FragmentReader<BM, false, WM> pr;
  FragmentReader<BN, false, WN> qr;
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
      qf[to][q] = qr.read(st + PB, q, kk);
    else
      pf[to][q - FN] = pr.read(st, q - FN, kk);
  };
  constexpr int NM = FM * FN, NR = FM + FN, SUBS = kKS / 16;
  auto sub_step = [&](auto k, const unsigned char *st) __attribute__((always_inline)) {
    constexpr int kk = decltype(k)::value;
    constexpr bool LOAD = kk == SUBS - 1;
    static_assert(NR <= NM && I <= NM, "one of each beside a product");
#pragma unroll
    for (int q = 0; q < (LOAD && 2 * I > NM ? 2 * I : NM); ++q) {
      if (q < NM) acc[q / FM][q % FM] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          qf[kk & 1][q / FM], pf[kk & 1][q % FM], acc[q / FM][q % FM], 0, 0, 0);
      if (q < NR) read((kk + 1) & 1, q, st, (kk + 1) % SUBS);
      if (kk == 0 && q < I) ready_one(q);
      if (kk == 1 && q < I) fetch_one(q);
      if (LOAD && q < 2 * I) issue_one(q);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto first_stages = [&]() __attribute__((always_inline)) {
    settle();
#pragma unroll
    for (int i = 0; i < I; ++i) ready_one(i);
#pragma unroll
    for (int i = 0; i < I; ++i) fetch_one(i);
    settle();
#pragma unroll
    for (int q = 0; q < 2 * I; ++q) issue_one(q);
    advance();
  };

  aim(t);
  f_r0 = li.r0;
  f_left = li.rows;
#pragma unroll
  for (int i = 0; i < I; ++i) fetch_one(i);
  look();
  Tile x = li;                                      // the tile being computed
  first_stages();
  vm_wait<0>();                                     // the first stage has landed
  if (x.rows < kKS) zero_tail(x.rows, 0);
  lgkm_barrier();
  first_stages();
#pragma unroll
  for (int q = 0; q < NR; ++q) read(0, q, smem, 0);
  zero_acc();
  int kt = 0, b = 0;
  while (true) {
    sub_step(std::integral_constant<int, 0>{}, smem + b * STAGE);
    sub_step(std::integral_constant<int, 1>{}, smem + b * STAGE);
    sub_step(std::integral_constant<int, 2>{}, smem + b * STAGE);
    const bool last = kt + 1 == x.stages;
    const Tile done = x;
    if (last && t + stride < t_end) x = tile_of(t + stride);
    kt = last ? 0 : kt + 1;                         // the next stage, of x
    pin();
    vm_wait<0>();                                   // it has landed
    settle();
    if ((kt + 1) * kKS > x.rows) zero_tail(x.rows - kt * kKS, b ^ 1);
    lgkm_barrier();                                 // it is there, and this one has been read
    __builtin_amdgcn_s_setprio(1);
    sub_step(std::integral_constant<int, 3>{}, smem + (b ^ 1) * STAGE);
    __builtin_amdgcn_s_setprio(0);
    pin();
    advance();
    b ^= 1;
    if (!last) continue;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int row = done.m0 + (wm * FM + i) * 32, col = done.n0 + (wn * FN + j) * 32;
        const int64_t at = done.e * g.w_stride + (int64_t)row * g.ldo + col;
        unsigned char *const lds = smem + kRing * STAGE + kExpertTab + wid * 2048;
        if constexpr (F32OUT)
          store_fragment<true, true>(lds, acc[j][i], l, static_cast<float *>(g.out) + at, g.ldo,
                                     M - row, N - col, g.accumulate);
        else if (g.accumulate)
          store_fragment<false, true>(lds, acc[j][i], l, static_cast<bf16_t *>(g.out) + at, g.ldo,
                                      M - row, N - col, true);
        else
          store_fragment<false, false>(lds, acc[j][i], l, static_cast<bf16_t *>(g.out) + at, g.ldo,
                                       M - row, N - col, false);
      }
    t += stride;
    if (t >= t_end) break;
    zero_acc();
    pin();
  }
  vm_wait<0>();                                     // no load outlives the workgroup's LDS
}

template <bool F32OUT, bool GATHER> void launch_weights(const ExpertGemmArgs &g, hipStream_t stream) {
  if (experts_weights_large(g.M, g.N, g.n_experts))
    hipLaunchKernelGGL((experts_weights_kernel<256, 256, 2, 4, 1, F32OUT, GATHER>), dim3(kCUs), dim3(512),
                       0, stream, g);
  else
    hipLaunchKernelGGL((experts_weights_kernel<128, 128, 2, 2, 2, F32OUT, GATHER>), dim3(kCUs * 2),
                       dim3(256), 0, stream, g);
}

}  // namespace

hipError_t launch_experts_gemm_weights(const void *dY, int64_t lddy, const void *X, int64_t ldx,
                                       const ExpertView &ex, void *dW, int64_t lddw, int dtype,
                                       bool accumulate, int M, int N, hipStream_t stream) {
  ExpertGemmArgs g = expert_args(dY, lddy, X, ldx, dW, lddw, M, N, 0, ex);
  g.accumulate = accumulate;
  // (without choices there is no first one to read)
  const bool gather = ex.sorted_choice && ex.n_choices > 0;
  if (dtype == LORA_F32)
    gather ? launch_weights<true, true>(g, stream) : launch_weights<true, false>(g, stream);
  else
    gather ? launch_weights<false, true>(g, stream) : launch_weights<false, false>(g, stream);
  return hipGetLastError();
}

}  // namespace lora
