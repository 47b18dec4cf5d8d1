// Launches of the base product with a bf16 or FP8 weight (the MFMA tiles of
// gemm_tile.cuh) and of the fp32 product (VALU tiles, below).
#include "gemm_tile.cuh"

namespace lora {
namespace {

// ----------------------------------------------------------------------------
// fp32: plain VALU tiles (64 x 64 per block, 4 x 4 per thread) through LDS;
// the fused increment is a direct sum over k < r per output element.
// ----------------------------------------------------------------------------
struct GemmF32Args {
  const float *X;
  int64_t ldx;
  const float *W;
  int64_t ldw;
  float *Y;
  int64_t ldy;
  int M, K, N;
  const float *H;
  const float *Bt;
  const int32_t *row_segment, *seg_slot, *seg_rank;
  const float *seg_scale;
  int r_max;
  const float *dora;
  ProjView proj;
};

template <bool LORA>
__global__ __launch_bounds__(256) void gemm_f32_kernel(GemmF32Args g) {
  constexpr int BMF = 64, BNF = 64, BKF = 16;
  __shared__ float sA[BKF][BMF + 4];
  __shared__ float sB[BKF][BNF + 4];
  const int tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;
  const int m0 = blockIdx.y * BMF, n0 = blockIdx.x * BNF;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += BKF) {
    {
      const int row = tid >> 2, kq = (tid & 3) * 4;
      const int gm = m0 + row, gk = k0 + kq;
      float4 va = make_float4(0.f, 0.f, 0.f, 0.f), vb = va;
      if (gm < g.M && gk < g.K) va = *reinterpret_cast<const float4 *>(g.X + (int64_t)gm * g.ldx + gk);
      const int gn = n0 + row;
      if (gn < g.N && gk < g.K) vb = *reinterpret_cast<const float4 *>(g.W + (int64_t)gn * g.ldw + gk);
      sA[kq + 0][row] = va.x; sA[kq + 1][row] = va.y; sA[kq + 2][row] = va.z; sA[kq + 3][row] = va.w;
      sB[kq + 0][row] = vb.x; sB[kq + 1][row] = vb.y; sB[kq + 2][row] = vb.z; sB[kq + 3][row] = vb.w;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < BKF; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = sA[kk][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = sB[kk][tx * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = m0 + ty * 4 + i;
    if (row >= g.M) continue;
    if constexpr (LORA) {
      const int s = g.row_segment[row];
      const int r = g.seg_rank[s];
      if (r > 0) {
        const float sc = g.seg_scale[s];
        const float *hrow = g.H + (int64_t)row * g.r_max;
        const float *bt = g.Bt + (int64_t)g.seg_slot[s] * g.proj.rs * g.N;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = n0 + tx * 4 + j;
          if (col >= g.N) continue;
          const int qoff = proj_of(g.proj, col) * g.proj.rs;
          float d = 0.f;
          for (int k = 0; k < r; ++k)
            d = fmaf(hrow[qoff + k], bt[(int64_t)k * g.N + col], d);
          acc[i][j] += sc * d;
          if (g.dora) acc[i][j] *= g.dora[(int64_t)g.seg_slot[s] * g.N + col];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int col = n0 + tx * 4 + j;
      if (col < g.N) g.Y[(int64_t)row * g.ldy + col] = acc[i][j];
    }
  }
}

template <int BM, int BN, int WM, int WN, int BK, int STAGES, int KG>
hipError_t launch_bf16(const GemmArgs &g, bool lora, hipStream_t stream) {
  return launch_tile<BM, BN, WM, WN, BK, STAGES, KG, kBf16>(g, lora, stream);
}
template <int BM, int BN, int WM, int WN, int BK, int STAGES, int KG>
hipError_t launch_fp8w(const GemmArgs &g, bool lora, hipStream_t stream) {
  return launch_tile<BM, BN, WM, WN, BK, STAGES, KG, kFp8W>(g, lora, stream);
}

// The one-launch layer on small tiles: one workgroup per tile, and at least
// one per row (workgroups past the tiles only do their row).
template <int WQ, int BM, int BN, int WM, int WN, int BK, int STAGES, int KG>
hipError_t launch_layer_t(const GemmArgs &g, hipStream_t stream) {
  const int tiles = tile_grid((g.M + BM - 1) / BM, (g.N + BN - 1) / BN);
  dim3 grid(tiles > g.M ? tiles : g.M);
  dim3 block(WM * WN * KG * kWave);
  if (g.dora)
    hipLaunchKernelGGL((gemm_bf16_kernel<BM, BN, WM, WN, BK, STAGES, KG, 1, true, WQ, true>),
                       grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((gemm_bf16_kernel<BM, BN, WM, WN, BK, STAGES, KG, 1, false, WQ, true>),
                       grid, block, 0, stream, g);
  return hipGetLastError();
}

// Tile configuration for a batch of g.M rows, and the launch.
hipError_t launch_bf16_rows(const GemmArgs &g, bool lora, hipStream_t stream) {
  const int M = g.M, N = g.N;
  const bool mid = mid_tiles(M, N), use192 = large192_tiles(M, N);
  if (g.wscale) {
    if (M <= LORA_GEMM_SMALL_M) return launch_fp8w<LORA_GEMM_SMALL_F8>(g, lora, stream);
    if (mid) return launch_fp8w<LORA_GEMM_MID_F8>(g, lora, stream);
    if (use192) return launch_fp8w<LORA_GEMM_LARGE192_F8>(g, lora, stream);
    return launch_fp8w<LORA_GEMM_LARGE_F8>(g, lora, stream);
  }
  if (M <= LORA_GEMM_SMALL_M) {
    using S = TileCfg<LORA_GEMM_SMALL>;
    const int64_t tiles = (int64_t)((M + S::kBM - 1) / S::kBM) * ((N + S::kBN - 1) / S::kBN);
    if (tiles > kCUs) return launch_bf16<LORA_GEMM_SMALL_WIDE>(g, lora, stream);
    return launch_bf16<LORA_GEMM_SMALL>(g, lora, stream);
  }
  if (mid) return launch_bf16<LORA_GEMM_MID>(g, lora, stream);
  if (use192) return launch_bf16<LORA_GEMM_LARGE192>(g, lora, stream);
  return launch_bf16<LORA_GEMM_LARGE>(g, lora, stream);
}

}  // namespace

hipError_t launch_gemm(const void *X, int64_t ldx, const void *W, int64_t ldw, void *Y,
                       int64_t ldy, int M, int K, int N, int dtype, const float *H,
                       const SegView *seg, const PoolView *pool, hipStream_t stream,
                       const float *wscale) {
  const bool lora = seg != nullptr;
  if (dtype == 1) {
    GemmArgs g = gemm_args(X, ldx, W, ldw, Y, ldy, M, K, N, H, seg, pool);
    g.wscale = wscale;
    return launch_rows_split(
        g, lora, [&](const GemmArgs &a) { return launch_bf16_rows(a, lora, stream); });
  }
  GemmF32Args g{(const float *)X, ldx, (const float *)W, ldw, (float *)Y, ldy, M, K, N,
                H, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr};
  g.proj.n_proj = 1;
  g.proj.rs = 64;
  for (int q = 0; q <= kMaxProj; ++q) g.proj.col_off[q] = q ? N : 0;
  if (lora) {
    g.proj = pool->proj;
    g.Bt = (const float *)pool->Bt;
    g.dora = pool->dora;
    g.row_segment = seg->row_segment;
    g.seg_slot = seg->seg_slot;
    g.seg_rank = seg->seg_rank;
    g.seg_scale = seg->seg_scale;
    g.r_max = pool->r_max;
  }
  dim3 grid((N + 63) / 64, (M + 63) / 64);
  if (lora)
    hipLaunchKernelGGL(gemm_f32_kernel<true>, grid, dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL(gemm_f32_kernel<false>, grid, dim3(256), 0, stream, g);
  return hipGetLastError();
}

hipError_t launch_layer(const void *X, int64_t ldx, const void *W, int64_t ldw, void *Y,
                        int64_t ldy, int M, const PoolView &pool, const LayerArgs &lay,
                        hipStream_t stream, const float *wscale) {
  if (pool.dtype != 1 || M < 1 || M > kLayerMaxRows) return hipErrorNotSupported;
  const int K = pool.d_in, N = pool.d_out;
  GemmArgs g{};
  g.X = (const bf16_t *)X;
  g.ldx = ldx;
  g.W = (const bf16_t *)W;
  g.ldw = ldw;
  g.Y = (bf16_t *)Y;
  g.ldy = ldy;
  g.M = M;
  g.K = K;
  g.N = N;
  g.H = lay.H;
  g.wscale = wscale;
  g.proj = pool.proj;
  g.Bt = (const bf16_t *)pool.Bt;
  g.Bn = (const bf16_t *)pool.B;
  g.dora = pool.dora;
  g.r_max = pool.r_max;
  g.policy = pool.policy;
  g.lay = lay;
  using S = TileCfg<LORA_GEMM_SMALL>;
  const int64_t tiles = (int64_t)((M + S::kBM - 1) / S::kBM) * ((N + S::kBN - 1) / S::kBN);
  // FP8 weights: the four-stage ring only (the two-stage ring of codes is
  // too small to hold a large pool's build tables)
  if (wscale) return launch_layer_t<kFp8W, LORA_GEMM_SMALL_F8>(g, stream);
  if (tiles > kCUs) return launch_layer_t<kBf16, LORA_GEMM_SMALL_WIDE>(g, stream);
  return launch_layer_t<kBf16, LORA_GEMM_SMALL>(g, stream);
}

}  // namespace lora
