// Products of up to 16 rows with an MXFP4 weight: Y = X dq(W)^T for small decode
// batches, and the experts' decode products (a few rows on each expert's weight).
//
// Bound by reading W (17/32 byte a weight) from HBM, so W goes from memory
// straight to registers: a workgroup takes NT tiles of W rows, its KW waves every
// KW-th 256 codes of K, and their sums meet in LDS at the end.  A block of 32
// codes is a lane's 16 bytes; it feeds four v_mfma_f32_16x16x32_bf16 with 8 codes
// each widened to bf16 under the block's scale (exact), and the K order inside
// is the same permutation for X, whose rows are the MFMA's columns.
//
// KP 1: a tile is 16 rows of W and up to 16 of X; a load takes 64 bytes of each
// W row, half of its 128-byte line, and the next load the other half.
// KP 2: up to 8 rows of X, whose columns the MFMA has twice over.  A tile is 8
// rows of W, a load takes their whole 128-byte lines: the MFMA's rows (and
// columns) 0 to 7 are the tile's (and X's) rows at the first 128 codes of K, 8 to
// 15 the same rows at the next 128; D[r][m] + D[r + 8][m + 8] is the sum, and the
// mixed quarters go unused.
// The next loads are issued before a load's products; registers for two
// workgroups of eight waves on a CU.
//
// 1 x 8192 -> 28672 (125 MB): 28.4 us, 4.4 TB/s (KP 1: 35.4, as W's rows, a power of
// two apart, share few cache sets and the second half of a line was often fetched
// again).  Non-temporal loads of W, which lose half lines: 41 us with KP 1.  64 x 8
// choices on 128 experts of 2048 -> 1536 (212 MB): 56 to 58 us.
#pragma once

#include "gemm_tile.cuh"

namespace lora {
namespace {

template <int NT>
struct StreamLoad {
  u32x4 w[NT], x[4];
  uint32_t sc[NT];
};

template <int NT, int KW, int KP, bool GROUPED, bool LORA, bool DORA>
__global__ __launch_bounds__(KW *kWave, 4) void mx_stream_kernel(GemmArgs g) {
  constexpr int T = KW * kWave, RW = 16 / KP, BN = RW * NT, BM = 16 / KP;
  static_assert(KP == 1 || KP == 2, "K parts");
  __shared__ __align__(16) float red[KW][NT][kWave * 4];
  const int tid = threadIdx.x, l = tid & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int N = g.N, K = g.K;
  int m0 = 0, m1 = g.M, n_idx = blockIdx.x;
  const unsigned char *W = reinterpret_cast<const unsigned char *>(g.W), *SW = g.mx.w;
  if constexpr (GROUPED) {
    const int tiles_n = (N + BN - 1) / BN;
    int *s = reinterpret_cast<int *>(red);
    const ExpertTiles et = expert_tiles<BM, T>(g.ex, s);
    if ((int)blockIdx.x >= et.total * tiles_n) return;
    int e;
    n_idx = blockIdx.x % tiles_n;
    expert_of_tile<BM, T>(g.ex, et, blockIdx.x / tiles_n, s, e, m0, m1);
    W += (int64_t)e * g.ex.w_stride;
    SW += (int64_t)e * g.ex.s_stride;
  }
  const int n0 = n_idx * BN;
  const int rows = min(m1 - m0, BM);

  // this lane's W rows and X rows (rows past the ends read the last one), from
  // its block of a load's K on
  const int rw = l & (RW - 1), kp = (l & 15) / RW, gq = l >> 4, kb = kp * 128 + gq * 32;
  const unsigned char *const wb = W + (int64_t)n0 * (g.ldw / 2), *const sb = SW + (int64_t)n0 * g.mx.ldw;
  uint32_t wo[NT], so[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint32_t row = min(j * RW + rw, N - 1 - n0);
    wo[j] = row * (uint32_t)(g.ldw / 2) + kb / 2;
    so[j] = row * (uint32_t)g.mx.ldw;
  }
  const int p0 = m0 + min(rw, rows - 1);
  const int x_row = GROUPED && g.ex.sorted_choice ? g.ex.sorted_choice[p0] / g.ex.top_k : p0;
  const bf16_t *const xp = g.X + (int64_t)x_row * g.ldx + kb;
  const int steps = (K + 255) / 256, last_word = (K / 32 - 1) / 4;
  const int mine = (steps - wid + KW - 1) / KW;     // steps of this wave (negative: none)
  const int loads = KP == 1 ? 2 * mine : mine;
  auto k_of = [&](int p) { return KP == 1 ? ((p >> 1) * KW + wid) * 256 + (p & 1) * 128 : (p * KW + wid) * 256; };
  // blocks past K read their row's start, their X is zeroed and their scale 1 (a
  // NaN would spoil the zeros)
  auto load = [&](StreamLoad<NT> &t, int p) __attribute__((always_inline)) {
    const int k = k_of(p);
    const bool in = k + kb < K;
    const int kx = in ? k : -kb;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      t.w[j] = *reinterpret_cast<const u32x4 *>(wb + (wo[j] + (uint32_t)(kx / 2)));
      t.sc[j] = *reinterpret_cast<const uint32_t *>(sb + (so[j] + 4 * (uint32_t)min(k / 128 + kp, last_word)));
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const u32x4 v = *reinterpret_cast<const u32x4 *>(xp + kx + kk * 8);
      t.x[kk] = in ? v : u32x4{0, 0, 0, 0};
    }
  };
  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const StreamLoad<NT> &t, int p) __attribute__((always_inline)) {
    const bool in = k_of(p) + kb < K;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float f = in ? __uint_as_float((t.sc[j] >> (gq * 8) & 0xffu) << 23) : 1.f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const mfma_bf16x8 w = fp4x8_to_bf16x8(t.w[j][kk], f);
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, as_bf16x8(t.x[kk]), acc[j], 0, 0, 0);
      }
    }
  };

  StreamLoad<NT> a, b;
  if (loads > 0) load(a, 0);
  for (int p = 0; p < loads; p += 2) {
    if (p + 1 < loads) load(b, p + 1);
    multiply(a, p);
    if (p + 2 < loads) load(a, p + 2);
    if (p + 1 < loads) multiply(b, p + 1);
  }

  // the waves' sums: slot (j, lane) holds W rows [4 (lane / 16), +4) of the MFMA's
  // 16 and its column lane % 16
#pragma unroll
  for (int j = 0; j < NT; ++j) *reinterpret_cast<f32x4 *>(&red[wid][j][l * 4]) = acc[j];
  __syncthreads();
  // a thread finishes 8 columns of one row
  for (int q = tid; q < NT * BM * (RW / 8); q += T) {
    const int r = q % BM, h = q / BM % (RW / 8), j = q / (BM * (RW / 8));
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < KW; ++w)
#pragma unroll
      for (int c = 0; c < KP; ++c) {
        const int at = r + c * BM + 16 * (c * (4 / KP) + 2 * h);
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(&red[w][j][at * 4]);
        const f32x4 hi = *reinterpret_cast<const f32x4 *>(&red[w][j][(at + 16) * 4]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] += lo[e];
          o[4 + e] += hi[e];
        }
      }
    const int row = m0 + r, col = n0 + j * RW + h * 8;
    if (r < rows && col < N) {                      // N % 8 == 0: all 8 columns or none
      if constexpr (LORA) {
        const int sg = g.row_segment[row], rank = g.seg_rank[sg];
        if (rank > 0) lora_row8<DORA>(g, row, col, g.seg_slot[sg], rank, g.seg_scale[sg], o);
      }
      stg16(g.Y + (int64_t)row * g.ldy + col, Elem<bf16_t>::pack(o));
    }
  }
}

template <int NT, int KW, int KP>
hipError_t launch_stream(const GemmArgs &g, bool lora, hipStream_t stream) {
  constexpr int BN = 16 / KP * NT;
  const dim3 grid((g.N + BN - 1) / BN), block(KW * kWave);
  if (lora && g.dora)
    hipLaunchKernelGGL((mx_stream_kernel<NT, KW, KP, false, true, true>), grid, block, 0, stream, g);
  else if (lora)
    hipLaunchKernelGGL((mx_stream_kernel<NT, KW, KP, false, true, false>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((mx_stream_kernel<NT, KW, KP, false, false, false>), grid, block, 0, stream, g);
  return hipGetLastError();
}

inline hipError_t launch_mx_stream(const GemmArgs &g, MxKernel k, bool lora, hipStream_t stream) {
  // (kMxStream16: N below 64 kCUs / 2, where one tile of 16 a workgroup gives no more
  // than two workgroups to a CU)
  if (k == kMxStream16) return launch_stream<1, 8, 1>(g, lora, stream);
  const int tiles = mx_stream8_tiles(g.N);
  if (tiles == 4) return launch_stream<4, 8, 2>(g, lora, stream);
  if (tiles == 2) return launch_stream<2, 8, 2>(g, lora, stream);
  return launch_stream<1, 8, 2>(g, lora, stream);
}

template <int NT, int KP>
hipError_t launch_experts_stream(const GemmArgs &g, int tiles_m, hipStream_t stream) {
  constexpr int BN = 16 / KP * NT;
  const int64_t tn = (g.N + BN - 1) / BN;
  hipLaunchKernelGGL((mx_stream_kernel<NT, 4, KP, true, false, false>), dim3((unsigned)(tn * tiles_m)),
                     dim3(4 * kWave), 0, stream, g);
  return hipGetLastError();
}

}  // namespace
}  // namespace lora
