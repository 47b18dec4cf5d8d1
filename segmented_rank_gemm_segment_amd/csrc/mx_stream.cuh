// Products of few rows with an MXFP4 weight: Y = X dq(W)^T for decode batches,
// and for the experts' decode products (a few rows on each expert's weight).
//
// Bound by reading W (17/32 byte a weight) from HBM, so W goes from memory
// straight to registers and each byte is read once: a workgroup takes 16 NT rows
// of W, its KW waves every KW-th 256 codes of K, and their sums meet in LDS at
// the end.  A wave works in half steps of 128 codes: lane l holds row l % 16 of
// each 16-row tile and block l / 16 of the half step's four 32-code blocks (16
// bytes, one scale); the two half steps of a row make whole 128-byte lines.  A
// block feeds four v_mfma_f32_16x16x32_bf16 with 8 codes widened to bf16 under
// its scale (exact); the K order inside is the same permutation for X, whose
// rows are the MFMA's columns: 16 MT of them.  A half step's loads are issued
// before the products of the one before it; registers for two workgroups of
// eight waves on a CU.
//
// 1 x 8192 -> 28672 (125 MB): 35.4 us, 3.5 TB/s; 28 us where W's rows are not a
// power of two apart (such rows share few cache sets, so the second half of a
// line is often fetched again).  64 x 8 choices on 128 experts of 2048 -> 1536
// (212 MB): 58 us.  Non-temporal loads of W lose the half lines: 41 us.
#pragma once

#include "gemm_tile.cuh"

namespace lora {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int NT, int MT>
struct StreamHalf {
  u32x4 w[NT], x[MT][4];
};

template <int NT, int KW, int MT, bool GROUPED, bool LORA, bool DORA>
__global__ __launch_bounds__(KW *kWave, MT == 1 ? 4 : 2) void mx_stream_kernel(GemmArgs g) {
  constexpr int T = KW * kWave, BN = 16 * NT, BM = 16 * MT;
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
  const int rows = min(m1 - m0, BM), parts = (rows + 15) / 16;

  // this lane's W rows and X row (rows past the ends read the last one)
  const int r16 = l & 15, gq = l >> 4;
  const unsigned char *wp[NT], *sp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int row = min(n0 + j * 16 + r16, N - 1);
    wp[j] = W + (int64_t)row * (g.ldw / 2) + gq * 16;
    sp[j] = SW + (int64_t)row * g.mx.ldw;
  }
  const bf16_t *xp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int p = m0 + min(i * 16 + r16, rows - 1);
    const int row = GROUPED && g.ex.sorted_choice ? g.ex.sorted_choice[p] / g.ex.top_k : p;
    xp[i] = g.X + (int64_t)row * g.ldx + gq * 32;
  }
  const int steps = (K + 255) / 256, last_word = (K / 32 - 1) / 4;
  // half step b of step s: blocks past K read their row's start, their X is
  // zeroed and their scale 1 (a NaN would spoil the zeros)
  auto load = [&](StreamHalf<NT, MT> &t, int s, int b) __attribute__((always_inline)) {
    const int k = s * 256 + b * 128;
    const bool in = k + gq * 32 < K;
    const int kx = in ? k : -gq * 32;
#pragma unroll
    for (int j = 0; j < NT; ++j) t.w[j] = *reinterpret_cast<const u32x4 *>(wp[j] + kx / 2);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const u32x4 v = *reinterpret_cast<const u32x4 *>(xp[i] + kx + kk * 8);
        t.x[i][kk] = in ? v : u32x4{0, 0, 0, 0};
      }
  };
  auto load_scales = [&](u32x2 (&sc)[NT], int s) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        sc[j][b] = *reinterpret_cast<const uint32_t *>(sp[j] + min(s * 2 + b, last_word) * 4);
  };
  f32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const StreamHalf<NT, MT> &t, const u32x2 (&sc)[NT], int s, int b)
                      __attribute__((always_inline)) {
    const bool in = s * 256 + b * 128 + gq * 32 < K;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float f = in ? __uint_as_float((sc[j][b] >> (gq * 8) & 0xffu) << 23) : 1.f;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const mfma_bf16x8 w = fp4x8_to_bf16x8(t.w[j][kk], f);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, as_bf16x8(t.x[i][kk]), acc[j][i], 0, 0, 0);
      }
    }
  };

  StreamHalf<NT, MT> h0, h1;
  u32x2 sc0[NT], sc1[NT];
  int s = wid;
  if (s < steps) {
    load_scales(sc0, s);
    load(h0, s, 0);
  }
  for (; s < steps; s += KW) {
    load(h1, s, 1);
    multiply(h0, sc0, s, 0);
    const bool more = s + KW < steps;
    if (more) {
      load_scales(sc1, s + KW);
      load(h0, s + KW, 0);
    }
    multiply(h1, sc0, s, 1);
    if (more)
#pragma unroll
      for (int j = 0; j < NT; ++j) sc0[j] = sc1[j];
  }

  // the waves' sums, 16 rows of X at a time: slot (j, lane) holds columns
  // [16 j + 4 (lane / 16), +4) of row lane % 16
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i >= parts) break;
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4 *>(&red[wid][j][l * 4]) = acc[j][i];
    __syncthreads();
    // a thread finishes 8 columns: two neighbouring slots
    for (int q = tid; q < NT * 32; q += T) {
      const int j = q / 32, r = q % 16, h = q / 16 % 2;
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(&red[w][j][(r + 32 * h) * 4]);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(&red[w][j][(r + 32 * h + 16) * 4]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] += a[e];
          o[4 + e] += b[e];
        }
      }
      const int row = m0 + i * 16 + r, col = n0 + j * 16 + h * 8;
      if (row < m1 && i * 16 + r < rows && col < N) {   // N % 8 == 0: all 8 columns or none
        if constexpr (LORA) {
          const int sg = g.row_segment[row], rank = g.seg_rank[sg];
          if (rank > 0) lora_row8<DORA>(g, row, col, g.seg_slot[sg], rank, g.seg_scale[sg], o);
        }
        stg16(g.Y + (int64_t)row * g.ldy + col, Elem<bf16_t>::pack(o));
      }
    }
    if (i + 1 < parts) __syncthreads();
  }
}

template <int NT, int KW, int MT>
hipError_t launch_stream(const GemmArgs &g, bool lora, hipStream_t stream) {
  const dim3 grid((g.N + 16 * NT - 1) / (16 * NT)), block(KW * kWave);
  if (lora && g.dora)
    hipLaunchKernelGGL((mx_stream_kernel<NT, KW, MT, false, true, true>), grid, block, 0, stream, g);
  else if (lora)
    hipLaunchKernelGGL((mx_stream_kernel<NT, KW, MT, false, true, false>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((mx_stream_kernel<NT, KW, MT, false, false, false>), grid, block, 0, stream, g);
  return hipGetLastError();
}

// Most rows of a dense batch that the kernel takes.
constexpr int kStreamRows = 32;

inline hipError_t launch_mx_stream(const GemmArgs &g, bool lora, hipStream_t stream) {
  // the widest workgroups that still give every CU one
  const int nt = (g.N + 63) / 64 >= kCUs ? 4 : (g.N + 31) / 32 >= kCUs ? 2 : 1;
  if (g.M <= 16)
    return nt == 4   ? launch_stream<4, 8, 1>(g, lora, stream)
           : nt == 2 ? launch_stream<2, 8, 1>(g, lora, stream)
                     : launch_stream<1, 8, 1>(g, lora, stream);
  return nt == 4   ? launch_stream<4, 8, 2>(g, lora, stream)
         : nt == 2 ? launch_stream<2, 8, 2>(g, lora, stream)
                   : launch_stream<1, 8, 2>(g, lora, stream);
}

inline hipError_t launch_experts_stream(const GemmArgs &g, int tiles_m, hipStream_t stream) {
  const int64_t tn = (g.N + 63) / 64;
  hipLaunchKernelGGL((mx_stream_kernel<4, 4, 1, true, false, false>), dim3((unsigned)(tn * tiles_m)),
                     dim3(4 * kWave), 0, stream, g);
  return hipGetLastError();
}

}  // namespace
}  // namespace lora
