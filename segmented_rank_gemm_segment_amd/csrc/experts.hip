// Expert routing: the batch's token choices sorted by expert, rows moved into
// that order and combined back with the router's weights, and the gradients.
//
// Sort: a counting sort, stable, with no float and no atomic whose order could
// show.  A wave ranks its 64 choices against each other with one ballot per key
// bit; per-wave counts in LDS give each wave its base, and a scan over the
// experts each expert its first row.  Up to kExpertOneGroupChoices choices one
// workgroup does it all; larger batches count per block of kBlockChoices, scan
// the blocks' counts, and place.
//
// Rows move in token order (gather, combine and its backward alike): a token's
// row is read once and its top_k sorted rows are written or read beside it, so
// each array passes HBM once.  All three are bound by HBM: 16 bytes per lane,
// four waves per token.
#include "lora_device.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kMaxE = LORA_MAX_EXPERTS;
static_assert(kMaxE <= kSortThreads, "one expert per thread in the scans");
constexpr int kOneGroupSteps = kExpertOneGroupChoices / kSortThreads;
constexpr int kBlockChoices = kExpertBlockChoices, kBlockSteps = kBlockChoices / kSortThreads;

constexpr int kScanBlocks = 64;

struct SortArgs {
  const int32_t *ids;
  int n, E;            // choices, experts
  int32_t *offsets, *sorted, *position, *status;
  int32_t *counts;     // [blocks][E + 1], the last entry: choices with a bad id
};

// Exclusive sum over the workgroup's threads, and the total; s: kSortWaves words.
__device__ __forceinline__ int block_scan(int v, int *s, int &total) {
  int inc = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int x = __shfl_up(inc, o);
    inc += (int)(threadIdx.x % kWave) >= o ? x : 0;
  }
  if (threadIdx.x % kWave == kWave - 1) s[threadIdx.x / kWave] = inc;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    before += w < (int)threadIdx.x / kWave ? s[w] : 0;
    total += s[w];
  }
  return before + inc - v;
}

struct SortLds {
  int cnt[kSortWaves * kMaxE];   // per wave and expert
  int off[kMaxE];
  int scan[kSortWaves];
  int bad;
};

// The workgroup's choices [base, base + STEPS kSortThreads), wave w's the w-th
// part of them in order.  On return key/rank hold each choice's expert (-1:
// none) and its rank among the wave's choices of that expert, L.cnt[w][e] how
// many wave w has, and L.bad the ids that are neither -1 nor an expert.
template <int STEPS>
__device__ __forceinline__ void rank_choices(const SortArgs &a, int base, SortLds &L,
                                             int (&key)[STEPS], int (&rank)[STEPS]) {
  const int l = lane_id(), w = threadIdx.x / kWave;
  const int first = base + w * STEPS * kWave + l;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = first + s * kWave;
    key[s] = c < a.n ? a.ids[c] : -1;
  }
  for (int i = threadIdx.x; i < kSortWaves * a.E; i += kSortThreads) L.cnt[i] = 0;
  if (threadIdx.x == 0) L.bad = 0;
  __syncthreads();
  const int bits = 32 - __clz(a.E - 1 | 1);
  volatile int *cnt = L.cnt + w * a.E;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const bool ok = (unsigned)key[s] < (unsigned)a.E;
    const uint64_t wrong = __ballot(!ok && key[s] != -1);
    if (wrong && l == 0) atomicAdd(&L.bad, (int)__popcll(wrong));
    if (!ok) key[s] = -1;
    uint64_t same = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(key[s] >> b & 1);
      same &= (key[s] >> b & 1) ? set : ~set;
    }
    const int r = (int)__popcll(same & lanemask_lt());
    if (ok) {
      const int old = cnt[key[s]];
      rank[s] = old + r;
      __builtin_amdgcn_wave_barrier();
      if (r == 0) cnt[key[s]] = old + (int)__popcll(same);
      __builtin_amdgcn_wave_barrier();
    }
  }
  __syncthreads();
}

// L.cnt[w][e] to the number of earlier waves' choices of e; returns thread
// e's expert's total.
__device__ __forceinline__ int wave_bases(int E, SortLds &L) {
  int run = 0;
  if ((int)threadIdx.x < E)
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int v = L.cnt[w * E + threadIdx.x];
      L.cnt[w * E + threadIdx.x] = run;
      run += v;
    }
  return run;
}

template <int STEPS>
__device__ __forceinline__ void place(const SortArgs &a, int base, const SortLds &L,
                                      const int (&key)[STEPS], const int (&rank)[STEPS]) {
  const int w = threadIdx.x / kWave, first = base + w * STEPS * kWave + lane_id();
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = first + s * kWave;
    if (c >= a.n) continue;
    const int p = key[s] < 0 ? -1 : L.off[key[s]] + L.cnt[w * a.E + key[s]] + rank[s];
    a.position[c] = p;
    if (p >= 0) a.sorted[p] = c;
  }
}

// One workgroup, STEPS kSortThreads choices at most.
template <int STEPS>
__global__ __launch_bounds__(kSortThreads) void sort_one_kernel(SortArgs a) {
  __shared__ SortLds L;
  int key[STEPS], rank[STEPS], total;
  rank_choices<STEPS>(a, 0, L, key, rank);
  const int mine = wave_bases(a.E, L);
  const int at = block_scan(mine, L.scan, total);
  if ((int)threadIdx.x < a.E) {
    L.off[threadIdx.x] = at;
    a.offsets[threadIdx.x] = at;
  }
  if (threadIdx.x == 0) {
    a.offsets[a.E] = total;
    *a.status = L.bad;
  }
  __syncthreads();
  place<STEPS>(a, 0, L, key, rank);
}

// Block b's choices of each expert.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int hist[kMaxE + 1];
  for (int e = threadIdx.x; e <= a.E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int base = blockIdx.x * kBlockChoices;
#pragma unroll
  for (int s = 0; s < kBlockSteps; ++s) {
    const int c = base + s * kSortThreads + threadIdx.x;
    const int k = c < a.n ? a.ids[c] : -1;
    if (k != -1) atomicAdd(&hist[(unsigned)k < (unsigned)a.E ? k : a.E], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += kSortThreads)
    a.counts[(int64_t)blockIdx.x * (a.E + 1) + e] = hist[e];
}

// The blocks' counts to their prefix sums, and the experts' first rows.
__global__ __launch_bounds__(kSortThreads) void sort_scan_kernel(SortArgs a, int blocks) {
  __shared__ int s[kSortWaves];
  int run = 0, total;
  for (int e = threadIdx.x; e <= a.E; e += kSortThreads) {   // e > 1023 only for the bad ids
    int32_t *p = a.counts + e;
    int sum = 0;
    for (int b = 0; b < blocks; ++b, p += a.E + 1) {
      const int v = *p;
      *p = sum;
      sum += v;
    }
    if (e == a.E) *a.status = sum;
    if (e < a.E) run = sum;
  }
  const int at = block_scan(run, s, total);
  if ((int)threadIdx.x < a.E) a.offsets[threadIdx.x] = at;
  if (threadIdx.x == 0) a.offsets[a.E] = total;
}

// The block's choices to their places.  SCAN: the counts are still per block;
// every workgroup sums them itself, and the first writes the experts' rows.
template <bool SCAN>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ SortLds L;
  int key[kBlockSteps], rank[kBlockSteps];
  const int base = blockIdx.x * kBlockChoices;
  const int e = threadIdx.x;
  int before = 0, all = 0, bad = 0;
  if constexpr (SCAN) {
    for (int b = 0; b < (int)gridDim.x; ++b) {
      const int32_t *c = a.counts + b * (a.E + 1);
      const int v = e < a.E ? c[e] : 0;
      before += b < (int)blockIdx.x ? v : 0;
      all += v;
      bad += c[a.E];
    }
  }
  rank_choices<kBlockSteps>(a, base, L, key, rank);
  wave_bases(a.E, L);
  if constexpr (SCAN) {
    int total;
    const int at = block_scan(all, L.scan, total);
    if (e < a.E) L.off[e] = at + before;
    if (blockIdx.x == 0) {
      if (e < a.E) a.offsets[e] = at;
      if (e == 0) {
        a.offsets[a.E] = total;
        *a.status = bad;
      }
    }
  } else if (e < a.E) {
    L.off[e] = a.offsets[e] + a.counts[(int64_t)blockIdx.x * (a.E + 1) + e];
  }
  __syncthreads();
  place<kBlockSteps>(a, base, L, key, rank);
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
struct RowArgs {
  int n, k, d;               // n: one past the launch's last token
  const int32_t *position;   // [n][k]
  const void *in;            // gather: X.  combine: Ys.  backward: dY
  int64_t ldi;
  const void *in2;           // backward: Ys
  int64_t ldi2;
  const float *w;            // [n][k] or null (ones)
  void *out;                 // gather: Xs.  combine: Y.  backward: dYs or null
  int64_t ldo;
  float *dw;                 // backward: [n][k] or null
  int first;                 // the launch's first token
};

constexpr int kRowWaves = 4;

// Token of this wave, its part of the row's 16-byte chunks [c, ...) step, and
// the token's sorted rows, one per lane (-1: dropped or past top_k).
template <int WPT>
__device__ __forceinline__ bool wave_token(const RowArgs &a, int64_t &i, int &part, int &pos) {
  const int w = threadIdx.x / kWave;
  i = a.first + (int64_t)blockIdx.x * (kRowWaves / WPT) + w / WPT;
  part = w % WPT;
  pos = i < a.n && lane_id() < a.k ? a.position[i * a.k + lane_id()] : -1;
  return i < a.n;
}

template <typename T, int WPT>
__global__ __launch_bounds__(kRowWaves *kWave) void gather_kernel(RowArgs a) {
  constexpr int V = Elem<T>::kVec;
  int64_t i;
  int part, pos;
  if (!wave_token<WPT>(a, i, part, pos)) return;
  const T *x = static_cast<const T *>(a.in) + i * a.ldi;
  for (int c = (part * kWave + lane_id()) * V; c < a.d; c += WPT * kWave * V) {
    const uint4 v = ldg16(x + c);
    for (int j = 0; j < a.k; ++j) {
      const int p = __builtin_amdgcn_readlane(pos, j);
      if (p >= 0) stg16(static_cast<T *>(a.out) + (int64_t)p * a.ldo + c, v);
    }
  }
}

template <typename T, int WPT>
__global__ __launch_bounds__(kRowWaves *kWave) void combine_kernel(RowArgs a) {
  constexpr int V = Elem<T>::kVec, JB = 8;
  int64_t i;
  int part, pos;
  if (!wave_token<WPT>(a, i, part, pos)) return;
  const float wl = !a.w ? 1.f : lane_id() < a.k ? a.w[i * a.k + lane_id()] : 0.f;
  T *y = static_cast<T *>(a.out) + i * a.ldo;
  for (int c = (part * kWave + lane_id()) * V; c < a.d; c += WPT * kWave * V) {
    float o[V] = {};
    for (int j0 = 0; j0 < a.k; j0 += JB) {
      uint4 raw[JB];                    // all of the block's loads before the first use
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        const int p = j0 + q < a.k ? __builtin_amdgcn_readlane(pos, j0 + q) : -1;
        if (p >= 0) raw[q] = ldg16(static_cast<const T *>(a.in) + (int64_t)p * a.ldi + c);
      }
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        const int p = j0 + q < a.k ? __builtin_amdgcn_readlane(pos, j0 + q) : -1;
        if (p < 0) continue;
        const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), j0 + q));
        float v[V];
        Elem<T>::unpack(raw[q], v);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(w, v[e], o[e]);
      }
    }
    stg16(y + c, Elem<T>::pack(o));
  }
}

template <typename T, int WPT>
__global__ __launch_bounds__(kRowWaves *kWave) void combine_backward_kernel(RowArgs a) {
  constexpr int V = Elem<T>::kVec, JB = 4;
  __shared__ float part_sum[kRowWaves][JB];
  int64_t i;
  int part, pos;
  const bool live = wave_token<WPT>(a, i, part, pos);
  if (WPT == 1 && !live) return;        // (WPT 4: the workgroup has one token, live for all)
  const float wl = !a.w ? 1.f : lane_id() < a.k ? a.w[i * a.k + lane_id()] : 0.f;
  const T *dy = static_cast<const T *>(a.in) + i * a.ldi;
  for (int j0 = 0; j0 < a.k; j0 += JB) {
    float dot[JB] = {};
    for (int c = (part * kWave + lane_id()) * V; c < a.d; c += WPT * kWave * V) {
      float g[V];
      const uint4 graw = ldg16(dy + c);
      uint4 raw[JB];                    // all of the block's loads before the first use
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        const int p = j0 + q < a.k ? __builtin_amdgcn_readlane(pos, j0 + q) : -1;
        if (p >= 0 && a.dw) raw[q] = ldg16(static_cast<const T *>(a.in2) + (int64_t)p * a.ldi2 + c);
      }
      Elem<T>::unpack(graw, g);
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        const int p = j0 + q < a.k ? __builtin_amdgcn_readlane(pos, j0 + q) : -1;
        if (p < 0) continue;
        if (a.dw) {
          float v[V];
          Elem<T>::unpack(raw[q], v);
#pragma unroll
          for (int e = 0; e < V; ++e) dot[q] = fmaf(g[e], v[e], dot[q]);
        }
        if (a.out) {
          const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wl), j0 + q));
          float o[V];
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = w * g[e];
          stg16(static_cast<T *>(a.out) + (int64_t)p * a.ldo + c, Elem<T>::pack(o));
        }
      }
    }
    if (!a.dw) continue;
#pragma unroll
    for (int q = 0; q < JB; ++q) dot[q] = wave_sum(dot[q]);
    if constexpr (WPT > 1) {
      if (lane_id() == 0)
#pragma unroll
        for (int q = 0; q < JB; ++q) part_sum[part][q] = dot[q];
      __syncthreads();
#pragma unroll
      for (int q = 0; q < JB; ++q) {
        dot[q] = 0.f;
#pragma unroll
        for (int w = 0; w < WPT; ++w) dot[q] += part_sum[w][q];
      }
      __syncthreads();
    }
    if (part == 0 && lane_id() == 0)
#pragma unroll
      for (int q = 0; q < JB; ++q)
        if (j0 + q < a.k) a.dw[i * a.k + j0 + q] = dot[q];
  }
}

// A token's row takes four waves, or one where that holds it in one step
// (16384 tokens x 4 of 8 KB: combine in 141 us with four waves, 157 with one).
template <typename T>
bool one_wave(int d) {
  return d <= kWave * Elem<T>::kVec;
}

// Tokens of a launch at most: a grid has less than 2^32 threads.
constexpr int kLaunchTokens = 1 << 22;

template <template <typename, int> class Launch>
void by_type(int dtype, RowArgs a, hipStream_t s) {
  const int n = a.n;
  for (a.first = 0; a.first < n; a.first += kLaunchTokens) {
    a.n = n - a.first < kLaunchTokens ? n : a.first + kLaunchTokens;
    if (dtype == LORA_BF16) {
      if (one_wave<bf16_t>(a.d)) Launch<bf16_t, 1>::go(a, s);
      else Launch<bf16_t, 4>::go(a, s);
    } else {
      if (one_wave<float>(a.d)) Launch<float, 1>::go(a, s);
      else Launch<float, 4>::go(a, s);
    }
  }
}
template <int WPT>
dim3 row_grid(const RowArgs &a) {
  return dim3((unsigned)(((int64_t)(a.n - a.first) * WPT + kRowWaves - 1) / kRowWaves));
}
template <typename T, int WPT> struct Gather {
  static void go(const RowArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((gather_kernel<T, WPT>), row_grid<WPT>(a), dim3(kRowWaves * kWave), 0, s, a);
  }
};
template <typename T, int WPT> struct Combine {
  static void go(const RowArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((combine_kernel<T, WPT>), row_grid<WPT>(a), dim3(kRowWaves * kWave), 0, s, a);
  }
};
template <typename T, int WPT> struct CombineBackward {
  static void go(const RowArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((combine_backward_kernel<T, WPT>), row_grid<WPT>(a),
                       dim3(kRowWaves * kWave), 0, s, a);
  }
};

}  // namespace

hipError_t launch_experts_sort(const int32_t *ids, int n_choices, int n_experts, int32_t *offsets,
                               int32_t *sorted, int32_t *position, int32_t *status,
                               int32_t *counts, hipStream_t stream) {
  const SortArgs a{ids, n_choices, n_experts, offsets, sorted, position, status, counts};
  const dim3 block(kSortThreads);
  if (n_choices <= kSortThreads) {
    hipLaunchKernelGGL(sort_one_kernel<1>, dim3(1), block, 0, stream, a);
  } else if (n_choices <= kExpertOneGroupChoices) {
    hipLaunchKernelGGL(sort_one_kernel<kOneGroupSteps>, dim3(1), block, 0, stream, a);
  } else {
    const int blocks = expert_blocks(n_choices);
    hipLaunchKernelGGL(sort_count_kernel, dim3(blocks), block, 0, stream, a);
    // one launch less while every workgroup can read all blocks' counts
    // (65536 choices, 64 experts: 17 us against 19 and a launch)
    if (blocks <= kScanBlocks) {
      hipLaunchKernelGGL(sort_place_kernel<true>, dim3(blocks), block, 0, stream, a);
    } else {
      hipLaunchKernelGGL(sort_scan_kernel, dim3(1), block, 0, stream, a, blocks);
      hipLaunchKernelGGL(sort_place_kernel<false>, dim3(blocks), block, 0, stream, a);
    }
  }
  return hipGetLastError();
}

hipError_t launch_experts_gather(const void *X, int64_t ldx, const int32_t *position, int n, int k,
                                 int d, int dtype, void *Xs, int64_t lds, hipStream_t stream) {
  by_type<Gather>(dtype, RowArgs{n, k, d, position, X, ldx, nullptr, 0, nullptr, Xs, lds, nullptr, 0},
                  stream);
  return hipGetLastError();
}

hipError_t launch_experts_combine(const void *Ys, int64_t lds, const float *w,
                                  const int32_t *position, int n, int k, int d, int dtype, void *Y,
                                  int64_t ldy, hipStream_t stream) {
  by_type<Combine>(dtype, RowArgs{n, k, d, position, Ys, lds, nullptr, 0, w, Y, ldy, nullptr, 0},
                   stream);
  return hipGetLastError();
}

hipError_t launch_experts_combine_backward(const void *dY, int64_t ldy, const void *Ys, int64_t lds,
                                           const float *w, const int32_t *position, int n, int k,
                                           int d, int dtype, void *dYs, int64_t ldds, float *dw,
                                           hipStream_t stream) {
  by_type<CombineBackward>(dtype, RowArgs{n, k, d, position, dY, ldy, Ys, lds, w, dYs, ldds, dw, 0},
                           stream);
  return hipGetLastError();
}

}  // namespace lora
