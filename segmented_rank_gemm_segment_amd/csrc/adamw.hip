// AdamW over many tensors at once (decoupled weight decay): for every element of
// every tensor that takes part,
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   w = (1 - lr wd) w - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps),
//
// with t the tensor's own step count.  Bound by memory: each of w, m and v is read
// and written once and g read once.  Measured: 201 M bf16 elements with fp32 masters and
// moments (28 bytes an element) 1052 us, 5.4 TB/s, what a copy of 1 GiB reaches (5.2);
// 176 M with 8-bit moments (10 bytes) 380 us, 4.6 TB/s, where the codes' arithmetic
// shows; 8.4 M of 16.8 M taking part 58 us, 4.3 TB/s; 18 k elements of 9 tensors 8 to
// 13 us, the launches' latency.  The factors of a tensor are formed by each of its
// workgroups: a launch of its own before this one took 3 to 5 us, which this hides.
//
// 8-bit moments: blocks of 256 consecutive elements share a float32 scale, their
// largest magnitude.  A first moment's code c (-127..127) stands for
// scale (c / 127) |c / 127|, a second moment's (0..255) for scale (c / 255)^4:
// relative steps of 2 / c and 4 / c down to 2^-14 and 2^-32 of the block's largest.
// With b2 = 0.999 a step moves v by less than a code's width, so rounding to the
// nearest code would hold it where it is; a value between two codes takes the upper
// one with the probability that makes the expectation the value itself.  A second
// moment above 0 takes code 1 at least: a quotient by a zero root would be huge.
#include <type_traits>

#include "lora_device.cuh"
#include "lora_kernels.h"
#include "tile_choice.h"

namespace lora {
namespace {

constexpr int kThreads = 256, kVec = 8;     // elements of a lane's load
constexpr int kStep = kThreads * kVec;      // elements of a workgroup's step
constexpr int kSteps = kAdamwChunk / kStep;
static_assert(kAdamwChunk % kStep == 0 && kAdamwBlock == 32 * kVec, "a block is half a wave");

// A 32-bit mixing: shifts and odd factors, in turn.
__host__ __device__ inline uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B1u;
  x ^= x >> 15;
  x *= 0x6A09E667u;
  return x ^ (x >> 16);
}

// The factors of a tensor's step, by two lanes.  The bias corrections are formed in 64
// bits, as 1 - b^t of the first steps is a small difference, and b^t by squaring.  A square
// doubles the relative error of its factor, so b^t is off by t 2^-53 of it at most and 1 - b^t,
// at least b^t t (1 - b), by 2^-53 / (1 - b) of it: what b's own last bit is to 1 - b.
struct Factors {
  float rate, root, keep;
  uint32_t key;
};
__device__ inline double power(double b, int t) {
  double p = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) p *= b;
  return p;
}
__device__ inline void write_factors(const AdamwArgs &a, int tensor, int lane, Factors &f) {
  const int t = a.step[tensor] + 1;
  const float left = (float)(1.0 - power(lane ? a.beta2 : a.beta1, t));
  if (lane) {
    f.root = 1.f / sqrtf(left);
    f.key = mix32(mix32(a.seed ^ ((uint32_t)t * 0x9E3779B1u)) + (uint32_t)tensor);
  } else {
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    f.rate = (float)lr / left;
    f.keep = (float)(1.0 - lr * a.weight_decay);
  }
}

// 8 elements as they are loaded.
template <typename T> struct Raw {
  static constexpr int N = kVec / Elem<T>::kVec;
  uint4 q[N];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = ldg16(p + i * Elem<T>::kVec);
  }
  // the first `count` of them (a tensor's last ones), zeros behind
  __device__ __forceinline__ void load_some(const T *p, int count) {
    float x[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = e < count ? Elem<T>::load1(p + e) : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = Elem<T>::pack(x + i * Elem<T>::kVec);
  }
  __device__ __forceinline__ void values(float (&x)[kVec]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) Elem<T>::unpack(q[i], x + i * Elem<T>::kVec);
  }
};
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; i += Elem<T>::kVec) stg16(p + i, Elem<T>::pack(x + i));
}
template <typename T>
__device__ __forceinline__ void store_some(T *p, int count, const float (&x)[kVec]) {
#pragma unroll
  for (int e = 0; e < kVec; ++e)
    if (e < count) Elem<T>::store1(p + e, x[e]);
}

__device__ __forceinline__ uint32_t byte_of(const uint2 &q, int e) {
  return ((e < 4 ? q.x : q.y) >> (8 * (e & 3))) & 0xffu;
}
// The first `count` codes (any number, a tensor's last ones), zeros behind.
__device__ __forceinline__ uint2 some_codes(uint2 q, int count) {
  const uint64_t keep = count <= 0 ? 0ull : count >= kVec ? ~0ull : ~(~0ull << (8 * count));
  return make_uint2(q.x & (uint32_t)keep, q.y & (uint32_t)(keep >> 32));
}
// c |c| and c^4 of the codes: the moments are these times the unit scales below.  Second
// moments are formed 2^8 times as large, kLift, beside 8-bit codes: the unit of a scale near
// 2^-100 is then a normal number, its reciprocal's 255^4 in range, and the root of what is
// at least a code's 2^-2 no zero.
constexpr float kLift = 256.f;
constexpr float kUnitM = 1.f / 16129.f, kUnitV = kLift / 4228250625.f;
__device__ __forceinline__ void powers_m(const uint2 &q, float (&x)[kVec]) {
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float c = (float)(int8_t)byte_of(q, e);
    x[e] = c * fabsf(c);
  }
}
__device__ __forceinline__ void powers_v(const uint2 &q, float (&x)[kVec]) {
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float c = (float)byte_of(q, e), c2 = c * c;
    x[e] = c2 * c2;
  }
}

// The largest of the 32 lanes that hold a block, as the bits of a float that is not
// negative (NaN above infinity above all numbers): within quads, then mirrored halves
// and rows of 16, then the two rows.
template <int CTRL> __device__ __forceinline__ uint32_t max_dpp(uint32_t b) {
  return max(b, (uint32_t)__builtin_amdgcn_update_dpp((int)b, (int)b, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t block_max(uint32_t b) {
  b = max_dpp<0xb1>(b);         // quad_perm 1, 0, 3, 2
  b = max_dpp<0x4e>(b);         // quad_perm 2, 3, 0, 1
  b = max_dpp<0x141>(b);        // row_half_mirror
  b = max_dpp<0x140>(b);        // row_mirror
  const auto rows = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return max((uint32_t)rows[0], (uint32_t)rows[1]);
}
// The scale of a block from its largest magnitude.  Below `tiny` the block is kept as
// zeros (its reciprocal would pass the range); 2^126 or more (whose reciprocal is no normal
// number), an infinity or NaN make it NaN.
constexpr uint32_t kTiny = (127u - 100u) << 23, kTinyV = kTiny + (8u << 23), kHuge = (127u + 126u) << 23;
__device__ __forceinline__ float block_scale(uint32_t top, uint32_t tiny) {
  return __uint_as_float(top < tiny ? 0u : top >= kHuge ? 0x7fc00000u : top);
}
// (one division, so that z below has two roundings: a share of the codes' distance that is
// off by them takes the other code that often)
__device__ __forceinline__ float over_scale(float top, float scale) {
  return scale > 0.f ? top / scale : 0.f;             // (NaN: 0, and codes of 0)
}

// 1 for what is above 0 (by 2^-126 or more), 0 for the rest: a product that is held to [0, 1]
__device__ __forceinline__ float one_above(float x) {
  return __builtin_amdgcn_fmed3f(x * 0x1p126f, 0.f, 1.f);
}

// The codes of first moments: z = 127^2 |x| / scale lies between c^2 and (c + 1)^2, and
// u (2 c + 1) < z - c^2 takes the upper one; u comes in 2^-16ths.  An error of the root
// changes c beside a whole number only, where the other c with the other share is the same.
// c is 126 at most and the upper one 127, which the block's largest takes whatever u is: its
// z - 126^2 is 253 within the 2^-9 of z's roundings, and 253 u at most 253 (1 - 2^-16).
__device__ __forceinline__ uint2 codes_m(const float (&x)[kVec], float scale,
                                         const float (&u)[kVec]) {
  const float inv = over_scale(16129.f, scale);
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float z = fabsf(x[e]) * inv;
    float c = fminf(floorf(__builtin_amdgcn_sqrtf(z)), 126.f);
    c += one_above(fmaf(-u[e], fmaf(c, 0x1p-15f, 0x1p-16f), fmaf(-c, c, z)));
    // a byte of c + 128, rounded (exact), less 128 by its upper bit
    q[e / 4] = __builtin_amdgcn_cvt_pk_u8_f32(copysignf(c, x[e]) + 128.f, e & 3, q[e / 4]);
  }
  return inv > 0.f ? make_uint2(q[0] ^ 0x80808080u, q[1] ^ 0x80808080u) : make_uint2(0u, 0u);
}
// Of second moments: z = 255^4 x / scale between c^4 and (c + 1)^4, which are
// (2 c + 1) (2 c^2 + 2 c + 1) apart.  root: of x, which the update needs too.
__device__ __forceinline__ uint2 codes_v(const float (&x)[kVec], const float (&root)[kVec],
                                         float scale, const float (&u)[kVec]) {
  const float inv = over_scale(4228250625.f, scale), rinv = __builtin_amdgcn_sqrtf(inv);
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float z = x[e] * inv;
    float c = floorf(__builtin_amdgcn_sqrtf(root[e] * rinv));
    const float c2 = c * c, t = c + c + 1.f;
    c += one_above(fmaf(-u[e] * fmaf(c, 0x1p-15f, 0x1p-16f), fmaf(c2, 2.f, t), fmaf(-c2, c2, z)));
    c = fmaxf(c, one_above(z));
    q[e / 4] = __builtin_amdgcn_cvt_pk_u8_f32(c, e & 3, q[e / 4]);        // (held to 255)
  }
  return inv > 0.f ? make_uint2(q[0], q[1]) : make_uint2(0u, 0u);
}

// The root by the instruction, within one unit in the last place, which takes what is below
// 2^-126 for zero.  The root of that is up to 2^-63: small numbers are taken 2^64 times as
// large.  Not beside 8-bit codes, whose eps is 2^-40 at least and v 2^8 times as large.
template <bool EIGHT> __device__ __forceinline__ float root_of(float v) {
  if constexpr (EIGHT) return __builtin_amdgcn_sqrtf(v);
  const bool small = v < 0x1p-64f;
  return __builtin_amdgcn_sqrtf(v * (small ? 0x1p64f : 1.f)) * (small ? 0x1p-32f : 1.f);
}

// A workgroup takes chunks of kAdamwChunk elements of one tensor.  P, G: the tensors'
// and gradients' types; MASTER: an fp32 copy of each tensor is what is updated, and
// the tensor its rounding; EIGHT: 8-bit moments.  Every workgroup forms the factors
// itself, while its loads are on their way.
template <typename P, typename G, bool MASTER, bool EIGHT>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const float b1 = (float)a.beta1, b2 = (float)a.beta2;
  const float c1 = (float)(1.0 - a.beta1), c2 = (float)(1.0 - a.beta2) * (EIGHT ? kLift : 1.f);
  __shared__ Factors shared[2];
  int turn = 0;
  for (int64_t chunk = blockIdx.x; chunk < a.n_chunks; chunk += gridDim.x) {
    const int ti = a.chunk_tensor[chunk];
    if (a.active && a.active[ti] == 0) continue;
    const AdamwTensor t = a.tensors[ti];
    const int64_t base = (chunk - t.first_chunk) * kAdamwChunk;
    // Every step's loads go out before the first step's arithmetic.  A block's lanes stay
    // together: the moments' buffers hold whole blocks, and lanes past the tensor's end, in its
    // last block, hold zeros (32-bit moments: anything, which meets no other element).
    using W = typename std::conditional<MASTER, float, P>::type;
    Raw<G> graw[kSteps];
    Raw<W> wraw[kSteps];
    Raw<float> mraw[EIGHT ? 1 : kSteps], vraw[EIGHT ? 1 : kSteps];
    uint2 mq[EIGHT ? kSteps : 1], vq[EIGHT ? kSteps : 1];
    float ms[EIGHT ? kSteps : 1], vs[EIGHT ? kSteps : 1];
    const int64_t in_tensor = t.numel - base;
    const int n = in_tensor < kAdamwChunk ? (int)in_tensor : kAdamwChunk;      // of the chunk
    const G *const gp = static_cast<const G *>(t.grad) + base;
    P *const pp = static_cast<P *>(t.param) + base;
    W *const wp = MASTER ? reinterpret_cast<W *>(t.master) + base : reinterpret_cast<W *>(pp);
    const int64_t st = t.start + base;
    float *const mf = static_cast<float *>(a.m) + st, *const vf = static_cast<float *>(a.v) + st;
    int8_t *const mc = static_cast<int8_t *>(a.m) + st;
    uint8_t *const vc = static_cast<uint8_t *>(a.v) + st;
    float *const msp = a.m_scale + st / kAdamwBlock, *const vsp = a.v_scale + st / kAdamwBlock;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int e0 = s * kStep + (int)threadIdx.x * kVec;
      if ((e0 & ~(kAdamwBlock - 1)) >= n) continue;
      if (e0 + kVec <= n) {
        graw[s].load(gp + e0);
        wraw[s].load(wp + e0);
      } else {
        graw[s].load_some(gp + e0, n - e0);
        wraw[s].load_some(wp + e0, n - e0);
      }
      if constexpr (EIGHT) {
        mq[s] = *reinterpret_cast<const uint2 *>(mc + e0);
        vq[s] = *reinterpret_cast<const uint2 *>(vc + e0);
        ms[s] = msp[e0 / kAdamwBlock];
        vs[s] = vsp[e0 / kAdamwBlock];
      } else {
        mraw[s].load(mf + e0);
        vraw[s].load(vf + e0);
      }
    }
    if (threadIdx.x < 2) write_factors(a, ti, threadIdx.x, shared[turn]);
    __syncthreads();
    Factors f = shared[turn];
    if (EIGHT) f.root *= 1.f / 16.f;                // (of kLift)
    turn ^= 1;         // (the next barrier lies between this chunk's reads and the write after)
    const uint32_t mkey = mix32(f.key + (uint32_t)(base >> 33)), pair = (uint32_t)(base >> 1);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int e0 = s * kStep + (int)threadIdx.x * kVec;
      if ((e0 & ~(kAdamwBlock - 1)) >= n) continue;
      float g[kVec], w[kVec], m[kVec], v[kVec], root[kVec];
      float mb = b1, vb = b2;                         // the old moments' factors
      graw[s].values(g);
      wraw[s].values(w);
      if constexpr (EIGHT) {
        if (e0 + kVec > n) {              // (what stands behind the tensor is no part of its block)
          mq[s] = some_codes(mq[s], n - e0);
          vq[s] = some_codes(vq[s], n - e0);
        }
        powers_m(mq[s], m);
        powers_v(vq[s], v);
        mb *= ms[s] * kUnitM;
        vb *= vs[s] * kUnitV;
      } else {
        mraw[s].values(m);
        vraw[s].values(v);
      }
      uint32_t mtop = 0u, vtop = 0u;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float ge = g[e] * gs;
        m[e] = fmaf(m[e], mb, ge * c1);
        v[e] = fmaf(v[e], vb, ge * ge * c2);
        root[e] = root_of<EIGHT>(v[e]);
        // (the instruction's reciprocal, within one unit in the last place, of what is no less
        // than eps and so a normal number)
        const float den = fmaf(root[e], f.root, a.eps);
        w[e] = fmaf(w[e], f.keep, -f.rate * (m[e] * __builtin_amdgcn_rcpf(den)));
        if constexpr (EIGHT) {
          mtop = max(mtop, __float_as_uint(fabsf(m[e])));
          vtop = max(vtop, __float_as_uint(fabsf(v[e])));
        }
      }
      if (e0 + kVec <= n) {
        if constexpr (MASTER) store8(wp + e0, w);
        store8(pp + e0, w);
      } else {
        if constexpr (MASTER) store_some(wp + e0, n - e0, w);
        store_some(pp + e0, n - e0, w);
      }
      if constexpr (EIGHT) {
        const float mscale = block_scale(block_max(mtop), kTiny);
        const float vscale = block_scale(block_max(vtop), kTinyV);
        float u[kVec];
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          const uint32_t h = mix32((pair + (uint32_t)(e0 + e) / 2) ^ mkey);
          u[e] = (float)(h & 0xffffu);
          u[e + 1] = (float)(h >> 16);
        }
        *reinterpret_cast<uint2 *>(mc + e0) = codes_m(m, mscale, u);
        *reinterpret_cast<uint2 *>(vc + e0) = codes_v(v, root, vscale, u);
        if ((threadIdx.x & 31) == 0) {
          msp[e0 / kAdamwBlock] = mscale;
          vsp[e0 / kAdamwBlock] = vscale * (1.f / kLift);
        }
      } else {
        store8(mf + e0, m);
        store8(vf + e0, v);
      }
    }
  }
}

// The steps are counted when all of the step's workgroups have read the counts: a launch
// of 2 us.  (Its last workgroup could do it, found by a counter for each tensor, but the
// workgroups' additions to the counters took 1.1 and 1.9 ms more in the first two
// figures above.)
__global__ __launch_bounds__(kThreads) void adamw_count_kernel(int32_t *step, const int32_t *active,
                                                               int n) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < n && (!active || active[i] != 0)) step[i] += 1;
}

// The values of 8-bit moments.
template <typename T>
__global__ __launch_bounds__(kThreads) void adamw_read_kernel(const int8_t *m, const uint8_t *v,
                                                              const float *m_scale,
                                                              const float *v_scale, int64_t total,
                                                              T *m_out, T *v_out) {
  for (int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kVec; e < total;
       e += (int64_t)gridDim.x * kStep) {
    float x[kVec], y[kVec];
    powers_m(*reinterpret_cast<const uint2 *>(m + e), x);
    powers_v(*reinterpret_cast<const uint2 *>(v + e), y);
    const float ms = m_scale[e / kAdamwBlock] * kUnitM, vs = v_scale[e / kAdamwBlock] * kUnitV;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      x[i] *= ms;
      y[i] = y[i] * (1.f / kLift) * vs;
    }
    store8(m_out + e, x);
    store8(v_out + e, y);
  }
}

// One workgroup a chunk (the bound keeps a grid's threads below 2^32): the next chunk's
// loads go out while this one's stores are on their way, which a loop over chunks in
// 8 or 16 workgroups a CU does less well (1119 us, 428 and 67 for 1050, 414 and 62 when it
// was tried).  Chunks of 4096: 2048 take 1066, 426 and 55 us for 1052, 401 and 58, 8192
// 1073, 414 and 61.
constexpr int64_t kStepGroups = 1 << 22;
constexpr int kReadGroups = kCUs * 8;

template <typename P, typename G, bool MASTER>
void launch_by_bits(const AdamwArgs &a, dim3 grid, hipStream_t s) {
  if (a.bits == 8)
    hipLaunchKernelGGL((adamw_kernel<P, G, MASTER, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((adamw_kernel<P, G, MASTER, false>), grid, dim3(kThreads), 0, s, a);
}
template <typename P, bool MASTER>
void launch_by_grad(const AdamwArgs &a, dim3 grid, hipStream_t s) {
  if (a.grad_dtype == LORA_BF16) launch_by_bits<P, bf16_t, MASTER>(a, grid, s);
  else launch_by_bits<P, float, MASTER>(a, grid, s);
}

}  // namespace

hipError_t launch_adamw(const AdamwArgs &a, hipStream_t stream) {
  if (a.n_chunks > 0) {
    const dim3 grid((unsigned)(a.n_chunks < kStepGroups ? a.n_chunks : kStepGroups));
    if (a.param_dtype == LORA_F32) launch_by_grad<float, false>(a, grid, stream);
    else if (a.master) launch_by_grad<bf16_t, true>(a, grid, stream);
    else launch_by_grad<bf16_t, false>(a, grid, stream);
  }
  hipLaunchKernelGGL(adamw_count_kernel, dim3((a.n_tensors + kThreads - 1) / kThreads),
                     dim3(kThreads), 0, stream, a.step, a.active, a.n_tensors);
  return hipGetLastError();
}

hipError_t launch_adamw_read(const void *m, const void *v, const float *m_scale,
                             const float *v_scale, int64_t total, int dtype, void *m_out,
                             void *v_out, hipStream_t stream) {
  const int64_t groups = (total + kStep - 1) / kStep;
  const dim3 grid((unsigned)(groups < kReadGroups ? groups : kReadGroups));
  const int8_t *mc = static_cast<const int8_t *>(m);
  const uint8_t *vc = static_cast<const uint8_t *>(v);
  if (dtype == LORA_BF16)
    hipLaunchKernelGGL(adamw_read_kernel<bf16_t>, grid, dim3(kThreads), 0, stream, mc, vc, m_scale,
                       v_scale, total, static_cast<bf16_t *>(m_out), static_cast<bf16_t *>(v_out));
  else
    hipLaunchKernelGGL(adamw_read_kernel<float>, grid, dim3(kThreads), 0, stream, mc, vc, m_scale,
                       v_scale, total, static_cast<float *>(m_out), static_cast<float *>(v_out));
  return hipGetLastError();
}

}  // namespace lora
