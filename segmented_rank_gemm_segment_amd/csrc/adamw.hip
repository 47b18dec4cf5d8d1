// AdamW over many tensors at once (decoupled weight decay): for every element of
// every tensor that takes part,
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   w = (1 - lr wd) w - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps),
//
// with t the tensor's own step count.  Bound by memory: each of w, m and v is read
// and written once and g read once.
//
// 8-bit moments: blocks of 256 consecutive elements share a float32 scale, their
// largest magnitude.  A first moment's code c (-127..127) stands for
// scale (c / 127) |c / 127|, a second moment's (0..255) for scale (c / 255)^4:
// relative steps of 2 / c and 4 / c down to 2^-14 and 2^-32 of the block's largest.
// With b2 = 0.999 a step moves v by less than a code's width, so rounding to the
// nearest code would hold it where it is; a value between two codes takes the upper
// one with the probability that makes the expectation the value itself.  A second
// moment above 0 takes code 1 at least: a quotient by a zero root would be huge.
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

// Each tensor's step count and the factors of this step.  The bias corrections are
// formed in 64 bits: 1 - b2^t of the first steps is a small difference.
__global__ __launch_bounds__(256) void adamw_factors_kernel(AdamwArgs a) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.n_tensors) return;
  const bool on = !a.active || a.active[i] != 0;
  int t = a.step[i];
  if (on) a.step[i] = ++t;
  const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
  AdamwFactors f;
  f.on = on;
  f.rate = (float)(lr / (1.0 - pow(a.beta1, (double)t)));
  f.root = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)t)));
  f.keep = (float)(1.0 - lr * a.weight_decay);
  f.key = mix32(mix32(a.seed ^ ((uint32_t)t * 0x9E3779B1u)) + (uint32_t)i);
  a.factors[i] = f;
}

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&x)[kVec]);
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&x)[kVec]) {
  Elem<float>::unpack(ldg16(p), x);
  Elem<float>::unpack(ldg16(p + 4), x + 4);
}
template <> __device__ __forceinline__ void load8<bf16_t>(const bf16_t *p, float (&x)[kVec]) {
  Elem<bf16_t>::unpack(ldg16(p), x);
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&x)[kVec]);
template <> __device__ __forceinline__ void store8<float>(float *p, const float (&x)[kVec]) {
  stg16(p, Elem<float>::pack(x));
  stg16(p + 4, Elem<float>::pack(x + 4));
}
template <> __device__ __forceinline__ void store8<bf16_t>(bf16_t *p, const float (&x)[kVec]) {
  stg16(p, Elem<bf16_t>::pack(x));
}
// The first `count` of 8 elements (a tensor's last ones).
template <typename T>
__device__ __forceinline__ void load_some(const T *p, int count, float (&x)[kVec]) {
#pragma unroll
  for (int e = 0; e < kVec; ++e) x[e] = e < count ? Elem<T>::load1(p + e) : 0.f;
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
__device__ __forceinline__ void values_m(const uint2 &q, float scale, float (&x)[kVec]) {
  const float s = scale * (1.f / 16129.f);
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float c = (float)(int8_t)byte_of(q, e);
    x[e] = s * (c * fabsf(c));
  }
}
__device__ __forceinline__ void values_v(const uint2 &q, float scale, float (&x)[kVec]) {
  const float s = scale * (1.f / 4228250625.f);
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float c = (float)byte_of(q, e), c2 = c * c;
    x[e] = s * (c2 * c2);
  }
}

// The largest of the 32 lanes that hold a block, as the bits of a float that is not
// negative (NaN above infinity above all numbers).
__device__ __forceinline__ uint32_t block_max(uint32_t b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) b = max(b, (uint32_t)__shfl_xor((int)b, o));
  return b;
}
// The scale of a block from its largest magnitude.  Below 2^-100 the block is kept as
// zeros (its reciprocal would pass the range); an infinity or NaN makes it NaN.
constexpr uint32_t kTiny = (127u - 100u) << 23, kInf = 0x7f800000u;
__device__ __forceinline__ float block_scale(uint32_t top) {
  return __uint_as_float(top < kTiny ? 0u : top >= kInf ? 0x7fc00000u : top);
}
__device__ __forceinline__ float inverse(float scale) {
  return scale > 0.f ? 1.f / scale : 0.f;             // (NaN: 0, and codes of 0)
}

// The codes of first moments: z = 127^2 |x| / scale lies between c^2 and (c + 1)^2,
// and u (2 c + 1) < z - c^2 takes the upper one.
__device__ __forceinline__ uint2 codes_m(const float (&x)[kVec], float scale,
                                         const float (&u)[kVec]) {
  const float inv = inverse(scale) * 16129.f;
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float z = inv > 0.f ? fabsf(x[e]) * inv : 0.f;
    float c = floorf(__builtin_amdgcn_sqrtf(z));
    c += u[e] * (2.f * c + 1.f) < fmaf(-c, c, z) ? 1.f : 0.f;
    const int i = (int)fminf(c, 127.f);
    q[e / 4] |= (uint32_t)((x[e] < 0.f ? -i : i) & 0xff) << (8 * (e & 3));
  }
  return make_uint2(q[0], q[1]);
}
// Of second moments: z = 255^4 x / scale between c^4 and (c + 1)^4, which are
// (2 c + 1) (2 c^2 + 2 c + 1) apart.
__device__ __forceinline__ uint2 codes_v(const float (&x)[kVec], float scale,
                                         const float (&u)[kVec]) {
  const float inv = inverse(scale) * 4228250625.f;
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    const float z = inv > 0.f ? x[e] * inv : 0.f;
    float c = floorf(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(z)));
    const float c2 = c * c, gap = (2.f * c + 1.f) * (2.f * c2 + 2.f * c + 1.f);
    c += u[e] * gap < fmaf(-c2, c2, z) ? 1.f : 0.f;
    const int i = (int)fminf(fmaxf(c, z > 0.f ? 1.f : 0.f), 255.f);
    q[e / 4] |= (uint32_t)i << (8 * (e & 3));
  }
  return make_uint2(q[0], q[1]);
}

// A workgroup takes chunks of kAdamwChunk elements of one tensor.  P, G: the tensors'
// and gradients' types; MASTER: an fp32 copy of each tensor is what is updated, and
// the tensor its rounding; EIGHT: 8-bit moments.
template <typename P, typename G, bool MASTER, bool EIGHT>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwArgs a) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.f;
  const float b1 = (float)a.beta1, b2 = (float)a.beta2;
  const float c1 = (float)(1.0 - a.beta1), c2 = (float)(1.0 - a.beta2);
  for (int64_t chunk = blockIdx.x; chunk < a.n_chunks; chunk += gridDim.x) {
    const int ti = a.chunk_tensor[chunk];
    const AdamwFactors f = a.factors[ti];
    if (!f.on) continue;
    const AdamwTensor t = a.tensors[ti];
    const int64_t base = (chunk - t.first_chunk) * kAdamwChunk;
    const uint32_t mkey = mix32(f.key + (uint32_t)(base >> 33));
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t e0 = base + s * kStep + threadIdx.x * kVec;
      // (a block's lanes stay together: lanes past the tensor's end hold zeros)
      if (base + s * kStep + (int64_t)(threadIdx.x & ~31) * kVec >= t.numel) continue;
      const int left = (int)min((int64_t)kVec, t.numel - e0);      // may be 0 or less
      const bool whole = left == kVec;
      P *const pp = static_cast<P *>(t.param) + e0;
      const G *const gp = static_cast<const G *>(t.grad) + e0;
      float *const wp = MASTER ? t.master + e0 : nullptr;
      const int64_t st = t.start + e0;
      float g[kVec], w[kVec], m[kVec], v[kVec];
      if (whole) {
        load8(gp, g);
        if constexpr (MASTER) load8(wp, w); else load8(pp, w);
      } else {
        load_some(gp, left, g);
        if constexpr (MASTER) load_some(wp, left, w); else load_some(pp, left, w);
      }
      // (the moments' buffers hold whole blocks)
      if constexpr (EIGHT) {
        const int64_t blk = st / kAdamwBlock;
        values_m(*reinterpret_cast<const uint2 *>(static_cast<int8_t *>(a.m) + st), a.m_scale[blk], m);
        values_v(*reinterpret_cast<const uint2 *>(static_cast<uint8_t *>(a.v) + st), a.v_scale[blk], v);
      } else {
        load8(static_cast<const float *>(a.m) + st, m);
        load8(static_cast<const float *>(a.v) + st, v);
      }
      uint32_t mtop = 0u, vtop = 0u;
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float ge = g[e] * gs;
        m[e] = fmaf(m[e], b1, ge * c1);
        v[e] = fmaf(v[e], b2, ge * ge * c2);
        w[e] = w[e] * f.keep - f.rate * (m[e] / (sqrtf(v[e]) * f.root + a.eps));
        if constexpr (EIGHT) {
          mtop = max(mtop, __float_as_uint(fabsf(m[e])));
          vtop = max(vtop, __float_as_uint(fabsf(v[e])));
        }
      }
      if (whole) {
        if constexpr (MASTER) store8(wp, w);
        store8(pp, w);
      } else {
        if constexpr (MASTER) store_some(wp, left, w);
        store_some(pp, left, w);
      }
      if constexpr (EIGHT) {
        const float ms = block_scale(block_max(mtop)), vs = block_scale(block_max(vtop));
        float u[kVec];
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          const uint32_t h = mix32((uint32_t)((uint64_t)(e0 + e) >> 1) ^ mkey);
          u[e] = (float)(h & 0xffffu) * 0x1p-16f;
          u[e + 1] = (float)(h >> 16) * 0x1p-16f;
        }
        *reinterpret_cast<uint2 *>(static_cast<int8_t *>(a.m) + st) = codes_m(m, ms, u);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(a.v) + st) = codes_v(v, vs, u);
        if ((threadIdx.x & 31) == 0) {
          a.m_scale[st / kAdamwBlock] = ms;
          a.v_scale[st / kAdamwBlock] = vs;
        }
      } else {
        store8(static_cast<float *>(a.m) + st, m);
        store8(static_cast<float *>(a.v) + st, v);
      }
    }
  }
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
    values_m(*reinterpret_cast<const uint2 *>(m + e), m_scale[e / kAdamwBlock], x);
    values_v(*reinterpret_cast<const uint2 *>(v + e), v_scale[e / kAdamwBlock], y);
    store8(m_out + e, x);
    store8(v_out + e, y);
  }
}

constexpr int kGroups = kCUs * 8;      // workgroups of a launch at most

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
  hipLaunchKernelGGL(adamw_factors_kernel, dim3((a.n_tensors + 255) / 256), dim3(256), 0, stream, a);
  if (a.n_chunks > 0) {
    const dim3 grid((unsigned)(a.n_chunks < kGroups ? a.n_chunks : kGroups));
    if (a.param_dtype == LORA_F32) launch_by_grad<float, false>(a, grid, stream);
    else if (a.master) launch_by_grad<bf16_t, true>(a, grid, stream);
    else launch_by_grad<bf16_t, false>(a, grid, stream);
  }
  return hipGetLastError();
}

hipError_t launch_adamw_read(const void *m, const void *v, const float *m_scale,
                             const float *v_scale, int64_t total, int dtype, void *m_out,
                             void *v_out, hipStream_t stream) {
  const int64_t groups = (total + kStep - 1) / kStep;
  const dim3 grid((unsigned)(groups < kGroups ? groups : kGroups));
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
