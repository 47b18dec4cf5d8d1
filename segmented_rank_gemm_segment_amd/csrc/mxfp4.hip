// MXFP4 (the OCP microscaling format): rows to codes and scales, and back.
//
//   s = 2^(floor(log2 amax) - 2)      amax over a block of 32 consecutive values
//   code = E2M1(x / s)                nearest, ties to the even code, past 6 to 6
//
// s is kept as its biased exponent (E8M0), max(0, exponent bits of amax - 2): of
// amax's float32 bits the exponent field is floor(log2 amax) + 127 (a subnormal
// amax has 0, and the format's least scale 2^-127).  A block that holds an
// infinity or NaN gets the scale NaN (255).  amax is the integer maximum of the
// absolute values' bits, which orders NaN above infinity above the finite
// values, and division by a power of two is exact, so the codes do not depend
// on how the work is split.
//
// Both kernels are bound by HBM: a lane moves 8 values (16 bytes of bf16), four
// neighbouring lanes make a block and find its maximum by two lane swaps, and
// the conversions are the hardware's (v_cvt_scalef32_pk_fp4_f32 and its
// inverses: one instruction for two values, exact by the definition above,
// scale 2^-127 and NaN included).
#include "lora_device.cuh"
#include "lora_kernels.h"

namespace lora {
namespace {

struct MxArgs {
  const void *X;       // rows of values (quantize reads, dequantize writes)
  int64_t ldx;
  unsigned char *q;    // codes, ldq bytes a row
  int64_t ldq;
  unsigned char *s;    // scales, lds bytes a row
  int64_t lds;
  int n, d;
};

constexpr int kMxThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
  Elem<T>::unpack(ldg16(p), v);
  if constexpr (Elem<T>::kVec == 4) {
    float hi[4];
    Elem<T>::unpack(ldg16(p + 4), hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 + e] = hi[e];
  }
}

// Threads (tx, ty): 8-value column blockIdx.x TX + tx of rows blockIdx.y TY + ty
// + i gridDim.y TY.
template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_kernel(MxArgs a, int TX) {
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, TY = kMxThreads / TX;
  const int c = blockIdx.x * TX + tx;
  if (c >= a.d / 8) return;             // d % 32 == 0: whole blocks of four lanes leave
  for (int row = blockIdx.y * TY + ty; row < a.n; row += gridDim.y * TY) {
    float v[8];
    load8(static_cast<const T *>(a.X) + (int64_t)row * a.ldx + c * 8, v);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    const uint32_t ebits = m >> 23;
    const bool bad = ebits == 255;      // an infinity or NaN
    const uint32_t byte = bad ? 255u : ebits > 2 ? ebits - 2 : 0u;
    const float sc = __uint_as_float(byte << 23);
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], sc, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], sc, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], sc, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], sc, 3);
    *reinterpret_cast<uint32_t *>(a.q + (int64_t)row * a.ldq + c * 4) = bad ? 0u : q;
    if (c % 4 == 0) a.s[(int64_t)row * a.lds + c / 4] = (unsigned char)byte;
  }
}

template <typename T>
__global__ __launch_bounds__(kMxThreads) void mx_dequantize_kernel(MxArgs a, int TX) {
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, TY = kMxThreads / TX;
  const int c = blockIdx.x * TX + tx;
  if (c >= a.d / 8) return;
  for (int row = blockIdx.y * TY + ty; row < a.n; row += gridDim.y * TY) {
    const uint32_t q = *reinterpret_cast<const uint32_t *>(a.q + (int64_t)row * a.ldq + c * 4);
    const float sc = __uint_as_float((uint32_t)a.s[(int64_t)row * a.lds + c / 4] << 23);
    T *out = static_cast<T *>(const_cast<void *>(a.X)) + (int64_t)row * a.ldx + c * 8;
    if constexpr (Elem<T>::kVec == 8) {
      uint4 o;
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, sc, 3));
      stg16(out, o);
    } else {
      const hw_f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 0);
      const hw_f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 1);
      const hw_f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 2);
      const hw_f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, sc, 3);
      const float lo[4] = {p0[0], p0[1], p1[0], p1[1]}, hi[4] = {p2[0], p2[1], p3[0], p3[1]};
      stg16(out, Elem<float>::pack(lo));
      stg16(out + 4, Elem<float>::pack(hi));
    }
  }
}

// Columns per workgroup: the narrowest power of two that holds a row, so short
// rows share a workgroup.
int columns(int d) {
  int tx = 4;
  while (tx < kMxThreads && tx * 8 < d) tx *= 2;
  return tx;
}
dim3 grid_of(int n, int d, int tx) {
  const int ty = kMxThreads / tx;
  const int64_t gy = ((int64_t)n + ty - 1) / ty;
  return dim3((d / 8 + tx - 1) / tx, gy < 65535 ? (int)gy : 65535);
}

}  // namespace

hipError_t launch_mx_quantize(const void *X, int64_t ldx, int n, int d, int dtype, void *q,
                              int64_t ldq, void *s, int64_t lds, hipStream_t stream) {
  const MxArgs a{X, ldx, (unsigned char *)q, ldq, (unsigned char *)s, lds, n, d};
  const int tx = columns(d);
  if (dtype == LORA_BF16)
    hipLaunchKernelGGL(mx_quantize_kernel<bf16_t>, grid_of(n, d, tx), dim3(kMxThreads), 0, stream, a, tx);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<float>, grid_of(n, d, tx), dim3(kMxThreads), 0, stream, a, tx);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void *q, int64_t ldq, const void *s, int64_t lds, int n,
                                int d, int dtype, void *X, int64_t ldx, hipStream_t stream) {
  const MxArgs a{X, ldx, (unsigned char *)const_cast<void *>(q), ldq,
                 (unsigned char *)const_cast<void *>(s), lds, n, d};
  const int tx = columns(d);
  if (dtype == LORA_BF16)
    hipLaunchKernelGGL(mx_dequantize_kernel<bf16_t>, grid_of(n, d, tx), dim3(kMxThreads), 0, stream, a, tx);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<float>, grid_of(n, d, tx), dim3(kMxThreads), 0, stream, a, tx);
  return hipGetLastError();
}

}  // namespace lora
