// LDS staging helpers for the MFMA kernels (gfx950).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora_device.cuh"

namespace lora {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Direct global -> LDS loads (gfx950 global_load_lds_dwordx4).  Each
// instruction moves 64 lanes x 16 bytes into 1 KB of LDS starting at M0, here
// the scalar `base` plus the constant `at` (known once the loop around is
// unrolled).  Issued through inline asm so that the compiler does not add
// conservative waits on them; completion is tracked by hand with s_waitcnt
// vmcnt(0) only (a wave waits for all of its loads, never for a count of them, so
// no wait depends on the order in which loads complete).  Between the write of M0
// and the load that reads it the ISA asks for one wait state, which the compiler
// does not add inside asm; the addition in the write of M0 pays for it.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

#define LORA_SET_M0 "s_add_u32 m0, %0, %1\n\ts_nop 0\n\t"
__device__ __forceinline__ void dma16(uint32_t base, int at, const void *src) {
  asm volatile(LORA_SET_M0 "global_load_lds_dwordx4 %2, off" ::"s"(base), "i"(at), "v"(src)
               : "memory", "m0", "scc");
}

// The same with the source given as a 64-bit scalar base plus a 32-bit
// per-lane byte offset (the instruction's saddr form).
__device__ __forceinline__ void dma16_s(uint32_t base, int at, uint32_t off, const void *src) {
  asm volatile(LORA_SET_M0 "global_load_lds_dwordx4 %2, %3" ::"s"(base), "i"(at), "v"(off), "s"(src)
               : "memory", "m0", "scc");
}

// One dword per lane: 64 lanes x 4 bytes into 256 bytes of LDS.
__device__ __forceinline__ void dma4(uint32_t base, int at, const void *src) {
  asm volatile(LORA_SET_M0 "global_load_lds_dword %2, off" ::"s"(base), "i"(at), "v"(src)
               : "memory", "m0", "scc");
}
__device__ __forceinline__ void dma4_s(uint32_t base, int at, uint32_t off, const void *src) {
  asm volatile(LORA_SET_M0 "global_load_lds_dword %2, %3" ::"s"(base), "i"(at), "v"(off), "s"(src)
               : "memory", "m0", "scc");
}
#undef LORA_SET_M0

// The same unless `skip` (a wave's scalar) is other than 0.  The branch is inside the
// asm: one that the compiler saw would split the block of products around it.  The
// comparison and the branch are the wait state.
#define LORA_SET_M0_UNLESS \
  "s_add_u32 m0, %0, %1\n\ts_cmp_lg_u32 %2, 0\n\ts_cbranch_scc1 .Ldma_skip_%=\n\t"
__device__ __forceinline__ void dma16_s_unless(uint32_t skip, uint32_t base, int at, uint32_t off, const void *src) {
  asm volatile(LORA_SET_M0_UNLESS "global_load_lds_dwordx4 %3, %4\n.Ldma_skip_%=:" ::"s"(base), "i"(at), "s"(skip),
               "v"(off), "s"(src)
               : "memory", "m0", "scc");
}
__device__ __forceinline__ void dma4_s_unless(uint32_t skip, uint32_t base, int at, uint32_t off, const void *src) {
  asm volatile(LORA_SET_M0_UNLESS "global_load_lds_dword %3, %4\n.Ldma_skip_%=:" ::"s"(base), "i"(at), "s"(skip),
               "v"(off), "s"(src)
               : "memory", "m0", "scc");
}
#undef LORA_SET_M0_UNLESS

// Wait until at most N of this wave's vector-memory operations are
// outstanding, then LDS-fence and barrier the workgroup.
template <int N>
__device__ __forceinline__ void vm_wait_barrier() {
  static_assert(N >= 0 && N <= 63, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void vm_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void lgkm_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ mfma_bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(mfma_bf16x8, v); }

// Row of element v (0..15) of a 32x32 MFMA accumulator held by lane l
// (its column is l % 32).
__device__ __forceinline__ int acc_row(int v, int l) { return (v >> 2) * 8 + (l >> 5) * 4 + (v & 3); }

}  // namespace lora
