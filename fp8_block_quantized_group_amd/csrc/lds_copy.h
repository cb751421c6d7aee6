// Copies from HBM into LDS that bypass the registers, and the waits for them.
//
// The loads are issued from inline asm, so the compiler does not know that LDS
// is written behind its back and neither drains the outstanding loads before
// every LDS read nor reorders around them: the waits here (asm with a memory
// clobber) are the only synchronisation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));
constexpr uint32_t kRsrcWord3 = 0x00020000u;   // raw buffer, 32-bit data format

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"

// Wait until at most N of this wave's LDS-bound loads are in flight and its
// own LDS reads have completed, then barrier.
template <int N>
__device__ __forceinline__ void wait_then_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
#endif
}

// Raw buffer resource over [base, base + num_records): offsets at or past
// num_records read zeros.  Kept in SGPRs.
__device__ __forceinline__ v4i buffer_rsrc(const void* base, uint32_t num_records) {
  const uint64_t b = (uint64_t)base;
  return v4i{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
             __builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xFFFFu)),
             __builtin_amdgcn_readfirstlane((int)num_records), (int)kRsrcWord3};
}

// HBM -> LDS: lane l's 16 (4) bytes at rsrc + voffset land at lds + 16*l (4*l).
__device__ __forceinline__ void dma16(v4i rsrc, uint32_t lds, uint32_t voffset) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               ::"s"(lds), "v"(voffset), "s"(rsrc) : "memory", "m0");
#endif
}
// The same with the non-temporal hint, for data that no other block reads.
__device__ __forceinline__ void dma16_nt(v4i rsrc, uint32_t lds, uint32_t voffset) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
               ::"s"(lds), "v"(voffset), "s"(rsrc) : "memory", "m0");
#endif
}
// ... lane l's 4 bytes at lds + 4*l
__device__ __forceinline__ void dma4(v4i rsrc, uint32_t lds, uint32_t voffset) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               ::"s"(lds), "v"(voffset), "s"(rsrc) : "memory", "m0");
#endif
}
// At most N of this wave's loads are in flight; its own LDS reads have completed.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(N) : "memory");
#endif
}
// This wave's LDS accesses have completed, for a load into what they read.
__device__ __forceinline__ void wait_lds() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#endif
}
// A barrier for LDS alone: loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#endif
}
#pragma clang diagnostic pop

// f(integral_constant<int, v>) for a wave-uniform v in [0, N].
template <int N, class F>
__device__ __forceinline__ void with_constant(int v, F&& f) {
  if constexpr (N > 0) {
    if (v == N) {
      f(std::integral_constant<int, N>{});
      return;
    }
    with_constant<N - 1>(v, f);
  } else {
    f(std::integral_constant<int, 0>{});
  }
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

}  // namespace moe
