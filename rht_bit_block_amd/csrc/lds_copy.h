// Copies from HBM straight into LDS (buffer_load ... lds), issued from inline
// assembly and waited for with explicit vmcnt counts, so that the compiler's
// own wait insertion, which does not see them, never stalls on a prefetch.
// Lane i's 16 bytes land at M0 + 16 i; offsets at or past the buffer's size
// read as zeros.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ufp4 {

typedef int sgpr4 __attribute__((ext_vector_type(4)));

// Buffer resource over `bytes` bytes at a wave-uniform address.
__device__ __forceinline__ sgpr4 rsrc4(const void* base, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  sgpr4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF);   // stride 0
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}

__device__ __forceinline__ void lds_load16(uint32_t lds_addr, const sgpr4& r, uint32_t voff,
                                           uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(voff), "s"(r),
                 "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory");
}

// The same, 4 bytes per lane.
__device__ __forceinline__ void lds_load4(uint32_t lds_addr, const sgpr4& r, uint32_t voff,
                                          uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(voff), "s"(r),
                 "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

}  // namespace ufp4
