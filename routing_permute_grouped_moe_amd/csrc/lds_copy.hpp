// Copies HBM -> LDS without staging registers, and the waits that go with
// them.
#pragma once

#include "common.hpp"

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char_t;

// Raw buffer descriptor as four SGPR words (range-checked, stride 0).
__device__ __forceinline__ i32x4 raw_rsrc(const void* base, uint32_t bytes) {
  const unsigned long long b = (unsigned long long)base;
  return i32x4{uniform((int)(uint32_t)b), uniform((int)((b >> 32) & 0xffffu)), uniform((int)bytes),
               MOE_RSRC_DW3};
}

__device__ __forceinline__ uint32_t lds_addr(const char* p) {
  return (uint32_t)(uintptr_t)(const lds_char_t*)p;
}

// One 1 KB HBM -> LDS copy: lane l's 16 bytes at voff + soff land at
// lds + 16 l.  Issued as inline assembly so that the compiler does not guard
// every later LDS read with a wait on all outstanding copies; the kernel
// waits for exactly the copies it needs (wait_vm) before a barrier.  The LDS
// address goes through M0, and an LDS-DMA load needs one wait state after
// the write of M0 (the compiler's hazard checks do not look inside inline
// assembly): M0 is written here, followed by s_nop 0.  Without the nop, a
// copy issued right after its M0 write could land at the previous copy's
// LDS address (seen as wrong, non-deterministic weight gradients whenever
// the scheduler put the two instructions back to back).
__device__ __forceinline__ void dma16(const i32x4& rs, uint32_t lds, uint32_t voff, int soff) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rs), "s"(uniform(soff)), "s"(uniform((int)lds))
               : "memory", "m0");
}

// Wait until at most n of this wave's buffer loads are outstanding.
template <int n>
__device__ __forceinline__ void wait_vm() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
