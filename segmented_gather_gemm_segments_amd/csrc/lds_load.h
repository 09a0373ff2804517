// Loads from memory straight into LDS, and the waits that go with them.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace {

// At most N vector-memory operations of this wave outstanding, the other counters not waited
// for (vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Every LDS operation of this wave done.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

// 16 bytes a lane from anywhere in memory to LDS, lane l's to byte `to` + 16 l (`to` the same in all lanes).
// Written out because the compiler, which cannot tell that a transposed LDS read and such a load in
// flight touch different stages, would wait for every load before the first of those reads.  It has no
// register result, and puts m0 back; who reads the stage calls wait_vm first.
__device__ __forceinline__ void load_lds16(const void *from, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(to), "v"(from)
               : "memory");
}
// The same from byte `off` behind an address that all lanes share.
__device__ __forceinline__ void load_lds16(const void *base, uint32_t off, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(to), "v"(off), "s"(base)
               : "memory");
}
// One byte a lane, lane l's to the 32 bits at byte `to` + 4 l.
__device__ __forceinline__ void load_lds1(const void *from, uint32_t to) {
  uint32_t m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_ubyte %2, off\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(to), "v"(from)
               : "memory");
}
__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)p;
}

}  // namespace
