// Loads from memory straight to LDS, and the waits that order them, for the tiled
// products.
#pragma once

#include "moe_device.hpp"

namespace moe {

// Buffer descriptor of `bytes` bytes at p (both wave-uniform): loads past the
// end return zeros.
__device__ __forceinline__ u32x4 buf_of(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) & 0xFFFFu,
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00027000u};
}
// Memory to LDS, 16 (4) bytes a lane: lane l's bytes at voff + soff land at
// lds + 16 l (4 l).  No register is written.  In asm because the compiler
// would wait for every such load before the next LDS read of any buffer; the
// kernel's own waits below order them.  m0 is reserved in the compiler (it may
// not be named as overwritten), which keeps nothing in it between instructions;
// that nothing else touches it is tested on the built code.  A memory instruction
// may read it one state after it was written.  ONCE: the bytes are not read again
// (non-temporal).
// A wave-uniform offset for these, in a scalar register that a memory
// instruction may read: one that a vector instruction wrote needs 5 states.
__device__ __forceinline__ uint32_t dma_offset(uint32_t v) {
  uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
  asm volatile("s_nop 4" : "+s"(s));
  return s;
}
template <bool ONCE = false>
__device__ __forceinline__ void dma_b128(u32x4 buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  if (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(lds),
                 "v"(voff), "s"(buf), "s"(soff)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds),
                 "v"(voff), "s"(buf), "s"(soff)
                 : "memory");
}
__device__ __forceinline__ void dma_b32(u32x4 buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds),
               "v"(voff), "s"(buf), "s"(soff)
               : "memory");
}
// All but the wave's last N memory operations are done, and all its LDS reads;
// then the block's waves meet.
template <int N>
__device__ __forceinline__ void wait_step() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The block's waves meet, each with its LDS reads done.
__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

}  // namespace moe
