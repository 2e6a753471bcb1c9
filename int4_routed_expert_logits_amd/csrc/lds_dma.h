// Loads from global memory straight into LDS, shared by the tiled products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// LDS byte address of a pointer into a __shared__ array.
__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8*)p));
}

// One LDS DMA instruction: every active lane's 16 (or 4) bytes at g go to LDS
// at m0 + 16 (or 4) * lane.  Written as asm rather than the builtin: the
// compiler's own wait bookkeeping cannot tell the stages of a loop apart and
// would wait for every fetch in flight before each read of a stage; the loops
// wait for a stage's fetches themselves.  The s_nop is the wait state that the
// load needs behind a scalar write of m0, which the compiler sees to only where
// it emits both.  The statement has no register outputs; the address register
// is read when it issues.
__device__ __forceinline__ void dma16(const uint8_t* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t* g, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(g), "s"(lds)
               : "memory", "m0");
}

}  // namespace moe
