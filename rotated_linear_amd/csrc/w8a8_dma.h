// Loads straight into LDS (CDNA4 global_load_lds), shared by the 8-bit product kernels.
#pragma once

#include "q8_device.h"

namespace paro {

// 16 (4) bytes per lane straight into LDS: lane l's land at lds + 16 l (4 l). The compiler does not
// see these loads, so a kernel waits for them itself; they have no output register.
__device__ inline void dma16(uint32_t lds, uint32_t voff, const void* base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(voff), "s"(base)
      : "memory", "m0");
}
__device__ inline void dma4(uint32_t lds, uint32_t voff, const void* base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2"
      :
      : "s"(lds), "v"(voff), "s"(base)
      : "memory", "m0");
}

// Byte offset of chunk c (16 bytes) of a tile row in a stage: rows of 128 bytes, the chunk index
// mixed with the row so that 16 consecutive rows' chunk c lie in 16 distinct slots modulo 256 bytes.
__device__ inline uint32_t swz(uint32_t row, uint32_t c) { return row * 128 + ((c ^ ((row >> 1) & 7)) << 4); }

// The LDS address of a pointer into dynamic shared memory.
__device__ inline uint32_t lds_address(const char* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p));
}

}  // namespace paro
