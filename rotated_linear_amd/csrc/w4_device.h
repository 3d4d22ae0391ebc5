// Device helpers of the INT4 linears on the matrix cores: 4-bit codes to float16 operands.
#pragma once

#include "paro_internal.h"

namespace paro {

// Float32 values in two float16 parts. The lower part is what the rounding of v to h takes away times 2^11, which makes it
// as large as v at most: it has its 11 bits as long as h has its own. The two leave 2^-22 of v, or 2^-36 where that is more
// (under 2^-14). (The lower part is 0 where v has no number, and where h has none, past 65504.)
constexpr float kRestUp = 0x1p11f, kRestDown = 0x1p-11f;
__device__ inline uint16_t rest16(float v, _Float16 h) {
  const float d = (v - static_cast<float>(h)) * kRestUp;
  return __builtin_bit_cast(uint16_t, static_cast<_Float16>(fabsf(d) < 65504.0f ? d : 0.0f));
}
// 2^e, -126 <= e <= 127.
__device__ inline float power2(int e) { return __builtin_bit_cast(float, (e + 127) << 23); }

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));

__device__ inline uint32_t and_or(uint32_t a, uint32_t m, uint32_t c) {
  uint32_t r;
  asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(m), "v"(c));
  return r;
}

// 8 nibbles of one 32-bit word -> exact (q - z) as float16 in the order [0,4,1,5,2,6,3,7].
// zlo = -(1024 + z) and zhi = -(64 + z), both as float16 pairs.
__device__ inline h8 dequant_word(uint32_t u, h2 zlo, h2 zhi, uint32_t m0, uint32_t m1, uint32_t e) {
  const h2 sixteenth = {static_cast<_Float16>(0.0625f), static_cast<_Float16>(0.0625f)};
  const uint32_t v = u >> 8;
  const h2 a0 = __builtin_bit_cast(h2, and_or(u, m0, e)) + zlo;                                        // 0, 4
  const h2 a1 = __builtin_elementwise_fma(__builtin_bit_cast(h2, and_or(u, m1, e)), sixteenth, zhi);  // 1, 5
  const h2 a2 = __builtin_bit_cast(h2, and_or(v, m0, e)) + zlo;                                        // 2, 6
  const h2 a3 = __builtin_elementwise_fma(__builtin_bit_cast(h2, and_or(v, m1, e)), sixteenth, zhi);  // 3, 7
  const uint4 o = {__builtin_bit_cast(uint32_t, a0), __builtin_bit_cast(uint32_t, a1),
                   __builtin_bit_cast(uint32_t, a2), __builtin_bit_cast(uint32_t, a3)};
  return __builtin_bit_cast(h8, o);
}

// A row's 8-channel word in the order dequant_word gives them.
__device__ inline h8 decode_order(h8 a) { return __builtin_shufflevector(a, a, 0, 4, 1, 5, 2, 6, 3, 7); }

}  // namespace paro
