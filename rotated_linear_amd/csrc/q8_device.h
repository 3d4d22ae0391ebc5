// Device helpers of the 8-bit path: 16-bit element conversions, the row quantiser's last step and
// the gated activation.
#pragma once

#include "q8_internal.h"

namespace paro {

// Element types of rows (DT: PARO_F16, PARO_BF16, PARO_F32): float32 values to and from storage.
template <int DT>
__device__ inline float from_bits16(uint32_t h) {  // the element in the low 16 bits of h
  if constexpr (DT == PARO_F16) {
    return static_cast<float>(__builtin_bit_cast(_Float16, uint16_t(h)));
  } else {
    return __builtin_bit_cast(float, h << 16);
  }
}
template <int DT>
__device__ inline uint32_t to_bits16(float v) {  // rounded to nearest, ties to even
  if constexpr (DT == PARO_F16) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
  } else {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
}
template <int DT>
__device__ inline void unpack8(const u32x4& w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = from_bits16<DT>(w[i] & 0xFFFFu);
    f[2 * i + 1] = DT == PARO_F16 ? from_bits16<DT>(w[i] >> 16) : __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
  }
}
template <int DT>
__device__ inline u32x4 pack8(const float (&f)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = to_bits16<DT>(f[2 * i]) | (to_bits16<DT>(f[2 * i + 1]) << 16);
  return w;
}

// |v| as an ordered integer: larger for larger magnitudes, an infinity above every number and a
// NaN above that, so a maximum over a row keeps both.
__device__ inline uint32_t abs_order(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }
constexpr uint32_t kAbsInf = 0x7F800000u;

// The row quantiser's scale and code step from the row's largest magnitude (as abs_order): codes
// are rint(v * 127 / c), step + low = 127 / c to twice float32's precision. A row with an infinity or
// a NaN: scale NaN and `bad` (codes 0).
struct RowQuant {
  float scale, step, low;
  bool bad;
};
// code_top: the largest magnitude of the values that the codes are made from, where these are not the
// row itself but the row over a factor.
__device__ inline RowQuant row_quant(uint32_t top, uint32_t code_top) {
  RowQuant r;
  r.bad = top >= kAbsInf;
  r.scale = r.bad ? __builtin_nanf("") : fmaxf(__builtin_bit_cast(float, top), kQ8MinTop) / kQ8Max;
  const float c = fmaxf(__builtin_bit_cast(float, code_top), kQ8MinTop);
  r.step = kQ8Max / c;
  r.low = __builtin_fmaf(-r.step, c, kQ8Max) / c;  // the division's remainder is exact
  return r;
}
__device__ inline RowQuant row_quant(uint32_t top) { return row_quant(top, top); }
// The nearest whole number (ties to even) of |p| <= 127 in the low byte: adding 1.5 * 2^23 leaves it in
// the sum's low mantissa bits.
__device__ inline uint32_t whole_bits(float p) { return __builtin_bit_cast(uint32_t, p + 12582912.0f); }
// The code of v, its product rounded once from nearly exact. A 16-bit row whose maximum is 127 times a
// small number holds many values exactly half way between two codes: this way they stay half way and
// go to the even code, where the product with a rounded step would go either way.
__device__ inline uint32_t code_bits(float v, const RowQuant& q) {
  return whole_bits(__builtin_fmaf(v, q.step, v * q.low));
}
// Four codes as one word.
__device__ inline uint32_t codes4(float a, float b, float c, float d, const RowQuant& q) {
  const uint32_t ab = __builtin_amdgcn_perm(code_bits(b, q), code_bits(a, q), 0x0c0c0400u);
  const uint32_t cd = __builtin_amdgcn_perm(code_bits(d, q), code_bits(c, q), 0x04000c0cu);
  return ab | cd;
}

// One output of an 8-bit product before its last rounding: sum * xs * ws, two float32 roundings.
// Opaque to the compiler, which otherwise folds the last product into the conversion to float16
// in some kernels and not in others: every kernel gives the same bits.
__device__ inline float scaled(int sum, float xs, float ws) {
  float v = float(sum) * xs * ws;
  asm("" : "+v"(v));
  return v;
}

// silu(g) u = g u / (1 + exp(-g)) for an output of type DT. 16-bit outputs: exp(-g) past float32 gives an
// infinity and the quotient -0, the reciprocal instruction may give 0 for one under 2^-126 already, and the
// rounded argument of exp2 costs up to 1.2 |g| units of 2^-24, which a result of 11 or 8 bits does not
// see. float32 outputs: exp(-|g|), which does not overflow, from the math library, and a quotient, each to
// float32's last digit.
template <int DT>
__device__ inline float silu_mul(float g, float u) {
  float v;
  if constexpr (DT == PARO_F32) {
    const float e = expf(-fabsf(g)), den = 1.0f + e, num = g < 0 ? g * e : g;
    // num / den from the reciprocal and its remainder; an infinite g, and any past 17, has den = 1
    const float r = __builtin_amdgcn_rcpf(den), q = num * r;
    v = (den == 1.0f ? num : __builtin_fmaf(__builtin_fmaf(-q, den, num), r, q)) * u;
  } else {
    v = g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896f)) * u;
  }
  asm("" : "+v"(v));
  return v;
}

}  // namespace paro
