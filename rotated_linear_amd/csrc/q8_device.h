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

// erfc(z) exp(z^2) / 2 for z >= 0 to 2^-19 of its value: t times a polynomial of degree 6 in t = 1 / (1 + z / 2),
// fitted for the smallest relative error over 0 <= z <= 10 (least squares, reweighted by the error).
__device__ inline float half_erfcx(float z) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(z, 0.5f, 1.0f));
  float p = 0.04410196840763092f;
  p = __builtin_fmaf(p, t, -0.17836840450763702f);
  p = __builtin_fmaf(p, t, 0.19461128115653992f);
  p = __builtin_fmaf(p, t, 0.018946044147014618f);
  p = __builtin_fmaf(p, t, 0.14075161516666412f);
  p = __builtin_fmaf(p, t, 0.13879111409187317f);
  p = __builtin_fmaf(p, t, 0.14116570353507996f);
  return p * t;
}

// act(v) for an output of type DT, as silu_mul is: float32 outputs from the math library's exp and erfc, 16-bit
// outputs to their own last digits (a result under 2^-126 may count as 0 there). Every sum of products is a
// fused one, written out, so that all kernels give the same bits.
template <int DT, int V>
__device__ inline void activate(float (&v)[V], int act) {
  if (act == PARO_ACT_RELU || act == PARO_ACT_RELU2) {  // (a NaN stays one)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float r = v[i] < 0 ? 0.0f : v[i];
      v[i] = act == PARO_ACT_RELU ? r : r * r;
    }
  } else if (act == PARO_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = silu_mul<DT>(v[i], 1.0f);
  } else if (act == PARO_ACT_GELU) {
    // half = erfc(|v| / sqrt(2)) / 2; v - v half where v is positive and v half where it is not keep their digits
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float a = fabsf(v[i]), z = a * 0.70710678118654752f;
      float half;
      if constexpr (DT == PARO_F32)
        half = 0.5f * erfcf(z);
      else
        half = half_erfcx(z) * __builtin_amdgcn_exp2f(a * a * -0.72134752044448170f);
      v[i] = v[i] < 0 ? v[i] * half : half == 0.0f ? v[i] : __builtin_fmaf(-v[i], half, v[i]);  // (an infinity stays one)
    }
  } else if (act == PARO_ACT_GELU_TANH) {  // v (1 + tanh(t / 2)) / 2 = v / (1 + exp(-t))
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float t = v[i] * __builtin_fmaf(0.071354816272600251f, v[i] * v[i], 1.5957691216057308f);
      if constexpr (DT == PARO_F32) {
        const float e = expf(-fabsf(t)), num = v[i] < 0 ? v[i] * e : v[i];
        v[i] = num / (1.0f + e);
      } else {
        v[i] = v[i] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.44269504088896f));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) asm("" : "+v"(v[i]));
}

// The steps of an output with an epilogue, behind scaled(): float32 each, the last one rounded to the output's
// type by the caller. Opaque, as scaled() is.
__device__ inline float plus(float v, float w) {
  v += w;
  asm("" : "+v"(v));
  return v;
}
// Element i of an array of type ydtype.
__device__ inline float load_element(const void* p, size_t i, int ydtype) {
  if (ydtype == PARO_F32) return static_cast<const float*>(p)[i];
  const uint32_t h = static_cast<const uint16_t*>(p)[i];
  return ydtype == PARO_F16 ? from_bits16<PARO_F16>(h) : from_bits16<PARO_BF16>(h);
}
// An output of a call with an epilogue, from its product, its bias (0 without one) and what there is of a residual.
__device__ inline float epilogue(const W8A8Call& c, float v, float bias, float residual) {
  float o[1] = {plus(v, bias)};
  if (c.ydtype == PARO_F32)
    activate<PARO_F32>(o, c.act);
  else
    activate<PARO_F16>(o, c.act);
  return c.residual ? plus(o[0], residual) : o[0];
}

}  // namespace paro
