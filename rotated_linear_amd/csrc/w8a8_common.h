// Device code that the 8-bit product kernels share: storing scaled results.
#pragma once

#include "q8_device.h"

namespace paro {

// y[m][n .. n + 3] = v in the output's type; columns past N are left out.
__device__ inline void store4(const W8A8Call& c, int m, int n, const float (&v)[4]) {
  const size_t at = size_t(m) * c.N + n;
  const bool whole = (c.N & 3) == 0;  // then rows start at multiples of four elements and n + 3 < N
  if (whole ? n >= c.N : false) return;
  if (c.ydtype == PARO_F32) {
    float* y = static_cast<float*>(c.y) + at;
    if (whole) {
      *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < c.N) y[e] = v[e];
    }
  } else {
    uint16_t* y = static_cast<uint16_t*>(c.y) + at;
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = c.ydtype == PARO_F16 ? to_bits16<PARO_F16>(v[e]) : to_bits16<PARO_BF16>(v[e]);
    if (whole) {
      *reinterpret_cast<uint2*>(y) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < c.N) y[e] = uint16_t(b[e]);
    }
  }
}

}  // namespace paro
