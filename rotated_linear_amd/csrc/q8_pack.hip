// Build-time weights in 8 bits: each row of W, with the transform folded in or as it is, quantised
// in float64 by its largest magnitude.
//
// One workgroup per weight row, the row in LDS as float64. Bound by LDS: every stage gathers and
// rewrites the row. Measured, K = 8: 4096 x 4096 86 us, 1024 x 14336 92 us; 256 x 1536 (a pair per
// thread and stage) 9.9 us, 11.6 with four. Loading the next stage's records ahead did not pay: it takes
// registers, and with them the waves that hide LDS's latency. Compiled with -ffp-contract=off: each product
// and each sum of the fold is rounded on its own, so the codes are those of the stated definition (the
// quantiser asks for its one fused product by name).
#include <algorithm>

#include "q8_device.h"

namespace paro {
namespace {

template <int DT>
__global__ __launch_bounds__(1024) void pack_q8_kernel(int N, int D, int K, const uint16_t* W, const PairRec* recs,
                                                       const float* s, int8_t* q, float* scales) {
  extern __shared__ double brow[];  // [D]
  __shared__ unsigned long long stop;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int P = D / 2;
  for (size_t n = blockIdx.x; n < size_t(N); n += gridDim.x) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(W + n * D);
    if (tid == 0) stop = 0;
    for (int p = tid; p < P; p += nt) {
      const uint32_t v = w[p];
      brow[2 * p] = from_bits16<DT>(v & 0xFFFFu);
      brow[2 * p + 1] = from_bits16<DT>(v >> 16);
    }
    __syncthreads();
    for (int k = 0; k < K; ++k) {
      for (int p = tid; p < P; p += nt) {
        const PairRec r = recs[size_t(k) * P + p];
        const int i = int((r.ij & 0xFFFFu) >> 2), j = int(r.ij >> 18);  // the fields are 4 i and 4 j
        const double c = r.c, sn = r.s;
        const double bi = brow[i], bj = brow[j];
        brow[i] = c * bi + sn * bj;
        brow[j] = c * bj - sn * bi;
      }
      __syncthreads();
    }
    unsigned long long top = 0;  // |v| as an ordered integer (an infinity, then a NaN, on top)
    for (int p = tid; p < P; p += nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        double b = brow[2 * p + e];
        if (s) {
          b = b * static_cast<double>(s[2 * p + e]);
          brow[2 * p + e] = b;
        }
        top = max(top, __builtin_bit_cast(unsigned long long, b) & 0x7FFFFFFFFFFFFFFFull);
      }
    }
    for (int off = 32; off >= 1; off >>= 1) top = max(top, __shfl_xor(top, off));
    if ((tid & 63) == 0) atomicMax(&stop, top);
    __syncthreads();
    top = stop;
    const bool bad = top >= 0x7FF0000000000000ull;
    const double c0 = fmax(__builtin_bit_cast(double, top), double(kQ8MinTop));
    // 127 / c0 to twice float64's precision, so that a weight half way between two codes stays there
    const double step = 127.0 / c0, low = __builtin_fma(-step, c0, 127.0) / c0;
    for (int p = tid; p < P; p += nt) {
      const uint32_t lo = uint32_t(int(__builtin_rint(__builtin_fma(brow[2 * p], step, brow[2 * p] * low)))) & 0xFFu;
      const uint32_t hi = uint32_t(int(__builtin_rint(__builtin_fma(brow[2 * p + 1], step, brow[2 * p + 1] * low)))) & 0xFFu;
      reinterpret_cast<uint16_t*>(q + n * D)[p] = bad ? uint16_t(0) : uint16_t(lo | (hi << 8));
    }
    if (tid == 0) scales[n] = bad ? __builtin_nanf("") : float(c0 / 127.0);
    __syncthreads();  // the row and its maximum are done with
  }
}

}  // namespace

hipError_t launch_pack_q8(const DevRot& R, int N, int dtype, const void* W, int8_t* q, float* scales, hipStream_t st) {
  const size_t lds = size_t(R.D) * sizeof(double);
  const void* fn = dtype == PARO_F16 ? reinterpret_cast<const void*>(&pack_q8_kernel<PARO_F16>)
                                     : reinterpret_cast<const void*>(&pack_q8_kernel<PARO_BF16>);
  if (lds + 64 > 64 * 1024)
    if (hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, int(lds))) return e;
  const int share = N <= 256 ? 1 : 4;  // pairs of a thread per stage
  const int nt = std::min(1024, (R.D / 2 / share + 63) / 64 * 64);
  const dim3 grid(unsigned(std::min(N, 1 << 20)));
  if (dtype == PARO_F16)
    hipLaunchKernelGGL((pack_q8_kernel<PARO_F16>), grid, dim3(nt), lds, st, N, R.D, R.K, static_cast<const uint16_t*>(W), R.rec,
                       R.s, q, scales);
  else
    hipLaunchKernelGGL((pack_q8_kernel<PARO_BF16>), grid, dim3(nt), lds, st, N, R.D, R.K, static_cast<const uint16_t*>(W), R.rec,
                       R.s, q, scales);
  return hipGetLastError();
}

}  // namespace paro
