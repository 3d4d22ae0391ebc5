// Build-time weights in 8 bits: each row of W, with the transform folded in or as it is, quantised
// in float64 by its largest magnitude.
//
// One workgroup per weight row, the row in LDS as float64. Every stage gathers and rewrites the row: at D =
// 4096 about 27 us a 4096 rows at LDS's full rate, and as much again for some 16 float64 instructions a pair.
// The two hardly overlap. Measured (graph replays, cold W), K = 8: 4096 x 4096 73.6 us, 1024 x 14336 86, 256 x
// 1536 6.4. Rows without a transform take the same passes with no stages: 4096 x 4096 26.2 us (10.6 of bytes),
// 28672 x 4096 154, 4096 x 14336 118, 256 x 1536 3.6. Two or four rows a workgroup, which read a record once for all, were no faster (77 us
// where this takes 70): the records come from L2 in time, and wider LDS accesses move no more bytes a
// cycle. Loading the next stage's records ahead did not pay either: it takes registers, and with them the
// waves that hide LDS's latency. Compiled with -ffp-contract=off: each product and each sum of the fold is
// rounded on its own, so the codes are those of the stated definition (the quantiser asks for its fused
// products by name).
#include <algorithm>

#include "q8_device.h"

namespace paro {
namespace {

// A thread takes U pairs of a stage at once (a stage's pairs are disjoint).
template <int DT, int U>
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
      const PairRec* const stage = recs + size_t(k) * P;
      for (int p = tid; p < P; p += U * nt) {
        PairRec rec[U];
        double bi[U], bj[U];
#pragma unroll
        for (int u = 0; u < U; ++u) rec[u] = stage[min(p + u * nt, P - 1)];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          bi[u] = brow[(rec[u].ij & 0xFFFFu) >> 2];  // the fields are 4 i and 4 j
          bj[u] = brow[rec[u].ij >> 18];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u && p + u * nt >= P) break;
          const double c = rec[u].c, sn = rec[u].s;
          brow[(rec[u].ij & 0xFFFFu) >> 2] = c * bi[u] + sn * bj[u];
          brow[rec[u].ij >> 18] = c * bj[u] - sn * bi[u];
        }
      }
      __syncthreads();
    }
    double top = 0, nan = 0;  // the largest |v| that is a number; NaN where any v is an infinity or a NaN
    for (int c = tid; c < D; c += nt) {
      double b = brow[c];
      if (s) brow[c] = b = b * static_cast<double>(s[c]);
      top = fmax(top, fabs(b));
      nan = __builtin_fma(b, 0.0, nan);
    }
    if (nan != nan) top = __builtin_inf();
    unsigned long long bits = __builtin_bit_cast(unsigned long long, top);
    for (int off = 32; off >= 1; off >>= 1) bits = max(bits, __shfl_xor(bits, off));
    if ((tid & 63) == 0) atomicMax(&stop, bits);
    __syncthreads();
    bits = stop;
    const bool bad = bits >= 0x7FF0000000000000ull;
    const double c0 = fmax(__builtin_bit_cast(double, bits), double(kQ8MinTop));
    // 127 / c0 to twice float64's precision, so that a weight half way between two codes stays there
    const double step = 127.0 / c0, low = __builtin_fma(-step, c0, 127.0) / c0;
    // 1.5 * 2^52 + v: v rounded to an integer, ties to even, in the low bits
    auto code = [&](double b) {
      const double v = __builtin_fma(b, step, b * low) + 0x1.8p52;
      return uint32_t(__builtin_bit_cast(unsigned long long, v)) & 0xFFu;
    };
    for (int p = tid; p < P; p += nt) {
      const uint32_t v = code(brow[2 * p]) | code(brow[2 * p + 1]) << 8;
      reinterpret_cast<uint16_t*>(q + n * D)[p] = bad ? uint16_t(0) : uint16_t(v);
    }
    if (tid == 0) scales[n] = bad ? __builtin_nanf("") : float(c0 / 127.0);
    __syncthreads();  // the row and its maximum are done with
  }
}

template <int DT, int U>
hipError_t launch(const DevRot& R, int N, int nt, const void* W, int8_t* q, float* scales, hipStream_t st) {
  const auto kernel = &pack_q8_kernel<DT, U>;
  const size_t lds = size_t(R.D) * sizeof(double);
  if (lds + 64 > 64 * 1024)
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, int(lds)))
      return e;
  hipLaunchKernelGGL(kernel, dim3(unsigned(std::min(N, 1 << 20))), dim3(nt), lds, st, N, R.D, R.K,
                     static_cast<const uint16_t*>(W), R.rec, R.s, q, scales);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pack_q8(const DevRot& R, int N, int dtype, const void* W, int8_t* q, float* scales, hipStream_t st) {
  // Few rows: a pair per thread and stage (16 x 4096: 10.4 us; with four 11.6). Many: four pairs a thread,
  // taken at once (4096 x 4096 with W in the Infinity Cache 70 us; one after the other 75).
  const int P = R.D / 2;
  const int nt = std::min(1024, (P / (N <= 256 ? 1 : 4) + 63) / 64 * 64);
  const bool four = P > 3 * nt;
  if (dtype == PARO_F16)
    return four ? launch<PARO_F16, 4>(R, N, nt, W, q, scales, st) : launch<PARO_F16, 1>(R, N, nt, W, q, scales, st);
  return four ? launch<PARO_BF16, 4>(R, N, nt, W, q, scales, st) : launch<PARO_BF16, 1>(R, N, nt, W, q, scales, st);
}

}  // namespace paro
