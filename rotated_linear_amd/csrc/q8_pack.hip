// Build-time weights in 8 bits: each row of W, with the transform folded in or as it is, quantised
// in float64 by its largest magnitude.
//
// One workgroup per weight row, the row in LDS as float64. Compiled with -ffp-contract=off: each
// product and each sum is rounded on its own, so the codes are those of the stated definition.
#include "q8_device.h"

namespace paro {
namespace {

constexpr int kThreads = 256;

template <int DT>
__global__ __launch_bounds__(kThreads) void pack_q8_kernel(int D, int K, const uint16_t* W, const PairRec* recs,
                                                           const float* s, int8_t* q, float* scales) {
  extern __shared__ double brow[];  // [D]
  __shared__ unsigned long long stop;
  const size_t n = blockIdx.x;
  if (threadIdx.x == 0) stop = 0;
  for (int c = threadIdx.x; c < D; c += kThreads) brow[c] = from_bits16<DT>(W[n * D + c]);
  __syncthreads();
  const int P = D / 2;
  for (int k = 0; k < K; ++k) {
    for (int p = threadIdx.x; p < P; p += kThreads) {
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
  for (int c = threadIdx.x; c < D; c += kThreads) {
    if (s) brow[c] = brow[c] * static_cast<double>(s[c]);
    top = max(top, __builtin_bit_cast(unsigned long long, brow[c]) & 0x7FFFFFFFFFFFFFFFull);
  }
  atomicMax(&stop, top);
  __syncthreads();
  top = stop;
  const bool bad = top >= 0x7FF0000000000000ull;
  const double c0 = fmax(__builtin_bit_cast(double, top), double(kQ8MinTop));
  const double step = 127.0 / c0;
  for (int c = threadIdx.x; c < D; c += kThreads)
    q[n * D + c] = bad ? int8_t(0) : int8_t(__builtin_rint(brow[c] * step));
  if (threadIdx.x == 0) scales[n] = bad ? __builtin_nanf("") : float(c0 / 127.0);
}

}  // namespace

hipError_t launch_pack_q8(const DevRot& R, int N, int dtype, const void* W, int8_t* q, float* scales, hipStream_t st) {
  const size_t lds = size_t(R.D) * sizeof(double);
  auto fn = dtype == PARO_F16 ? pack_q8_kernel<PARO_F16> : pack_q8_kernel<PARO_BF16>;
  if (lds + 64 > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                                       int(lds));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3(N), dim3(kThreads), lds, st, R.D, R.K, static_cast<const uint16_t*>(W), R.rec, R.s, q,
                     scales);
  return hipGetLastError();
}

}  // namespace paro
