// The row quantiser behind the activation-side transform: K stages of disjoint-pair Givens
// rotations and the division by the channel scales in float32, then 8-bit codes.
#include "q8_device.h"

namespace paro {
namespace {

constexpr int kThreads = 256;

template <int DT>
__global__ __launch_bounds__(kThreads) void rotate_q8_kernel(int D, int K, const uint16_t* x, const PairRec* recs,
                                                             const float* inv_s, int8_t* q, float* scales) {
  extern __shared__ __attribute__((aligned(16))) float row[];  // [D]
  __shared__ uint32_t stop;
  const size_t m = blockIdx.x;
  if (threadIdx.x == 0) stop = 0;
  for (int c = threadIdx.x; c < D; c += kThreads) row[c] = from_bits16<DT>(x[m * D + c]);
  __syncthreads();
  const int P = D / 2;
  for (int k = 0; k < K; ++k) {
    for (int p = threadIdx.x; p < P; p += kThreads) {
      const PairRec r = recs[size_t(k) * P + p];
      const int i = int((r.ij & 0xFFFFu) >> 2), j = int(r.ij >> 18);  // the fields are 4 i and 4 j
      const float a = row[i], b = row[j];
      row[i] = __builtin_fmaf(r.c, a, r.s * b);
      row[j] = __builtin_fmaf(r.c, b, -(r.s * a));
    }
    __syncthreads();
  }
  uint32_t top = 0;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    row[c] *= inv_s[c];
    top = max(top, abs_order(row[c]));
  }
  atomicMax(&stop, top);
  __syncthreads();
  const RowQuant rq = row_quant(stop);
  for (int c = threadIdx.x; c < D; c += kThreads)
    q[m * D + c] = rq.bad ? int8_t(0) : int8_t(__builtin_rintf(row[c] * rq.step));
  if (threadIdx.x == 0) scales[m] = rq.scale;
}

}  // namespace

hipError_t launch_rotate_q8(const DevRot& R, int M, int dtype, const void* x, int8_t* q, float* scales,
                            hipStream_t st) {
  const size_t lds = size_t(R.D) * sizeof(float);
  auto fn = dtype == PARO_F16 ? rotate_q8_kernel<PARO_F16> : rotate_q8_kernel<PARO_BF16>;
  if (lds + 64 > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                                       int(lds));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3(M), dim3(kThreads), lds, st, R.D, R.K, static_cast<const uint16_t*>(x), R.rec, R.inv_s, q,
                     scales);
  return hipGetLastError();
}

}  // namespace paro
