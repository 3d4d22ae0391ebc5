// Row kernels of the 8-bit path: residual addition + RMS norm (8-bit or 16-bit output), the row
// quantiser, and reading 8-bit rows back.
#include "q8_device.h"

namespace paro {
namespace {

constexpr int kRowThreads = 256;

// Maximum (as abs_order) and float64 sum over the workgroup.
__device__ inline void block_reduce(uint32_t& top, double& sum) {
  __shared__ uint32_t stop[kRowThreads / 64];
  __shared__ double ssum[kRowThreads / 64];
  for (int off = 32; off >= 1; off >>= 1) {
    top = max(top, uint32_t(__shfl_xor(int(top), off)));
    sum += __shfl_xor(sum, off);
  }
  if ((threadIdx.x & 63) == 0) {
    stop[threadIdx.x >> 6] = top;
    ssum[threadIdx.x >> 6] = sum;
  }
  __syncthreads();
  top = stop[0];
  sum = ssum[0];
  for (int w = 1; w < kRowThreads / 64; ++w) {
    top = max(top, stop[w]);
    sum += ssum[w];
  }
}

// One workgroup per row. NORM: the norm, else v = x.
template <int DT, bool NORM, bool Q8>
__global__ __launch_bounds__(kRowThreads) void rows_kernel(const NormArgs a) {
  const size_t row = blockIdx.x;
  const int chunks = a.D / 8;
  const u32x4* x = reinterpret_cast<const u32x4*>(a.x) + row * chunks;
  const u32x4* res = a.residual ? reinterpret_cast<const u32x4*>(a.residual) + row * chunks : nullptr;
  u32x4* ro = a.residual_out ? reinterpret_cast<u32x4*>(a.residual_out) + row * chunks : nullptr;
  const u32x4* gamma = reinterpret_cast<const u32x4*>(a.gamma);
  // t = h * gamma in float32 (v = x without the norm)
  auto load = [&](int c, float(&h)[8], float(&t)[8]) {
    unpack8<DT>(x[c], h);
    if constexpr (NORM) {
      if (res) {
        float r[8];
        unpack8<DT>(res[c], r);
        for (int i = 0; i < 8; ++i) h[i] = from_bits16<DT>(to_bits16<DT>(h[i] + r[i]));
      }
      float g[8];
      unpack8<DT>(gamma[c], g);
      for (int i = 0; i < 8; ++i) t[i] = h[i] * g[i];
    } else {
      for (int i = 0; i < 8; ++i) t[i] = h[i];
    }
  };
  uint32_t top = 0;
  double sum = 0;
  for (int c = threadIdx.x; c < chunks; c += kRowThreads) {
    float h[8], t[8];
    load(c, h, t);
    for (int i = 0; i < 8; ++i) {
      top = max(top, abs_order(t[i]));
      if constexpr (NORM) sum += double(h[i]) * double(h[i]);
    }
  }
  block_reduce(top, sum);
  float inv = 1.0f;
  if constexpr (NORM) {
    inv = float(1.0 / sqrt(sum / a.D + double(a.eps)));
    top = abs_order(__builtin_bit_cast(float, top) * inv);
  }
  const RowQuant rq = row_quant(top);
  for (int c = threadIdx.x; c < chunks; c += kRowThreads) {
    float h[8], t[8];
    load(c, h, t);
    for (int i = 0; i < 8; ++i) t[i] = t[i] * inv;
    if (NORM && ro) ro[c] = pack8<DT>(h);
    if constexpr (Q8) {
      const float lo[4] = {t[0], t[1], t[2], t[3]}, hi[4] = {t[4], t[5], t[6], t[7]};
      uint32_t* q = reinterpret_cast<uint32_t*>(a.q + row * a.D) + 2 * c;
      q[0] = rq.bad ? 0u : codes4(lo, rq.step);
      q[1] = rq.bad ? 0u : codes4(hi, rq.step);
    } else {
      reinterpret_cast<u32x4*>(a.y)[row * chunks + c] = pack8<DT>(t);
    }
  }
  if (Q8 && threadIdx.x == 0) a.scales[row] = rq.scale;
}

template <int DT>
__global__ __launch_bounds__(kRowThreads) void dequantize_kernel(int M, int D, const int8_t* q, const float* scales,
                                                                 void* x) {
  const size_t i = size_t(blockIdx.x) * kRowThreads + threadIdx.x;  // 8 codes each
  if (i >= size_t(M) * (D / 8)) return;
  const float s = scales[i / (D / 8)];
  float f[8];
  for (int k = 0; k < 8; ++k) f[k] = float(q[8 * i + k]) * s;
  if constexpr (DT == PARO_F32) {
    for (int k = 0; k < 8; ++k) reinterpret_cast<float*>(x)[8 * i + k] = f[k];
  } else {
    reinterpret_cast<u32x4*>(x)[i] = pack8<DT>(f);
  }
}

template <bool NORM, bool Q8>
hipError_t launch_rows(const NormArgs& a, hipStream_t st) {
  if (a.dtype == PARO_F16)
    hipLaunchKernelGGL((rows_kernel<PARO_F16, NORM, Q8>), dim3(a.M), dim3(kRowThreads), 0, st, a);
  else
    hipLaunchKernelGGL((rows_kernel<PARO_BF16, NORM, Q8>), dim3(a.M), dim3(kRowThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st) {
  return a.q ? launch_rows<true, true>(a, st) : launch_rows<true, false>(a, st);
}

hipError_t launch_quantize_q8(int M, int D, int dtype, const void* x, int8_t* q, float* scales, hipStream_t st) {
  NormArgs a{};
  a.M = M;
  a.D = D;
  a.dtype = dtype;
  a.x = x;
  a.q = q;
  a.scales = scales;
  return launch_rows<false, true>(a, st);
}

hipError_t launch_dequantize_q8(int M, int D, const int8_t* q, const float* scales, void* x, int dtype,
                                hipStream_t st) {
  const unsigned grid = unsigned((size_t(M) * (D / 8) + kRowThreads - 1) / kRowThreads);
  if (dtype == PARO_F16)
    hipLaunchKernelGGL((dequantize_kernel<PARO_F16>), dim3(grid), dim3(kRowThreads), 0, st, M, D, q, scales, x);
  else if (dtype == PARO_BF16)
    hipLaunchKernelGGL((dequantize_kernel<PARO_BF16>), dim3(grid), dim3(kRowThreads), 0, st, M, D, q, scales, x);
  else
    hipLaunchKernelGGL((dequantize_kernel<PARO_F32>), dim3(grid), dim3(kRowThreads), 0, st, M, D, q, scales, x);
  return hipGetLastError();
}

}  // namespace paro
