// The 8-bit products: y = xs ws (xq . wq^T), and the gated pair of them.
//
// One wave per 16 x 16 tile of y (16 rows of w as the matrix instruction's A operand, 16 rows of x
// as its B), both read straight from memory, 64 channels per v_mfma_i32_16x16x64_i8.
#include "q8_device.h"

namespace paro {
namespace {

template <bool GATED>
__global__ __launch_bounds__(64) void w8a8_tile_kernel(const W8A8Call c) {
  const int lane = threadIdx.x;
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16;
  const int wr = min(n0 + (lane & 15), c.N - 1), xr = min(m0 + (lane & 15), c.M - 1);
  const i32x4* x = reinterpret_cast<const i32x4*>(c.x + size_t(xr) * c.D) + (lane >> 4);
  const i32x4* w = reinterpret_cast<const i32x4*>(c.w + size_t(wr) * c.D) + (lane >> 4);
  const i32x4* w2 = reinterpret_cast<const i32x4*>(c.w + (size_t(wr) + c.N) * c.D) + (lane >> 4);
  i32x4 acc = {0, 0, 0, 0}, acc2 = {0, 0, 0, 0};
  for (int k = 0; k < c.D / 16; k += 4) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[k], x[k], acc, 0, 0, 0);
    if constexpr (GATED) acc2 = __builtin_amdgcn_mfma_i32_16x16x64_i8(w2[k], x[k], acc2, 0, 0, 0);
  }
  const int m = m0 + (lane & 15);
  if (m >= c.M) return;
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + (lane >> 4) * 4 + i;
    if (n >= c.N) continue;
    float v = scaled(acc[i], c.xs[m], c.ws[n]);
    if constexpr (GATED) v = silu_mul(v, scaled(acc2[i], c.xs[m], c.ws[c.N + n]));
    const size_t at = size_t(m) * c.N + n;
    if (c.ydtype == PARO_F32)
      static_cast<float*>(c.y)[at] = v;
    else
      static_cast<uint16_t*>(c.y)[at] = c.ydtype == PARO_F16 ? to_bits16<PARO_F16>(v) : to_bits16<PARO_BF16>(v);
  }
}

}  // namespace

size_t w8a8_workspace_bytes(int M, int D, int N, bool gated) {
  return M > 64 ? w8a8_gemm_workspace_bytes(M, D, N, gated) : 0;
}

hipError_t launch_w8a8(const W8A8Call& c, void* work, hipStream_t st) {
  if (c.M > 64) return launch_w8a8_gemm(c, static_cast<int*>(work), st);
  const dim3 grid((c.N + 15) / 16, (c.M + 15) / 16);
  if (c.gated)
    hipLaunchKernelGGL((w8a8_tile_kernel<true>), grid, dim3(64), 0, st, c);
  else
    hipLaunchKernelGGL((w8a8_tile_kernel<false>), grid, dim3(64), 0, st, c);
  return hipGetLastError();
}

}  // namespace paro
