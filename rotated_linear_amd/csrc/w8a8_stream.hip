// The 8-bit products for a row or two of x: the weights are streamed once, straight into registers.
// Bound by HBM: M = 1, gated 4096 -> 14336 20.0 us, 5.9 TB/s of weights; 14336 -> 4096 12.3 us, 4.8
// TB/s; below about 20 MB by the launch and the first loads (4096 -> 4096 5.4 us).
#include "q8_device.h"

namespace paro {
namespace {

constexpr int kRing = 4;  // steps in flight per wave

// A workgroup of W waves owns WT tiles of R = 16 / P rows of w and all rows of x (up to R); its waves
// take turns with the steps of 64 P channels. A virtual operand row i (of the 16 that
// v_mfma_i32_16x16x64_i8 takes) is row i % R in part i / R of the step's channels, on both sides: the
// products of equal parts, P diagonal blocks, add up to the result, and a wave-wide load of w reads
// 64 P consecutive bytes of R rows. The matrix instructions idle anyway; wide pieces of a row and
// small tiles (so that narrow layers fill the GPU too) are what a short x gains by it.
template <int P, int WT, int W, bool GATED>
__global__ __launch_bounds__(64 * W) void w8a8_stream_kernel(const W8A8Call c) {
  constexpr int R = 16 / P;
  constexpr int YT = GATED ? WT / 2 : WT;  // tiles of y's columns
  __shared__ i32x4 red[W][WT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, h = lane >> 4;
  const int n0 = blockIdx.x * (YT * R);
  const size_t koff = (i / R) * 64 + h * 16;
  const i32x4* wp[WT];
#pragma unroll
  for (int t = 0; t < WT; ++t) {
    const int n = min(n0 + (GATED ? t % YT : t) * R + i % R, c.N - 1);
    const size_t row = GATED && t >= YT ? size_t(n) + c.N : size_t(n);
    wp[t] = reinterpret_cast<const i32x4*>(c.w + row * c.D + koff);
  }
  const i32x4* const xp = reinterpret_cast<const i32x4*>(c.x + size_t(min(i % R, c.M - 1)) * c.D + koff);

  const int steps = c.D / (64 * P);
  const int mine = (steps - wave + W - 1) / W;  // steps wave, wave + W, ...
  i32x4 acc[WT];
#pragma unroll
  for (int t = 0; t < WT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  i32x4 wr[kRing][WT], xr[kRing];
  auto load = [&](int slot, int s) {  // this wave's s-th step
    const size_t k = size_t(wave + s * W) * (4 * P);
#pragma unroll
    for (int t = 0; t < WT; ++t) wr[slot][t] = __builtin_nontemporal_load(wp[t] + k);
    xr[slot] = xp[k];
  };
  auto mma = [&](int slot) {
#pragma unroll
    for (int t = 0; t < WT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wr[slot][t], xr[slot], acc[t], 0, 0, 0);
  };
  // Whole rounds of the ring load without a branch, so that the compiler's wait counts stay exact;
  // no step past the end is loaded (loading the last step again instead took 10.0 us where this
  // takes 5.4: M = 1, D = N = 4096).
#pragma unroll
  for (int q = 0; q < kRing; ++q)
    if (q < mine) load(q, q);
  int s = 0;
  for (; s + 2 * kRing <= mine; s += kRing) {
#pragma unroll
    for (int q = 0; q < kRing; ++q) {
      mma(q);
      load(q, s + kRing + q);
    }
  }
#pragma unroll
  for (int q = 0; q < kRing; ++q) {
    if (s + q < mine) mma(q);
    if (s + kRing + q < mine) load(q, s + kRing + q);
  }
#pragma unroll
  for (int q = 0; q < kRing - 1; ++q)
    if (s + kRing + q < mine) mma(q);
#pragma unroll
  for (int t = 0; t < WT; ++t) red[wave][t][i * 4 + h] = acc[t];  // [row of x][row of w]: ints i * 16 + 4 h + e
  __syncthreads();

  // y[m][n]: the waves' sums and the P diagonal blocks
  const int* const sums = reinterpret_cast<const int*>(red);
  const int cols = YT * R;
  for (int o = threadIdx.x; o < cols * c.M; o += 64 * W) {
    const int nn = o % cols, m = o / cols, n = n0 + nn;
    if (n >= c.N) continue;
    const int t = nn / R, r = nn % R;
    auto sum = [&](int tile) {
      int v = 0;
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int p = 0; p < P; ++p) v += sums[((w * WT + tile) * 16 + m + p * R) * 16 + r + p * R];
      return v;
    };
    const float xs = c.xs[m];
    float v = scaled(sum(t), xs, c.ws[n]);
    if constexpr (GATED) {
      const float u = scaled(sum(t + YT), xs, c.ws[size_t(c.N) + n]);
      v = c.ydtype == PARO_F32 ? silu_mul<PARO_F32>(v, u) : silu_mul<PARO_F16>(v, u);
    }
    const size_t at = size_t(m) * c.N + n;
    if (c.ydtype == PARO_F32)
      static_cast<float*>(c.y)[at] = v;
    else
      static_cast<uint16_t*>(c.y)[at] = uint16_t(c.ydtype == PARO_F16 ? to_bits16<PARO_F16>(v) : to_bits16<PARO_BF16>(v));
  }
}

template <int P, int WT, int W, bool GATED>
hipError_t launch(const W8A8Call& c, hipStream_t st) {
  constexpr int cols = 16 / P * (GATED ? WT / 2 : WT);
  hipLaunchKernelGGL((w8a8_stream_kernel<P, WT, W, GATED>), dim3((c.N + cols - 1) / cols), dim3(64 * W), 0, st, c);
  return hipGetLastError();
}

// Eight waves where there is at most one workgroup per CU, else four. Measured on MI355X, cold
// weights: M = 1, 8960 -> 1536 (192 workgroups) 5.0 us with eight, 5.8 with four; gated 4096 -> 14336
// (3584) 20.3 and 18.9 us (6.2 TB/s).
template <int P, bool GATED>
hipError_t launch_waves(const W8A8Call& c, hipStream_t st) {
  constexpr int cols = 16 / P * (GATED ? 1 : 2);
  return (c.N + cols - 1) / cols <= 256 ? launch<P, 2, 8, GATED>(c, st) : launch<P, 2, 4, GATED>(c, st);
}

template <bool GATED>
hipError_t launch_rows(const W8A8Call& c, hipStream_t st) {
  return c.D % 256 == 0 ? launch_waves<4, GATED>(c, st) : launch_waves<2, GATED>(c, st);
}

}  // namespace

// Measured against the kernel that brings x and w through LDS, cold weights: M = 1, 4096 -> 4096 5.2
// us here, 5.2 there; 8960 -> 1536 5.0 and 6.2; gated 4096 -> 14336 19.0 and 21.4. From a few rows on
// the other is ahead: M = 4, 14336 -> 4096 12.3 and 12.1; M = 8, 8960 -> 1536 9.1 and 7.0.
// (A grid of more than 2^32 threads cannot be launched: layers of more than 2^24 columns go to the
// tiled kernel, whose grid does not grow with them.)
bool w8a8_stream_takes(int M, int N) { return M <= 2 && N <= 1 << 24; }

hipError_t launch_w8a8_stream(const W8A8Call& c, hipStream_t st) {
  return c.gated ? launch_rows<true>(c, st) : launch_rows<false>(c, st);
}

}  // namespace paro
