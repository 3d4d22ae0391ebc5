// The 8-bit products for a short batch of x: a workgroup owns 16 columns of y and all rows of x, and
// its waves share out the channels, so no sum leaves the workgroup.
#include <algorithm>
#include <cmath>

#include "w8a8_dma.h"

namespace paro {
namespace {

// FM fragments of 16 rows of x against 16 rows of w (kGated: 16 gate and 16 up rows). Wave s takes the
// steps s, s + W, ... of 128 channels: rows of x and w come straight into a ring of S stages of its
// own in LDS, S steps ahead, so the waves never wait for each other until their sums are added.
//
// Bound by HBM up to 32 rows (M = 16, 14336 -> 4096: 13.4 us, 4.4 TB/s of weights; gated 4096 ->
// 14336: 23.3 us, 5.0 TB/s; M = 32, 4096 -> 4096: 6.8 us); at 64 rows, where a CU pulls four bytes of
// x for each byte of w, by the CU's loads: about 52 bytes a ns, x and w together (w alone or x alone
// would take half the time, but a wave's loads end in order, so a stage waits for both). Each
// workgroup starts its walk over the channels one step after its neighbour, since rows a multiple of
// 2 KB apart lie in the same L2 channel: M = 12, 4096 -> 4096 6.0 -> 5.4 us.
// Tried: a wave of its own that touches the weights ahead of the others (64 x 14336 -> 4096 23.9 ->
// 25.5 us), w's loads before x's (no change).
template <int FM, Output KIND, int W, int S>
__global__ __launch_bounds__(64 * W) void w8a8_column_kernel(const W8A8Call c) {
  constexpr bool GATED = KIND == kGated;
  constexpr int WN = GATED ? 2 : 1;
  constexpr int ROWS = 16 * (FM + WN), STAGE = ROWS * 128, LOADS = ROWS / 8;
  extern __shared__ __attribute__((aligned(1024))) char smem[];  // [W][S][STAGE]
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 16;

  const char* const xb = reinterpret_cast<const char*>(c.x);
  const char* const wb = reinterpret_cast<const char*>(c.w) + size_t(n0) * c.D;
  const char* const ub = wb + size_t(c.N) * c.D;
  uint32_t voff[LOADS];  // rows past the end are the last row again
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int row = i * 8 + lane / 8;
    const uint32_t ch = ((lane % 8) * 16) ^ (swz(row, 0) - row * 128);  // the chunk that this slot holds
    const int r = i < 2 * FM ? min(row, c.M - 1) : min((row - 16 * FM) & 15, c.N - 1 - n0);
    voff[i] = uint32_t(r) * uint32_t(c.D) + ch;
  }
  char* const ring = smem + wave * S * STAGE;
  const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_address(ring));
  const int steps = c.D / 128;
  const int mine = (steps - wave + W - 1) / W;
  const int start = int(blockIdx.x / 8) % steps;  // neighbours on an XCD are 8 workgroups apart
  auto issue = [&](int s, uint32_t buf) {  // this wave's step s
    int t = wave + s * W + start;
    if (t >= steps) t -= steps;
    const size_t k = size_t(t) * 128;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      dma16(lds + buf * STAGE + i * 1024, voff[i], (i < 2 * FM ? xb : i < 2 * FM + 2 ? wb : ub) + k);
  };

  // An epilogue's operands, on their way while the sums are formed.
  constexpr int OUTS = (FM * 256 + 64 * W - 1) / (64 * W);  // outputs of a thread
  float bias[OUTS], res[OUTS];
  if constexpr (KIND == kEpilogue) {
#pragma unroll
    for (int i = 0; i < OUTS; ++i) {
      const int o = threadIdx.x + i * 64 * W, n = n0 + o % 16, m = o / 16;
      bias[i] = c.bias && n < c.N ? load_element(c.bias, n, c.ydtype) : 0.0f;
      res[i] = c.residual && n < c.N && m < c.M ? load_element(c.residual, size_t(m) * c.N + n, c.ydtype) : 0.0f;
    }
  }

  i32x4 acc[WN][FM];
#pragma unroll
  for (int j = 0; j < WN; ++j)
#pragma unroll
    for (int f = 0; f < FM; ++f) acc[j][f] = i32x4{0, 0, 0, 0};
  if (mine > 0) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s < mine) issue(s, s);
    uint32_t buf = 0;
    for (int s = 0; s < mine; ++s) {
      // stages s + 1 .. s + S - 1 may still be on their way; near the end fewer were asked for
      if (s + S <= mine)
        asm volatile("s_waitcnt vmcnt(%0)" : : "n"((S - 1) * LOADS) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
      i32x4 fx[2][FM], fw[2][WN];
      const char* const st = ring + buf * STAGE;
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        const uint32_t ch = sub * 4 + (lane >> 4);
#pragma unroll
        for (int f = 0; f < FM; ++f) fx[sub][f] = *reinterpret_cast<const i32x4*>(st + swz(f * 16 + (lane & 15), ch));
#pragma unroll
        for (int j = 0; j < WN; ++j)
          fw[sub][j] = *reinterpret_cast<const i32x4*>(st + swz((FM + j) * 16 + (lane & 15), ch));
      }
      if (s + S < mine) {
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");  // the stage has been read: its buffer is free
        issue(s + S, buf);
      }
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
          for (int f = 0; f < FM; ++f)
            acc[j][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[sub][j], fx[sub][f], acc[j][f], 0, 0, 0);
      buf = buf + 1 == S ? 0 : buf + 1;
    }
  }
  // the wave's sums over its own stages (its loads have all been waited for): [gate / up][row of x][column of y]
  static_assert(WN * FM * 1024 <= S * STAGE, "the sums fit in a wave's ring");
  i32x4* const red = reinterpret_cast<i32x4*>(ring);
#pragma unroll
  for (int j = 0; j < WN; ++j)
#pragma unroll
    for (int f = 0; f < FM; ++f) red[(j * FM * 16 + f * 16 + (lane & 15)) * 4 + (lane >> 4)] = acc[j][f];
  __syncthreads();
  const int* const sums = reinterpret_cast<const int*>(smem);
#pragma unroll
  for (int i = 0; i < OUTS; ++i) {
    const int o = threadIdx.x + i * 64 * W, n = n0 + o % 16, m = o / 16;
    if (n >= c.N || m >= c.M) continue;
    int v[WN];
#pragma unroll
    for (int j = 0; j < WN; ++j) {
      v[j] = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) v[j] += sums[w * (S * STAGE / 4) + j * FM * 256 + o];
    }
    const float xs = c.xs[m];
    float y = scaled(v[0], xs, c.ws[n]);
    if constexpr (GATED) {
      const float u = scaled(v[1], xs, c.ws[size_t(c.N) + n]);
      y = c.ydtype == PARO_F32 ? silu_mul<PARO_F32>(y, u) : silu_mul<PARO_F16>(y, u);
    }
    if constexpr (KIND == kEpilogue) y = epilogue(c, y, bias[i], res[i]);
    const size_t at = size_t(m) * c.N + n;
    if (c.ydtype == PARO_F32)
      static_cast<float*>(c.y)[at] = y;
    else
      static_cast<uint16_t*>(c.y)[at] = uint16_t(c.ydtype == PARO_F16 ? to_bits16<PARO_F16>(y) : to_bits16<PARO_BF16>(y));
  }
}

template <int FM, Output KIND, int W, int S>
hipError_t launch(const W8A8Call& c, hipStream_t st) {
  constexpr int lds = W * S * (FM + (KIND == kGated ? 2 : 1)) * 2048;
  static_assert(lds <= 160 * 1024, "one CU's LDS");
  const void* fn = reinterpret_cast<const void*>(&w8a8_column_kernel<FM, KIND, W, S>);
  if (lds > 64 * 1024)
    if (hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds)) return e;
  hipLaunchKernelGGL((w8a8_column_kernel<FM, KIND, W, S>), dim3((c.N + 15) / 16), dim3(64 * W), lds, st, c);
  return hipGetLastError();
}

// At most one workgroup per CU: eight waves of two stages (as many as fit of the widest). More: four
// waves, so that several workgroups share a CU. Measured: M = 8, 8960 -> 1536 7.0 us with eight waves,
// 8.4 with four; M = 16, gated 4096 -> 14336 26.8 and 23.3 us.
template <int FM, Output KIND>
hipError_t launch_waves(const W8A8Call& c, hipStream_t st) {
  if ((c.N + 15) / 16 > 256) return launch<FM, KIND, 4, 2>(c, st);
  if constexpr (FM == 4 && KIND == kGated)
    return launch<FM, KIND, 4, 3>(c, st);
  else
    return launch<FM, KIND, 8, 2>(c, st);
}

template <Output KIND>
hipError_t launch_rows(const W8A8Call& c, hipStream_t st) {
  if (c.M <= 16) return launch_waves<1, KIND>(c, st);
  if (c.M <= 32) return launch_waves<2, KIND>(c, st);
  return launch_waves<4, KIND>(c, st);
}

}  // namespace

// Estimated microseconds (compared with the tiled kernel's estimate): a launch, then the CU's loads
// and the weights' way from HBM, joined like the tiled kernel's. Within 15 % of 20 measured shapes.
double w8a8_column_us(int M, int D, int N, bool gated) {
  if (M > 64 || N > 1 << 24) return 1e30;
  const int rows = (M <= 16 ? 16 : M <= 32 ? 32 : 64) + (gated ? 32 : 16);
  const double loads = std::max(1.0, (N + 15) / 16 / 256.0) * rows * D / 52e3;
  const double hbm = double(N) * (gated ? 2 : 1) * D / 5.5e6;
  return 2.7 + std::cbrt(loads * loads * loads + hbm * hbm * hbm);
}

hipError_t launch_w8a8_column(const W8A8Call& c, hipStream_t st) {
  return c.epilogue ? launch_rows<kEpilogue>(c, st) : c.gated ? launch_rows<kGated>(c, st) : launch_rows<kPlain>(c, st);
}

}  // namespace paro
