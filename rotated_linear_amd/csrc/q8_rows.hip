// Row kernels of the 8-bit path: residual addition + RMS norm (8-bit or 16-bit output), the row
// quantiser, and reading 8-bit rows back. All are bound by HBM: one pass over the row, which stays
// in registers between its statistics and its output. Measured (graph replays, cold rows): rmsnorm_q8 with
// residual 4096 x 4096 bf16 25.4 us (7 bytes a channel, 4.6 TB/s; a copy of 1 GiB runs at 4.7), rmsnorm
// 26.1 us (8 bytes, 5.1 TB/s), quantiser 13.0 us (3.9 TB/s), read-back 12.3 us (4.1 TB/s); a single row of
// 4096 2.7, 2.4, 2.1 and 1.9 us, a launch.
#include <algorithm>

#include "q8_device.h"

namespace paro {
namespace {

constexpr int kCUs = 256;

// One step of a reduction over the wave's lanes by data-parallel moves (row shifts, then broadcasts):
// lane 63 ends with the result. Lanes without a source keep `v` out of it (max with 0, plus 0).
template <int CTRL, int ROWS>
__device__ inline uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ inline void wave_step(uint32_t& top, double& sum, bool with_sum) {
  top = max(top, dpp<CTRL, ROWS>(top));
  if (with_sum) {
    const uint64_t b = __builtin_bit_cast(uint64_t, sum);
    sum += __builtin_bit_cast(double, uint64_t(dpp<CTRL, ROWS>(uint32_t(b))) | uint64_t(dpp<CTRL, ROWS>(uint32_t(b >> 32))) << 32);
  }
}
__device__ inline void wave_reduce(uint32_t& top, double& sum, bool with_sum) {
  wave_step<0x111, 0xF>(top, sum, with_sum);  // row_shr:1, 2, 4, 8
  wave_step<0x112, 0xF>(top, sum, with_sum);
  wave_step<0x114, 0xF>(top, sum, with_sum);
  wave_step<0x118, 0xF>(top, sum, with_sum);
  wave_step<0x142, 0xA>(top, sum, with_sum);  // row_bcast:15 into rows 1 and 3
  wave_step<0x143, 0xC>(top, sum, with_sum);  // row_bcast:31 into rows 2 and 3
}

// A workgroup walks rows blockIdx.x, + gridDim.x, ...; a thread holds VPT chunks of 8 channels. The
// next row is loaded before this row's statistics are complete. NORM: the norm, else v = x.
//
// With t = float32(h * gamma) and inv = float32(1 / sqrt(mean(h^2) + eps)), n = t * inv. Rounding is
// monotonic, so the row's largest |n| is the largest |t| times inv: one reduction (the sum of squares
// in float64 and the largest |t|) gives both the norm and the scale. The codes are those of t over its
// own maximum, the same numbers without the rounding of the product with inv.
//
// bfloat16 rows reach float32's ends: h * gamma may pass its range, or lose digits under 2^-126, where n is
// an ordinary number, and inv too may lie under 2^-126. Such a row (one branch for the whole workgroup,
// after the reduction) is read again and its n worked out in float64, with a reduction of its own.
// float16 rows stay within 2^-48 .. 2^32 and have no such branch.
template <int DT, bool NORM, bool Q8, int VPT>
__global__ __launch_bounds__(1024) void rows_kernel(const NormArgs a) {
  __shared__ uint32_t stop[2][16], ntop64[2][16];
  __shared__ double ssum[2][16];
  const int tid = threadIdx.x, nt = blockDim.x, waves = nt / 64;
  const int chunks = a.D / 8;
  const u32x4* const x = static_cast<const u32x4*>(a.x);
  const u32x4* const res = static_cast<const u32x4*>(a.residual);
  u32x4* const ro = static_cast<u32x4*>(a.residual_out);
  u32x4 gw[VPT], xw[VPT], rw[VPT];
  auto load = [&](size_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * nt;
      if (c < chunks) {
        xw[i] = x[row * chunks + c];
        if (NORM && res) rw[i] = res[row * chunks + c];
      }
    }
  };
  size_t row = blockIdx.x;
  load(row);
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (tid + i * nt < chunks) gw[i] = static_cast<const u32x4*>(a.gamma)[tid + i * nt];
  }
  for (int parity = 0;; parity ^= 1) {
    float t[VPT][8];
    u32x4 hw[VPT];
    uint32_t top = 0;
    double sum = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const bool live = tid + i * nt < chunks;
      float h[8];
      unpack8<DT>(xw[i], h);
      if constexpr (NORM) {
        if (res) {
          float r[8];
          unpack8<DT>(rw[i], r);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[e] += r[e];
          hw[i] = pack8<DT>(h);
          unpack8<DT>(hw[i], h);
        }
        float g[8];
        unpack8<DT>(gw[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[i][e] = h[e] * g[e];
        double s = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __builtin_fma(double(h[e]), double(h[e]), s);
        sum += live ? s : 0.0;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[i][e] = h[e];
      }
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, abs_order(t[i][e]));
      top = max(top, live ? m : 0u);
    }
    const size_t next = row + gridDim.x;
    if (next < size_t(a.M)) load(next);  // uniform
    if (NORM && res) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (tid + i * nt < chunks) ro[row * chunks + tid + i * nt] = hw[i];
    }
    float inv = 1.0f;
    RowQuant rq{};
    if (NORM || Q8) {
      wave_reduce(top, sum, NORM);
      if ((tid & 63) == 63) {
        stop[parity][tid >> 6] = top;
        if constexpr (NORM) ssum[parity][tid >> 6] = sum;
      }
      __syncthreads();  // one per row: the other parity's slots are rewritten only after the next one
      top = 0;
      sum = 0;
#pragma unroll 4
      for (int w = 0; w < waves; ++w) {  // (more sums at once would take the registers of a second workgroup)
        top = max(top, stop[parity][w]);
        if constexpr (NORM) sum += ssum[parity][w];
      }
      if constexpr (NORM) {
        const double inv64 = 1.0 / __builtin_sqrt(sum / a.D + double(a.eps));
        inv = float(inv64);
        uint32_t ntop = abs_order(__builtin_bit_cast(float, top) * inv);
        constexpr uint32_t kMinBits = __builtin_bit_cast(uint32_t, kQ8MinTop);
        if constexpr (DT == PARO_BF16) {
          // (beside a top of 2^-100 or more, what a product under 2^-126 loses is less than 2^-49 of it)
          if (top >= kAbsInf || (top < kMinBits && sum != 0) || inv < 0x1p-126f) {  // uniform
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
              const int c = tid + i * nt;
              if (c < chunks) {
                const u32x4* const from = res ? ro : x;  // (h: this thread's own stores)
                const u32x4 hr = from[row * chunks + c];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                  uint32_t gv = gw[i][w];
                  asm volatile("" : "+v"(gv));  // converted here again, not kept as floats from above
                  t[i][2 * w] = float(double(from_bits16<DT>(hr[w] & 0xFFFFu)) * double(from_bits16<DT>(gv & 0xFFFFu)) * inv64);
                  t[i][2 * w + 1] = float(double(from_bits16<DT>(hr[w] >> 16)) * double(from_bits16<DT>(gv >> 16)) * inv64);
                  m = max(m, max(abs_order(t[i][2 * w]), abs_order(t[i][2 * w + 1])));
                }
              }
            }
            double none = 0;
            wave_reduce(m, none, false);
            if ((tid & 63) == 63) ntop64[parity][tid >> 6] = m;
            __syncthreads();
            for (int w = 0; w < waves; ++w) m = max(m, ntop64[parity][w]);
            ntop = top = m;
            inv = 1.0f;
          }
        }
        // (a row under the smallest scale, or t under it, takes its codes from n itself)
        const bool from_t = Q8 && ntop >= kMinBits && top >= kMinBits;
        rq = row_quant(ntop, from_t ? top : ntop);
        if (from_t) inv = 1.0f;
      } else {
        rq = row_quant(top);
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * nt;
      if (NORM) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[i][e] *= inv;
      }
      if (c < chunks) {
        if constexpr (Q8) {
          uint2 q = make_uint2(codes4(t[i][0], t[i][1], t[i][2], t[i][3], rq),
                               codes4(t[i][4], t[i][5], t[i][6], t[i][7], rq));
          if (rq.bad) q = make_uint2(0, 0);
          reinterpret_cast<uint2*>(a.q)[row * chunks + c] = q;
        } else {
          static_cast<u32x4*>(a.y)[row * chunks + c] = pack8<DT>(t[i]);
        }
      }
    }
    if (Q8 && tid == 0) a.scales[row] = rq.scale;
    if (next >= size_t(a.M)) break;
    row = next;
  }
}

// Threads take 8 codes each: a wave reads and writes whole lines.
template <int DT>
__global__ __launch_bounds__(256) void dequantize_kernel(size_t total, uint32_t per_row, const uint2* q,
                                                         const float* scales, u32x4* x) {
  for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += size_t(gridDim.x) * 256) {
    const float s = scales[total <= 0xFFFFFFFFu ? uint32_t(i) / per_row : i / per_row];
    const uint2 w = q[i];
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = float(int8_t((k < 4 ? w.x : w.y) >> (8 * (k % 4)))) * s;
    if constexpr (DT == PARO_F32) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        x[2 * i + k] = u32x4{__builtin_bit_cast(uint32_t, f[4 * k]), __builtin_bit_cast(uint32_t, f[4 * k + 1]),
                             __builtin_bit_cast(uint32_t, f[4 * k + 2]), __builtin_bit_cast(uint32_t, f[4 * k + 3])};
    } else {
      x[i] = pack8<DT>(f);
    }
  }
}

template <int DT, bool NORM, bool Q8>
hipError_t launch_rows(const NormArgs& a, hipStream_t st) {
  const int chunks = a.D / 8;
  // Few rows: as many threads as chunks (latency). Many rows: two chunks a thread, whose next row is on
  // its way.
  const int vpt = chunks > 1024 || (a.M >= 512 && chunks > 64) ? 2 : 1;
  const int nt = std::max(64, ((chunks + vpt - 1) / vpt + 63) / 64 * 64);
  const unsigned grid = unsigned(std::min(a.M, kCUs * (2048 / nt)));
  if (vpt == 2)
    hipLaunchKernelGGL((rows_kernel<DT, NORM, Q8, 2>), dim3(grid), dim3(nt), 0, st, a);
  else
    hipLaunchKernelGGL((rows_kernel<DT, NORM, Q8, 1>), dim3(grid), dim3(nt), 0, st, a);
  return hipGetLastError();
}

template <bool NORM, bool Q8>
hipError_t launch_rows(const NormArgs& a, hipStream_t st) {
  return a.dtype == PARO_F16 ? launch_rows<PARO_F16, NORM, Q8>(a, st) : launch_rows<PARO_BF16, NORM, Q8>(a, st);
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
  const size_t total = size_t(M) * (D / 8);
  const dim3 grid(unsigned(std::min<size_t>((total + 255) / 256, 1 << 16)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, total, uint32_t(D / 8), reinterpret_cast<const uint2*>(q), scales,
                       static_cast<u32x4*>(x));
    return hipGetLastError();
  };
  return go(dtype == PARO_F16 ? dequantize_kernel<PARO_F16> : dtype == PARO_BF16 ? dequantize_kernel<PARO_BF16> : dequantize_kernel<PARO_F32>);
}

}  // namespace paro
