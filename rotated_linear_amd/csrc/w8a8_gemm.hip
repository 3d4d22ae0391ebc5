// The 8-bit products for more rows than the streaming kernel takes: tiled matrix-core GEMM.
#include <algorithm>

#include "q8_device.h"
#include "w8a8_common.h"

namespace paro {
namespace {

constexpr int kCUs = 256;
constexpr int kXcds = 8;

// One 16-byte load per lane straight into LDS: lane l's bytes land at lds + 16 l. The compiler does
// not see the load, so the kernel waits for it itself (stage_wait); it has no output register.
__device__ inline void dma16(uint32_t lds, uint32_t voff, const void* base) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(voff), "s"(base)
      : "memory", "m0");
}
// All but the N youngest of this wave's loads have landed and its LDS reads are done; then the
// workgroup's waves meet.
template <int N>
__device__ inline void stage_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

struct GemmArgs {
  W8A8Call c;
  int* part;     // split partial sums [S][M][rows], or nullptr
  int tiles_m, tiles_n, splits, steps_per_split;
};

template <int BM_, int BN_, int WM_, int WN_, int BK_, int S_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, S = S_;
  static constexpr int NT = WM * WN * 64;
  static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;  // 32 x 32 fragments of a wave
  static constexpr int ROWS = BM + BN;
  static constexpr int STAGE = ROWS * BK;
  static constexpr int RPI = 1024 / BK;                // tile rows of one wave-wide load
  static constexpr int LOADS = ROWS / RPI / (WM * WN); // a wave's loads per stage
  static_assert(ROWS % (RPI * WM * WN) == 0, "loads divide over the waves");
  static constexpr int LDS = STAGE * S;
};

// 16-byte slot of a tile row's chunk c: rows of BK bytes, the chunk index mixed with the row so
// that 16 consecutive rows' chunk c lie in 16 distinct slots modulo 256 bytes.
template <int BK>
__device__ inline uint32_t swz(uint32_t row, uint32_t c) {
  if constexpr (BK == 64)
    return row * 64 + ((c ^ ((row >> 2) & 3)) << 4);
  else
    return row * 128 + ((c ^ ((row >> 1) & 7)) << 4);
}

template <class T, bool GATED>
__global__ __launch_bounds__(T::NT) void w8a8_gemm_kernel(const GemmArgs a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const W8A8Call& c = a.c;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;

  // XCD-aware order: workgroups go round the XCDs, each XCD takes a contiguous range of tiles.
  const int total = a.tiles_m * a.tiles_n * a.splits;
  const int per = total / kXcds, rem = total % kXcds;
  const int xcd = blockIdx.x % kXcds, idx = blockIdx.x / kXcds;
  int tile = xcd * per + min(xcd, rem) + idx;
  const int split = tile % a.splits;
  tile /= a.splits;
  // within a range: columns of GM tile rows
  constexpr int GM = 4;
  const int group = tile / (GM * a.tiles_n);
  const int gm0 = group * GM, gsz = min(GM, a.tiles_m - gm0);
  const int in = tile - group * GM * a.tiles_n;
  const int tm = gm0 + in % gsz, tn = in / gsz;

  const int m0 = tm * T::BM;
  // columns of y per tile: a gated tile's rows of w alternate, 32 gate rows then their 32 up rows
  constexpr int YN = GATED ? T::BN / 2 : T::BN;
  const int n0 = tn * YN;

  // this lane's source offsets (x rows first, then w rows), rows past the end clamped to the last
  uint32_t voff[T::LOADS];
  const char* src[T::LOADS];
  const int8_t* xb = c.x + size_t(m0) * c.D;
  const int8_t* wb = c.w + size_t(n0) * c.D;
#pragma unroll
  for (int i = 0; i < T::LOADS; ++i) {
    const int r0 = (wave * T::LOADS + i) * T::RPI;  // first tile row of the load
    const int lr = lane / (T::BK / 16);
    const int row = r0 + lr;
    const uint32_t slot = (lane % (T::BK / 16)) * 16;
    const uint32_t ch = (swz<T::BK>(row, 0) - row * T::BK) ^ slot;  // the chunk that this slot holds
    if (r0 < T::BM) {
      src[i] = reinterpret_cast<const char*>(xb);
      voff[i] = uint32_t(min(row, c.M - 1 - m0)) * uint32_t(c.D) + ch;
    } else {
      const int br = row - T::BM, b0 = r0 - T::BM;
      if constexpr (GATED) {
        const bool up = (b0 >> 5) & 1;
        src[i] = reinterpret_cast<const char*>(wb) + (up ? size_t(c.N) * c.D : 0);
        voff[i] = uint32_t(min((br >> 6) * 32 + (br & 31), c.N - 1 - n0)) * uint32_t(c.D) + ch;
      } else {
        src[i] = reinterpret_cast<const char*>(wb);
        voff[i] = uint32_t(min(br, c.N - 1 - n0)) * uint32_t(c.D) + ch;
      }
    }
  }
  const int steps_all = c.D / T::BK;
  const int t0 = split * a.steps_per_split;
  const int steps = min(a.steps_per_split, steps_all - t0);
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)smem));
  auto issue = [&](int t) {  // stage t into buffer t % S (past the end: the last stage again, never read)
    const int kt = (t0 + min(t, steps - 1)) * T::BK;
    const uint32_t dst = lds0 + uint32_t(t % T::S) * T::STAGE + uint32_t(wave * T::LOADS) * 1024;
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i)
      dma16(__builtin_amdgcn_readfirstlane(dst + i * 1024), voff[i], src[i] + kt);
  };

  i32x16 acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; ++i)
#pragma unroll
    for (int j = 0; j < T::FN; ++j) acc[i][j] = i32x16{};

  constexpr int SUB = T::BK / 32;
  i32x4 fx[2][T::FM], fw[2][T::FN];
  auto read = [&](int t, int sub, int set) {
    const char* st = smem + (t % T::S) * T::STAGE;
    const uint32_t ch = sub * 2 + (lane >> 5);
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
      fx[set][i] = *reinterpret_cast<const i32x4*>(st + swz<T::BK>((wm * T::FM + i) * 32 + (lane & 31), ch));
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
      fw[set][j] = *reinterpret_cast<const i32x4*>(st + T::BM * T::BK + swz<T::BK>((wn * T::FN + j) * 32 + (lane & 31), ch));
  };
  auto mma = [&](int set) {
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
#pragma unroll
      for (int i = 0; i < T::FM; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[set][j], fx[set][i], acc[i][j], 0, 0, 0);
  };

#pragma unroll
  for (int s = 0; s < T::S; ++s) issue(s);
  stage_wait<(T::S - 1) * T::LOADS>();
  read(0, 0, 0);
  for (int t = 0; t < steps; ++t) {
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
      if (sub + 1 < SUB) {
        read(t, sub + 1, (sub + 1) & 1);
      } else {
        // every wave has read stage t: its buffer takes stage t + S, and stage t + 1 is in LDS
        stage_wait<(T::S - 2) * T::LOADS>();
        issue(t + T::S);
        read(t + 1, 0, 0);
      }
      mma(sub & 1);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads past the end

  // y[m][n]: lane's column of a fragment is m, its rows n come four at a time
  const int mrow = m0 + wm * T::FM * 32 + (lane & 31);
#pragma unroll
  for (int i = 0; i < T::FM; ++i) {
    const int m = mrow + i * 32;
    if (m >= c.M) continue;
    if (a.part) {
      const size_t rows = size_t(c.N) * (GATED ? 2 : 1);
      int* p = a.part + (size_t(split) * c.M + m) * rows;
#pragma unroll
      for (int j = 0; j < T::FN; ++j) {
        const int fj = wn * T::FN + j;
        const int nb = GATED ? n0 + (fj >> 1) * 32 : n0 + fj * 32;
        const size_t base = GATED && (fj & 1) ? size_t(c.N) : 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int n = nb + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
          if (n < c.N) p[base + n] = acc[i][j][e];
        }
      }
      continue;
    }
    const float xs = c.xs[m];
#pragma unroll
    for (int j = 0; j < T::FN; j += GATED ? 2 : 1) {
      const int fj = wn * T::FN + j;
      const int nb = GATED ? n0 + (fj >> 1) * 32 : n0 + fj * 32;
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const int n = nb + 8 * e4 + 4 * (lane >> 5);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int nc = min(n + e, c.N - 1);
          v[e] = float(acc[i][j][e4 * 4 + e]) * xs * c.ws[nc];
          if constexpr (GATED) v[e] = silu_mul(v[e], float(acc[i][j + 1][e4 * 4 + e]) * xs * c.ws[size_t(c.N) + nc]);
        }
        store4(c, m, n, v);
      }
    }
  }
}

template <class T, bool GATED>
hipError_t launch_tile(const W8A8Call& c, int* part, int splits, hipStream_t st) {
  GemmArgs a;
  a.c = c;
  a.part = splits > 1 ? part : nullptr;
  a.tiles_m = (c.M + T::BM - 1) / T::BM;
  const int yn = GATED ? T::BN / 2 : T::BN;
  a.tiles_n = (c.N + yn - 1) / yn;
  a.splits = splits;
  const int steps = c.D / T::BK;
  a.steps_per_split = (steps + splits - 1) / splits;
  const void* fn = reinterpret_cast<const void*>(&w8a8_gemm_kernel<T, GATED>);
  if (hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS)) return e;
  hipLaunchKernelGGL((w8a8_gemm_kernel<T, GATED>), dim3(a.tiles_m * a.tiles_n * splits), dim3(T::NT), T::LDS, st, a);
  return hipGetLastError();
}

using T256 = Tile<256, 256, 2, 2, 64, 4>;

}  // namespace

hipError_t launch_w8a8_gemm(const W8A8Call& c, int* part, hipStream_t st) {
  return c.gated ? launch_tile<T256, true>(c, part, 1, st) : launch_tile<T256, false>(c, part, 1, st);
}

}  // namespace paro
