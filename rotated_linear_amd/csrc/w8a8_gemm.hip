// The 8-bit products for more rows than the other kernels take: tiled matrix-core GEMM.
//
// sum_k xq[m][k] wq[n][k] on v_mfma_i32_16x16x64_i8, 16 rows of w as its A operand and 16 rows of x as
// its B. Tiles of x and w come straight into LDS (no registers, no instruction of the compiler's),
// S stages of 128 channels deep, and pass from one tile of y to the next without a break: a workgroup
// stays on its CU and stores a tile while the next one's stages land. Eight waves take the fragments
// they need from LDS, half a wave's rows of x at a time, read while the other half's products run.
//
// What bounds it, at 256 x 256 tiles (two waves on each SIMD, each 128 x 64 of the tile): the card's
// power limit. The same launches on codes that are all zero run 1.26 times as fast (8192^3: 330 us
// against 417; without the loads to LDS, in a copy for timing, 372). Hence the 16 x 16 x 64 product
// rather than 32 x 32 x 32, which reads and writes an accumulator twice for the same channels (457 ->
// 417 us). The library product of the same codes to plain 32-bit sums takes 461 us there; the gated
// 4096 x 4096 -> 14336 takes 379 us, the library's product of that size 468. Smaller tilings
// are bound by LDS and their loads about equally (1021 x 8960 -> 1537 in 128 x 64 tiles: loads alone
// 22.8 us, reads and products alone 25.8, both 29.2): the estimate below holds each one's time per step.
// The steps, at 8192^3: 256 x 256 tiles in four waves 575 us; in eight, reads between the products 507;
// results through LDS and the scales read from there 481; stages of 128 channels, two of them, instead
// of four of 64 464; loads that pass the ends of tiles 457; the 16 x 16 x 64 product 417.
#include <stddef.h>

#include <algorithm>
#include <cmath>

#include "w8a8_dma.h"

namespace paro {
namespace {

constexpr int kCUs = 256;
constexpr int kXcds = 8;

// All but the N youngest of this wave's memory operations are done and so are its LDS reads; then
// the workgroup's waves meet.
template <int N>
__device__ inline void stage_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// The lane index, made opaque where it is used: addresses formed from it once per tile are not
// hoisted out of the tile loop and kept live (or spilled) across the products.
__device__ inline int fresh_lane() {
  int t = int(threadIdx.x);
  asm volatile("" : "+v"(t));
  return t & 63;
}

struct GemmArgs {
  W8A8Call c;
  int* part;  // split partial sums [S][M][rows of w], or nullptr
  int tiles_m, tiles_n, splits, steps_per_split;
};

template <int BM_, int BN_, int WM_, int WN_, int BK_, int S_, int PR_ = 32>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, S = S_;
  static constexpr int NW = WM * WN, NT = NW * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // 16 x 16 fragments of a wave
  static constexpr int ROWS = BM + BN;
  static constexpr int STAGE = ROWS * BK;
  static constexpr int RPI = 1024 / BK;           // tile rows of one wave-wide load
  static constexpr int LOADS = ROWS / RPI / NW;   // a wave's loads per stage
  static_assert(BK == 128 && ROWS % (RPI * NW) == 0 && BM % RPI == 0, "loads divide over the waves");
  static_assert(FN % 2 == 0 && (FM == 1 || FM % 2 == 0), "16 gate and 16 up rows in turn; x fragments in halves");
  // Results leave through LDS in pieces of PR rows, up to 64 bytes of a row at a time, rows 80 bytes
  // apart.
  static constexpr int PR = FM == 1 ? 16 : PR_;
  static constexpr int EP = 80;
  static constexpr int OUT = STAGE * S;           // LDS: the stages, each wave's results, the scales
  static constexpr int SCALES = OUT + NW * PR * EP;
  static constexpr int XS = BM < 64 ? 64 : BM;    // scales of x rows (64 at least: they come 64 a load)
  static constexpr int LDS = SCALES + (XS + BN) * 4;
  static_assert(XS % 64 == 0 && BN % 64 == 0 && LDS <= 160 * 1024, "scales 64 a load; one CU's LDS");
  // With an epilogue, each wave's bias in float32 behind the scales.
  static constexpr int BIAS = LDS, WCOLS = FN * 16;
  static constexpr int LDS_EPILOGUE = BIAS + NW * WCOLS * 4;
  static_assert(WCOLS <= 64 && 160 * 1024 / LDS_EPILOGUE == 160 * 1024 / LDS, "a lane to each; no workgroup less on a CU");
};

// Where a tile lies.
struct Place {
  int m0, n0;  // first row and column of y
  int split, t0, steps;
  int start;  // the walk over the steps begins here and wraps
};

// Tile number `tile` (of tiles_m * tiles_n * splits): splits innermost, then groups of 4 tile rows
// walked column by column, so that tiles worked on at the same time share rows of x and of w.
template <class T, Output KIND>
__device__ inline Place place(const GemmArgs& a, int tile) {
  constexpr bool GATED = KIND == kGated;
  Place p;
  p.split = tile % a.splits;
  tile /= a.splits;
  constexpr int GM = 4;
  const int group = tile / (GM * a.tiles_n);
  const int gsz = min(GM, a.tiles_m - group * GM);
  const int in = tile - group * GM * a.tiles_n;
  p.m0 = (group * GM + in % gsz) * T::BM;
  p.n0 = (in / gsz) * (GATED ? T::BN / 2 : T::BN);
  p.t0 = p.split * a.steps_per_split;
  p.steps = min(a.steps_per_split, a.c.D / T::BK - p.t0);
  // With one row of tiles no two tiles share rows of w, and each starts its walk one step after its
  // neighbour: rows a multiple of 2 KB apart lie in the same L2 channel (M = 40, gated 4096 -> 14336:
  // 30.7 -> 26.4 us). Tiles that share rows of w keep together (starting them apart: up to 6 % slower).
  p.start = a.tiles_m == 1 ? in / gsz % p.steps : 0;
  return p;
}

// Four values in type DT at an address in LDS.
template <int DT>
__device__ inline void put4(char* at, const float (&v)[4]) {
  if constexpr (DT == PARO_F32) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __builtin_bit_cast(uint32_t, v[e]);
    *reinterpret_cast<u32x4*>(at) = w;
  } else {
    using u32x2 = uint32_t __attribute__((ext_vector_type(2)));
    *reinterpret_cast<u32x2*>(at) =
        u32x2{to_bits16<DT>(v[0]) | (to_bits16<DT>(v[1]) << 16), to_bits16<DT>(v[2]) | (to_bits16<DT>(v[3]) << 16)};
  }
}

// Four neighbouring elements of type DT as they are stored.
template <int DT>
struct alignas(DT == PARO_F32 ? 16 : 8) Four {
  uint32_t w[DT == PARO_F32 ? 4 : 2];
};
template <int DT>
__device__ inline float element(const Four<DT>& f, int e) {
  if constexpr (DT == PARO_F32) return __builtin_bit_cast(float, f.w[e]);
  if constexpr (DT != PARO_F32) return from_bits16<DT>(e % 2 ? f.w[e / 2] >> 16 : f.w[e / 2] & 0xFFFFu);
}
// Elements n .. n + 3 of a row that starts at `row` and has N of them (0 past its end). Rows of a multiple of
// four elements lie at multiples of their size.
template <int DT>
__device__ inline Four<DT> load4(const void* p, size_t row, int n, int N) {
  Four<DT> f{};
  if (N % 4 == 0) {
    if (n < N) f = *reinterpret_cast<const Four<DT>*>(static_cast<const char*>(p) + (row + n) * (DT == PARO_F32 ? 4 : 2));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < N) {
        if constexpr (DT == PARO_F32)
          f.w[e] = static_cast<const uint32_t*>(p)[row + n + e];
        else
          f.w[e / 2] |= uint32_t(static_cast<const uint16_t*>(p)[row + n + e]) << (e % 2 * 16);
      }
  }
  return f;
}

// Store one piece that the wave has put into buf: PR rows of PB bytes, 16 bytes a lane. dst: the
// piece's first element; rows ld bytes apart; `rows` rows and `cols` elements of EB bytes exist.
template <int EB, int EP, int PB, int PR>
__device__ inline void store_piece(const char* buf, char* dst, size_t ld, int rows, int cols, bool whole, int lane) {
  if (whole) {
    constexpr int L = PB / 16;  // lanes of a row
#pragma unroll
    for (int r0 = 0; r0 < PR; r0 += 64 / L) {
      const int r = r0 + lane / L, b = lane % L;
      if (r < min(rows, PR) && b * (16 / EB) < cols) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(buf + r * EP + b * 16);
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(dst + r * ld + b * 16));
      }
    }
  } else {
    constexpr int E = PB / EB;  // elements of a piece's row
    const int b = lane % E;
    for (int r = lane / E; r < PR; r += 64 / E)
      if (r < rows && b < cols) {
        if constexpr (EB == 4)
          *reinterpret_cast<uint32_t*>(dst + r * ld + b * 4) = *reinterpret_cast<const uint32_t*>(buf + r * EP + b * 4);
        else
          *reinterpret_cast<uint16_t*>(dst + r * ld + b * 2) = *reinterpret_cast<const uint16_t*>(buf + r * EP + b * 2);
      }
  }
}

// A wave's results: scaled (and gated) rows of y in type DT, or (PART) the int32 sums themselves.
// A lane's column of a fragment is a row of y, its rows are columns of y, four at a time.
template <class T, Output KIND, int DT, bool PART>
__device__ inline void store_tile(const GemmArgs& a, const Place& p, const i32x4 (&acc)[T::FM][T::FN], char* smem,
                                  int wave) {
  const W8A8Call& c = a.c;
  const int lane = fresh_lane();
  constexpr bool GATED = KIND == kGated;
  constexpr int EB = DT == PARO_F32 ? 4 : 2;
  constexpr bool G = GATED && !PART;
  constexpr int YF = G ? T::FN / 2 : T::FN;    // the wave's column fragments of the output,
  constexpr int CF = YF < 4 / EB ? YF : 4 / EB;  // and a piece's
  constexpr int RF = T::PR / 16;               // row fragments of a piece
  const int wm = wave / T::WN, wn = wave % T::WN;
  char* const buf = smem + T::OUT + wave * T::PR * T::EP;
  const float* const sc = reinterpret_cast<const float*>(smem + T::SCALES);
  const size_t ldc = PART ? size_t(c.N) * (GATED ? 2 : 1) : size_t(c.N);  // columns of the output
  char* const out = PART ? reinterpret_cast<char*>(a.part) + size_t(p.split) * c.M * ldc * 4 : static_cast<char*>(c.y);
  const bool whole = c.N % (16 / EB) == 0;  // pieces start at multiples of 16 bytes and end with a row
#pragma unroll
  for (int i = 0; i < T::FM; i += RF) {
    const int mf = (wm * T::FM + i) * 16;
    float xs[RF];
#pragma unroll
    for (int u = 0; u < RF; ++u) xs[u] = sc[mf + u * 16 + (lane & 15)];
#pragma unroll
    for (int y = 0; y < YF; y += CF) {
#pragma unroll
      for (int k = 0; k < CF; ++k) {
        const int j = G ? 2 * (y + k) : y + k;  // the fragment of w (gate fragments and their up fragments in turn)
        const float* const wsc = sc + T::XS + (wn * T::FN + j) * 16 + 4 * (lane >> 4);
#pragma unroll
        for (int u = 0; u < RF; ++u) {
          char* const at = buf + (u * 16 + (lane & 15)) * T::EP + (16 * k + 4 * (lane >> 4)) * EB;
          if constexpr (PART) {
            *reinterpret_cast<i32x4*>(at) = acc[i + u][j];
          } else {
            float v[4];
            const float4 w4 = *reinterpret_cast<const float4*>(wsc);
            const float w0[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scaled(acc[i + u][j][e], xs[u], w0[e]);
            if constexpr (G) {
              const float4 u4 = *reinterpret_cast<const float4*>(wsc + 16);
              const float u0[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = silu_mul<DT>(v[e], scaled(acc[i + u][j + 1][e], xs[u], u0[e]));
            }
            put4<DT>(at, v);
          }
        }
      }
      // one wave's LDS accesses are carried out in order; the compiler keeps them in order too
      asm volatile("" ::: "memory");
      // the piece's first column: of y (n), and in the output (the sums of a gated pair keep w's rows)
      const int r = wn * T::FN + y;  // fragment of w in the tile (not gated output)
      const int n = p.n0 + (G ? wn * YF + y : GATED ? r >> 1 : r) * 16;
      const size_t col = n + (PART && GATED && (r & 1) ? size_t(c.N) : 0);
      store_piece<EB, T::EP, CF * 16 * EB, T::PR>(buf, out + (size_t(p.m0 + mf) * ldc + col) * EB, ldc * EB,
                                                  c.M - p.m0 - mf, c.N - n, whole, lane);
      asm volatile("" ::: "memory");
    }
  }
}

// The same for a call with an epilogue. The residual is read as the lanes hold their sums, four columns of a row each, a
// piece ahead of the one that is worked on. With one tile for each CU this code runs once, from a cold instruction cache,
// so that its length counts (4096 x 14336 -> 4096 with a residual: 234 us with the pieces unrolled, 223 with the
// activations in the way, 200 to 207 so, the plain product 197; 64 x 4096 -> 14336 with GELU 13.4 us, plain 12.6; 1021 x 1536 ->
// 1537 with a float32 residual 13.2, plain 10.2): one copy of it serves all pieces, whose sums are first moved to registers of their own, and
// ACT, with an activation, is another. bias: of the wave's column `lane`.
template <class T, int DT, bool ACT>
__device__ inline void store_tile_epilogue(const W8A8Call& c, const Place& p, const i32x4 (&acc)[T::FM][T::FN], char* smem, int wave, float bias) {
  const int lane = fresh_lane();
  constexpr int EB = DT == PARO_F32 ? 4 : 2;
  constexpr int CF = T::FN < 4 / EB ? T::FN : 4 / EB;  // column and row fragments of a piece
  constexpr int RF = T::PR / 16;
  constexpr int ROW = T::FN / CF, PIECES = T::FM / RF * ROW;
  const int wm = wave / T::WN, wn = wave % T::WN;
  char* const buf = smem + T::OUT + wave * T::PR * T::EP;
  const float* const sc = reinterpret_cast<const float*>(smem + T::SCALES);
  float* const bs = reinterpret_cast<float*>(smem + T::BIAS) + wave * T::WCOLS;
  const bool whole = c.N % (16 / EB) == 0;
  const int mw = wm * T::FM * 16, nw = wn * T::WCOLS;  // the wave's first row and column in the tile
  Four<DT> res[RF][CF], next[RF][CF];
  // (only elements of y: in place of the residual, the others are another workgroup's to write)
  auto fetch = [&](int piece) {
#pragma unroll
    for (int u = 0; u < RF; ++u)
#pragma unroll
      for (int k = 0; k < CF; ++k) {
        const int m = p.m0 + mw + (piece / ROW * RF + u) * 16 + (lane & 15);
        const int n = p.n0 + nw + (piece % ROW * CF + k) * 16 + 4 * (lane >> 4);
        next[u][k] = m < c.M ? load4<DT>(c.residual, size_t(m) * c.N, n, c.N) : Four<DT>{};
      }
  };
  if (c.residual) fetch(0);
  if (lane < T::WCOLS) bs[lane] = bias;  // (0 without one)
  // one wave's LDS accesses are carried out in order; the compiler keeps them in order too
  asm volatile("" ::: "memory");
#pragma unroll 1
  for (int piece = 0; piece < PIECES; ++piece) {
    i32x4 sum[RF][CF];
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
      if (q == piece) {  // uniform
#pragma unroll
        for (int u = 0; u < RF; ++u)
#pragma unroll
          for (int k = 0; k < CF; ++k) sum[u][k] = acc[q / ROW * RF + u][q % ROW * CF + k];
      }
    if (c.residual) {
#pragma unroll
      for (int u = 0; u < RF; ++u)
#pragma unroll
        for (int k = 0; k < CF; ++k) res[u][k] = next[u][k];
      if (piece + 1 < PIECES) fetch(piece + 1);
    }
    const int mf = mw + piece / ROW * RF * 16, nf = piece % ROW * CF * 16;
    float v[RF * CF * 4];
#pragma unroll
    for (int k = 0; k < CF; ++k) {
      const int at = nf + k * 16 + 4 * (lane >> 4);
      const float4 w4 = *reinterpret_cast<const float4*>(sc + T::XS + nw + at), b4 = *reinterpret_cast<const float4*>(bs + at);
      const float ws[4] = {w4.x, w4.y, w4.z, w4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
      for (int u = 0; u < RF; ++u) {
        const float xs = sc[mf + u * 16 + (lane & 15)];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[(u * CF + k) * 4 + e] = plus(scaled(sum[u][k][e], xs, ws[e]), b[e]);
      }
    }
    if constexpr (ACT) activate<DT>(v, c.act);
    if (c.residual) {
#pragma unroll
      for (int u = 0; u < RF; ++u)
#pragma unroll
        for (int k = 0; k < CF; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[(u * CF + k) * 4 + e] = plus(v[(u * CF + k) * 4 + e], element<DT>(res[u][k], e));
    }
#pragma unroll
    for (int u = 0; u < RF; ++u)
#pragma unroll
      for (int k = 0; k < CF; ++k) {
        const float* const o = v + (u * CF + k) * 4;
        const float o4[4] = {o[0], o[1], o[2], o[3]};
        put4<DT>(buf + (u * 16 + (lane & 15)) * T::EP + (16 * k + 4 * (lane >> 4)) * EB, o4);
      }
    asm volatile("" ::: "memory");
    store_piece<EB, T::EP, CF * 16 * EB, T::PR>(buf, static_cast<char*>(c.y) + (size_t(p.m0 + mf) * c.N + p.n0 + nw + nf) * EB,
                                                size_t(c.N) * EB, c.M - p.m0 - mf, c.N - p.n0 - nw - nf, whole, lane);
    asm volatile("" ::: "memory");
  }
}

// The kernel's arguments, read again here: kept from the start, those that only the epilogue wants would take scalar
// registers from the main loop, which then keeps its own in lanes of vector registers.
__device__ inline W8A8Call call_again() {
  uintptr_t p = uintptr_t(__builtin_amdgcn_kernarg_segment_ptr());
  asm volatile("" : "+s"(p));
  const auto k = (const __attribute__((address_space(4))) W8A8Call*)p;
  W8A8Call c{};
  c.M = k->M;
  c.N = k->N;
  c.y = k->y;
  c.act = k->act;
  c.residual = k->residual;
  return c;
}
static_assert(offsetof(GemmArgs, c) == 0, "the call lies where the arguments begin");

template <class T, Output KIND, int DT>
__device__ inline void store_outputs(const GemmArgs& a, const Place& p, const i32x4 (&acc)[T::FM][T::FN], char* smem, int wave, float bias) {
  if constexpr (KIND == kEpilogue) {
    const W8A8Call c = call_again();
    if (c.act == PARO_ACT_NONE)
      store_tile_epilogue<T, DT, false>(c, p, acc, smem, wave, bias);
    else
      store_tile_epilogue<T, DT, true>(c, p, acc, smem, wave, bias);
  } else
    store_tile<T, KIND, DT, false>(a, p, acc, smem, wave);
}

template <class T, Output KIND>
__global__ __launch_bounds__(T::NT) void w8a8_gemm_kernel(const GemmArgs a) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  constexpr bool GATED = KIND == kGated;
  const W8A8Call& c = a.c;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;

  // Workgroups go round the XCDs; each XCD takes a contiguous range of tiles, its workgroups one
  // tile after another.
  const int total = a.tiles_m * a.tiles_n * a.splits;
  const int per = total / kXcds, rem = total % kXcds;
  const int xcd = blockIdx.x % kXcds;
  const int stride = (gridDim.x - xcd + kXcds - 1) / kXcds;  // workgroups on this XCD
  const int first = xcd * per + min(xcd, rem), end = first + per + (xcd < rem ? 1 : 0);
  int tile = first + blockIdx.x / kXcds;
  if (tile >= end) return;

  // The loads run S stages ahead of the products and pass from one tile to the next without a
  // break: `ahead` is the tile they are in, step `at` of it.
  int ahead = tile, at = 0;
  Place q = place<T, KIND>(a, ahead);
  uint32_t voff[T::LOADS];
  const char* src[T::LOADS];
  auto aim = [&]() {
    const int lane = fresh_lane();
    // this lane's source offsets in tile q; rows past the end are the last row again
    const char* const xb = reinterpret_cast<const char*>(c.x) + size_t(q.m0) * c.D + size_t(q.t0) * T::BK;
    const char* const wb = reinterpret_cast<const char*>(c.w) + size_t(q.n0) * c.D + size_t(q.t0) * T::BK;
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) {
      const int r0 = (wave * T::LOADS + i) * T::RPI;  // first tile row of the load
      const int row = r0 + lane / (T::BK / 16);
      const uint32_t slot = (lane % (T::BK / 16)) * 16;
      const uint32_t ch = (swz(row, 0) - row * T::BK) ^ slot;  // the chunk that this slot holds
      if (r0 < T::BM) {
        src[i] = xb;
        voff[i] = uint32_t(min(row, c.M - 1 - q.m0)) * uint32_t(c.D) + ch;
      } else {
        const int b = row - T::BM;
        const bool up = GATED && (((r0 - T::BM) >> 4) & 1);
        src[i] = wb + (up ? size_t(c.N) * c.D : 0);
        voff[i] = uint32_t(min(GATED ? (b >> 5) * 16 + (b & 15) : b, c.N - 1 - q.n0)) * uint32_t(c.D) + ch;
      }
    }
  };
  aim();
  const uint32_t lds0 = lds_address(smem);
  const uint32_t ldsw = __builtin_amdgcn_readfirstlane(lds0 + uint32_t(wave * T::LOADS) * 1024);
  auto issue = [&](uint32_t buf) {  // the next stage into buffer `buf`; after the last tile its last stage again
    if (at == q.steps) {
      if (ahead + stride < end) {
        ahead += stride;
        at = 0;
        q = place<T, KIND>(a, ahead);
        aim();
      } else {
        at = q.steps - 1;
      }
    }
    const int step = at + q.start < q.steps ? at + q.start : at + q.start - q.steps;
#pragma unroll
    for (int i = 0; i < T::LOADS; ++i) dma16(ldsw + buf * T::STAGE + i * 1024, voff[i], src[i] + size_t(step) * T::BK);
    ++at;
  };
  // The scales of a tile (x rows, then w rows) into LDS: the waves take 64 each.
  auto load_scales = [&](const Place& p) {
    const int lane = fresh_lane();
#pragma unroll
    for (int r0 = 0; r0 < T::XS + T::BN; r0 += 64 * T::NW) {
      const int rw = r0 + wave * 64;
      if (rw >= T::XS + T::BN) break;
      const uint32_t dst = lds0 + T::SCALES + rw * 4;
      if (rw < T::XS) {
        dma4(dst, uint32_t(min(rw + lane, c.M - 1 - p.m0)) * 4, c.xs + p.m0);
      } else {
        const int b = rw - T::XS + lane;
        const uint32_t o = GATED ? min((b >> 5) * 16 + (b & 15), c.N - 1 - p.n0) + ((b >> 4) & 1 ? uint32_t(c.N) : 0)
                                 : min(b, c.N - 1 - p.n0);
        dma4(dst, o * 4, c.ws + p.n0);
      }
    }
  };

  constexpr int SUB = T::BK / 64;
  // Half a wave's rows of x at a time (all of a single fragment): while one part's products run, the
  // next part's fragments (and, before a new 64-channel step, its fragments of w) are read.
  constexpr int NH = T::FM > 1 ? 2 : 1, HM = T::FM / NH;
  i32x4 fx[2][HM], fw[2][T::FN];
  auto read_x = [&](uint32_t buf, int h) {  // part h of a stage
    const char* const st = smem + buf * T::STAGE;
#pragma unroll
    for (int i = 0; i < HM; ++i)
      fx[h & 1][i] = *reinterpret_cast<const i32x4*>(
          st + swz((wm * T::FM + h % NH * HM + i) * 16 + (lane & 15), h / NH * 4 + (lane >> 4)));
  };
  auto read_w = [&](uint32_t buf, int sub) {
    const char* const st = smem + buf * T::STAGE + T::BM * T::BK;
#pragma unroll
    for (int j = 0; j < T::FN; ++j)
      fw[sub & 1][j] = *reinterpret_cast<const i32x4*>(st + swz((wn * T::FN + j) * 16 + (lane & 15), sub * 4 + (lane >> 4)));
  };

#pragma unroll
  for (int s = 0; s < T::S; ++s) issue(s);
  stage_wait<(T::S - 1) * T::LOADS>();
  read_w(0, 0);
  read_x(0, 0);
  uint32_t buf = 0;
  for (; tile < end; tile += stride) {
    const Place p = place<T, KIND>(a, tile);
    i32x4 acc[T::FM][T::FN];
#pragma unroll
    for (int i = 0; i < T::FM; ++i)
#pragma unroll
      for (int j = 0; j < T::FN; ++j) acc[i][j] = i32x4{};
    float bias = 0;  // asked for long before it is used
    if constexpr (KIND == kEpilogue) {
      const int col = wn * T::WCOLS + fresh_lane();
      if (c.bias && !a.part && col < (wn + 1) * T::WCOLS && p.n0 + col < c.N) bias = load_element(c.bias, p.n0 + col, c.ydtype);
    }
    for (int t = 0; t < p.steps; ++t) {
      const uint32_t nbuf = buf + 1 == T::S ? 0 : buf + 1;
#pragma unroll
      for (int h = 0; h < NH * SUB; ++h) {
        const int sub = h / NH;
        if (h + 1 < NH * SUB) {
          if ((h + 1) % NH == 0) read_w(buf, sub + 1);
          read_x(buf, h + 1);
        } else {
          // every wave has read this stage: its buffer takes the stage S further on, and the next
          // stage is in LDS
          stage_wait<(T::S - 2) * T::LOADS>();
          issue(buf);
          if (t == 0) load_scales(p);  // every wave has stored the last tile
          read_w(nbuf, 0);
          read_x(nbuf, 0);
        }
#pragma unroll
        for (int j = 0; j < T::FN; ++j)
#pragma unroll
          for (int i = 0; i < HM; ++i)
            acc[h % NH * HM + i][j] =
                __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[sub & 1][j], fx[h & 1][i], acc[h % NH * HM + i][j], 0, 0, 0);
        // a fragment read, then its share of the products, in turn
        constexpr int kShare = HM * T::FN / (HM + T::FN);
#pragma unroll
        for (int r = 0; r < T::FN + HM; ++r) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, kShare > 0 ? kShare : 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      asm volatile("" ::: "memory");  // the next stage's first reads stay in this iteration
      buf = nbuf;
    }
    // with S steps or more the scales' loads were waited for at a later stage's barrier
    if (p.steps < T::S) stage_wait<0>();
    if (a.part)
      store_tile<T, KIND, PARO_F32, true>(a, p, acc, smem, wave);
    else if (c.ydtype == PARO_F32)
      store_outputs<T, KIND, PARO_F32>(a, p, acc, smem, wave, bias);
    else if (c.ydtype == PARO_F16)
      store_outputs<T, KIND, PARO_F16>(a, p, acc, smem, wave, bias);
    else
      store_outputs<T, KIND, PARO_BF16>(a, p, acc, smem, wave, bias);
    if constexpr (KIND == kEpilogue) {  // read again: not kept in registers across the epilogue, which wants them
      read_w(buf, 0);
      read_x(buf, 0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads past the last stage land before the LDS is given up
}

// V elements from element i on (V = 4: i a multiple of 4) in float32.
template <int DT, int V>
__device__ inline void load_elements(const void* p, size_t i, float (&v)[V]) {
  if constexpr (V == 4) {
    const Four<DT> f = *reinterpret_cast<const Four<DT>*>(static_cast<const char*>(p) + i * (DT == PARO_F32 ? 4 : 2));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = element<DT>(f, e);
  } else {
    v[0] = load_element(p, i, DT);
  }
}

// y from the S partial sums of a split reduction: a thread takes V columns of a row (their sums of
// every split in flight together), the integer sums are exact in any order.
template <int V, Output KIND, int DT>
__global__ __launch_bounds__(256) void reduce_kernel(const W8A8Call c, const int* part, int splits) {
  using IV = int __attribute__((ext_vector_type(V)));
  constexpr bool GATED = KIND == kGated;
  const size_t rows = size_t(c.N) * (GATED ? 2 : 1), plane = size_t(c.M) * rows;
  const size_t per_row = c.N / V, total = per_row * c.M;
  for (size_t t = size_t(blockIdx.x) * 256 + threadIdx.x; t < total; t += size_t(gridDim.x) * 256) {
    const size_t m = t / per_row;
    const int n = int(t - m * per_row) * V;
    const int* const p = part + m * rows + n;
    IV g = IV(0), u = IV(0);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      g += *reinterpret_cast<const IV*>(p + s * plane);
      if constexpr (GATED) u += *reinterpret_cast<const IV*>(p + s * plane + c.N);
    }
    const float xs = c.xs[m];
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[e] = scaled(g[e], xs, c.ws[n + e]);
      if constexpr (GATED) v[e] = silu_mul<DT>(v[e], scaled(u[e], xs, c.ws[size_t(c.N) + n + e]));
    }
    if constexpr (KIND == kEpilogue) {
      float w[V] = {};
      if (c.bias) load_elements<DT, V>(c.bias, n, w);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = plus(v[e], w[e]);
      activate<DT>(v, c.act);
      if (c.residual) {
        load_elements<DT, V>(c.residual, m * c.N + n, w);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = plus(v[e], w[e]);
      }
    }
    if constexpr (V == 4) {
      put4<DT>(static_cast<char*>(c.y) + (m * c.N + n) * (DT == PARO_F32 ? 4 : 2), v);
    } else if constexpr (DT == PARO_F32) {
      static_cast<float*>(c.y)[m * c.N + n] = v[0];
    } else {
      static_cast<uint16_t*>(c.y)[m * c.N + n] = uint16_t(to_bits16<DT>(v[0]));
    }
  }
}

template <Output KIND>
hipError_t launch_reduce(const W8A8Call& c, const int* part, int splits, hipStream_t st) {
  const bool four = c.N % 4 == 0;
  const size_t total = size_t(c.M) * (c.N / (four ? 4 : 1));
  const dim3 grid(unsigned(std::min<size_t>((total + 255) / 256, 8192)));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, c, part, splits);
    return hipGetLastError();
  };
  if (c.ydtype == PARO_F32) return go(four ? reduce_kernel<4, KIND, PARO_F32> : reduce_kernel<1, KIND, PARO_F32>);
  if (c.ydtype == PARO_F16) return go(four ? reduce_kernel<4, KIND, PARO_F16> : reduce_kernel<1, KIND, PARO_F16>);
  return go(four ? reduce_kernel<4, KIND, PARO_BF16> : reduce_kernel<1, KIND, PARO_BF16>);
}

template <class T>
constexpr TilingQ8 tiling() {
  return TilingQ8{T::BM, T::BN, kCUs * int(160 * 1024 / T::LDS)};
}

template <class T, Output KIND>
hipError_t launch_tile(const W8A8Call& c, int* part, int splits, hipStream_t st) {
  GemmArgs a;
  a.c = c;
  a.tiles_m = (c.M + T::BM - 1) / T::BM;
  const int yn = KIND == kGated ? T::BN / 2 : T::BN;
  a.tiles_n = (c.N + yn - 1) / yn;
  const int steps = c.D / T::BK;
  a.steps_per_split = (steps + splits - 1) / splits;
  a.splits = (steps + a.steps_per_split - 1) / a.steps_per_split;  // every split has steps
  a.part = a.splits > 1 ? part : nullptr;
  const void* fn = reinterpret_cast<const void*>(&w8a8_gemm_kernel<T, KIND>);
  constexpr int lds = KIND == kEpilogue ? T::LDS_EPILOGUE : T::LDS;
  if (hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds)) return e;
  const long total = long(a.tiles_m) * a.tiles_n * a.splits;
  hipLaunchKernelGGL((w8a8_gemm_kernel<T, KIND>), dim3(unsigned(std::min<long>(total, tiling<T>().workgroups))), dim3(T::NT), lds, st, a);
  if (hipError_t e = hipGetLastError()) return e;
  return a.part ? launch_reduce<KIND>(c, part, a.splits, st) : hipSuccess;
}

// The tilings: waves side by side in rows and columns, stages in LDS. Eight waves where the tile has
// room for them: a CU's matrix cores then have a second wave each while the first waits (a 128 x 128
// tile's step of 128 channels takes 0.43 us with eight, 0.59 with four; a 128 x 64 tile's 0.29 and
// 0.44).
using T256 = Tile<256, 256, 2, 4, 128, 2>;     // one workgroup on a CU (by LDS)
using T256x128 = Tile<256, 128, 4, 2, 128, 3, 16>; // one; a third stage: 1427 x 9216 -> 5095 99 -> 82 us
using T128 = Tile<128, 128, 2, 4, 128, 4>;     // one
using T128Two = Tile<128, 128, 2, 4, 128, 2, 16>;  // two: for a little more than one tile per CU
using T128x64 = Tile<128, 64, 4, 2, 128, 4>;   // one
using T64 = Tile<64, 64, 4, 2, 128, 4>;        // two
using T32 = Tile<32, 64, 2, 2, 128, 4>;        // two

// Estimated time of a call in microseconds, from a fit to 2457 measured combinations of shape, tiling
// and split (MI355X, cold weights, 58 shapes: M = 18..4096, D = 128..16256, N = 64..23000; 11 % rms
// off): a launch; the units that a CU works through, per 128 channels of a unit (alone on a CU, and
// with `cap` units on it or on every CU) plus its start and end; the weights' way from HBM; these two
// joined as the cube root of the sum of their cubes, since they overlap but not wholly; and for a
// split a launch and the partial sums out and back. The choice by it was 1.5 % slower than the fastest
// measured one on average, 19 % at worst. The 256 x 128 tile had two stages when the fit was made; it has
// three now, so its times here are too high, and some shapes that would gain up to 5 % by it go to others.
// Lowering its row alone moved shapes to it that others do better (35 shapes, no faster as a whole): the
// whole table wants fitting again.
struct TileCost {
  int bm, bn, cap;
  double alone, full, end;
};
constexpr TileCost kTiles[] = {{256, 256, 1, 1.24, 1.56, 9.0}, {256, 128, 1, 0.836, 0.967, 5.44}, {128, 128, 1, 0.425, 0.526, 3.24},
                               {128, 128, 2, 0.651, 1.045, 3.05}, {128, 64, 1, 0.286, 0.366, 1.85}, {64, 64, 2, 0.198, 0.482, 1.46},
                               {32, 64, 2, 0.157, 0.316, 1.07}};
constexpr double kLaunchUs = 3.18, kSplitUs = 2.77, kHbmBytesPerUs = 4.57e6, kPartBytesPerUs = 5.37e6;

constexpr TilingQ8 kTilings[kTilingsQ8] = {tiling<T256>(),    tiling<T256x128>(), tiling<T128>(), tiling<T128Two>(),
                                           tiling<T128x64>(), tiling<T64>(),      tiling<T32>()};
constexpr bool costs_name_the_tilings() {
  for (int t = 0; t < kTilingsQ8; ++t)
    if (kTiles[t].bm != kTilings[t].bm || kTiles[t].bn != kTilings[t].bn || kTiles[t].cap * kCUs != kTilings[t].workgroups) return false;
  return sizeof(kTiles) / sizeof(kTiles[0]) == kTilingsQ8;
}
static_assert(costs_name_the_tilings(), "the cost table's rows are the tilings");

// Partial sums of a split reduction at most (larger ones cost more than a split gives).
constexpr double kMaxPartBytes = double(size_t(128) << 20);

}  // namespace

TilingQ8 tiling_w8a8(int tile) { return kTilings[tile]; }

size_t part_bytes_w8a8(int M, int N, bool gated, int splits) {
  return splits > 1 ? align256(size_t(splits) * M * N * (gated ? 2 : 1) * 4) : 0;
}

GemmPlanQ8 plan_gemm_w8a8(int M, int D, int N, bool gated) {
  const double rows = double(N) * (gated ? 2 : 1);
  const int steps = D / 128;
  GemmPlanQ8 best{1, 1, 0, 1e30};
  for (int t = 0; t < kTilingsQ8; ++t) {
    const TileCost& k = kTiles[t];
    const double tiles = std::ceil(double(M) / k.bm) * std::ceil(rows / k.bn);
    for (int s : {1, 2, 3, 4, 6, 8, 12, 16}) {
      const double part = double(s) * M * rows * 4;
      if (s > 1 && (s > steps || part > kMaxPartBytes)) break;
      const int per = (steps + s - 1) / s;
      const double on_cu = std::ceil(tiles * ((steps + per - 1) / per) / kCUs);  // units of the busiest CU
      const double rounds = std::floor(on_cu / k.cap), rest = on_cu - rounds * k.cap;
      double us = rounds * (per * k.full + k.end);
      if (k.cap == 1 && on_cu == 1) us = per * k.alone + k.end;
      if (rest > 0) us += per * (k.alone + (k.full - k.alone) * (rest - 1) / (k.cap - 1)) + k.end;
      const double hbm = rows * D / kHbmBytesPerUs;
      us = kLaunchUs + std::cbrt(us * us * us + hbm * hbm * hbm);
      if (s > 1) us += kSplitUs + 2 * part / kPartBytesPerUs;
      if (us < best.us) best = GemmPlanQ8{t, s, part_bytes_w8a8(M, N, gated, s), us};
    }
  }
  return best;
}

namespace {

template <Output KIND>
hipError_t launch_plan(const W8A8Call& c, const GemmPlanQ8& p, int* part, hipStream_t st) {
  switch (p.tile) {
    case 0: return launch_tile<T256, KIND>(c, part, p.splits, st);
    case 1: return launch_tile<T256x128, KIND>(c, part, p.splits, st);
    case 2: return launch_tile<T128, KIND>(c, part, p.splits, st);
    case 3: return launch_tile<T128Two, KIND>(c, part, p.splits, st);
    case 4: return launch_tile<T128x64, KIND>(c, part, p.splits, st);
    case 5: return launch_tile<T64, KIND>(c, part, p.splits, st);
    default: return launch_tile<T32, KIND>(c, part, p.splits, st);
  }
}

}  // namespace

hipError_t launch_w8a8_gemm(const W8A8Call& c, const GemmPlanQ8& p, int* part, hipStream_t st) {
  return c.epilogue ? launch_plan<kEpilogue>(c, p, part, st)
         : c.gated  ? launch_plan<kGated>(c, p, part, st)
                    : launch_plan<kPlain>(c, p, part, st);
}

}  // namespace paro
