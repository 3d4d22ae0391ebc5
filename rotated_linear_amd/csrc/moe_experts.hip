// The experts' products of a mixture-of-experts layer for a few tokens, on INT4 weights: gate and up with their
// activation, then down with the sum over a token's experts. Bound by the weights' way from HBM where the experts are
// large, and by launches where they are not. Measured (in a trace; a copy runs at 4.95 TB/s, reading alone at 5.95), gate and
// up, then down: 4 tokens, 2 of 8 experts, 5 of them reached, 4096 -> 14336 53 us (5.9 TB/s) and 38 us (4.1); 64 tokens, 8
// of 64, 4096 -> 1408 74 (5.3) and 57 (3.4); 32 tokens, 4 of 16, 4096 -> 2048 30 (4.6) and 21.5 (3.2); one token, 8 of 64,
// 2048 -> 1024 7.9 and 7.7.
#include <algorithm>
#include <cmath>

#include "moe_internal.h"
#include "w4_device.h"

namespace paro {
namespace {

constexpr int kCUs = 256;

// 128 channels (a group) of 16 weight rows are a contiguous kilobyte: a lane's 16 bytes are row lane & 15, channels
// 32 (lane >> 4) on. The same channels of 16 rows of x, 8-channel words in the order dequant_word gives them:
struct Rows {
  h8 v[4];
};

// sum[row of x][row of w] += the group's products. sz: the scale and, in the upper half, the zero of the lane's row.
// PARTS = 2: a[0] and a[1] are the rows' upper and lower parts, else there is a[0] alone.
template <int PARTS = 1>
__device__ inline void group_product(const uint4& w, uint32_t sz, const Rows* a, f4& sum) {
  const _Float16 z = __builtin_bit_cast(_Float16, uint16_t(sz >> 16));
  const _Float16 zl = -(static_cast<_Float16>(1024.0f) + z), zh = -(static_cast<_Float16>(64.0f) + z);
  const h2 zlo = {zl, zl}, zhi = {zh, zh};
  const uint32_t wv[4] = {w.x, w.y, w.z, w.w};
  f4 g = {0.f, 0.f, 0.f, 0.f}, low = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const h8 b = dequant_word(wv[k], zlo, zhi, 0x000F000Fu, 0x00F000F0u, 0x64006400u);
    g = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[0].v[k], b, g, 0, 0, 0);
    if constexpr (PARTS == 2) low = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[1].v[k], b, low, 0, 0, 0);
  }
  const float s = static_cast<float>(__builtin_bit_cast(_Float16, uint16_t(sz)));
  if constexpr (PARTS == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = __builtin_fmaf(kRestDown, low[i], g[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = __builtin_fmaf(s, g[i], sum[i]);
}

// Scales and zeros come four groups at a time, 16 lanes to a group: a load for each group would cost the CU's load
// path as much as the group's weights (gate and up of 4 tokens, 4096 -> 14336: 92 us against 54 without them, 53 now). Here
// every lane gets them all.
__device__ inline void spread4(uint32_t v, uint32_t (&o)[4]) {
  const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // groups 0 1 0 1, groups 2 3 2 3
  const auto lo = __builtin_amdgcn_permlane16_swap(halves[0], halves[0], false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(halves[1], halves[1], false, false);
  o[0] = lo[0];
  o[1] = lo[1];
  o[2] = hi[0];
  o[3] = hi[1];
}

template <class T>
using gptr = const T __attribute__((address_space(1)))*;

// A load from a uniform address plus a lane's own 32-bit offset, with the address in scalar registers. (The compiler is
// kept from hoisting the lane's part into 64-bit sums of its own, a pair of registers each: the address by the empty
// statement here, the offset by opaque() in the block of the load.)
template <class T>
__device__ inline T at(const void* base, uint32_t off, int more = 0) {
  uintptr_t p = reinterpret_cast<uintptr_t>(base);
  asm volatile("" : "+s"(p));
  return *(gptr<T>)((gptr<char>)p + off + more);
}
__device__ inline void opaque(uint32_t& off) { asm volatile("" : "+v"(off)); }
using u4 = uint32_t __attribute__((ext_vector_type(4)));
// ONCE: past the caches (see kOnceGateUp).
template <bool ONCE>
__device__ inline uint4 load_weights(const void* w, uint32_t& wo) {
  opaque(wo);
  if constexpr (ONCE) {
    uintptr_t p = reinterpret_cast<uintptr_t>(w);
    asm volatile("" : "+s"(p));
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load((gptr<u4>)((gptr<char>)p + wo)));
  } else {
    return __builtin_bit_cast(uint4, at<u4>(w, wo));
  }
}
__device__ inline void load_scales(uint32_t& scale, uint32_t& zero, const void* sp, const void* zp, uint32_t& so) {
  opaque(so);
  scale = at<uint16_t>(sp, so);
  zero = at<uint16_t>(zp, so);
}
// step: from a lane's 8 channels to its next 8.
__device__ inline void load_rows(Rows& r, const void* base, uint32_t& off, uint32_t step) {
  opaque(off);
#pragma unroll
  for (int k = 0; k < 4; ++k) r.v[k] = at<h8>(static_cast<const char*>(base) + k * step, off);
}
__device__ inline void load_rows(Rows& r, const void* base, uint32_t& off) {  // (16: as offsets of the instructions)
  opaque(off);
#pragma unroll
  for (int k = 0; k < 4; ++k) r.v[k] = at<h8>(base, off, k * 16);
}

// All that is computed up to here comes before whatever is loaded later.
__device__ inline void settled(f4& v) { asm volatile("" : "+v"(v) : : "memory"); }

// Where channel n of a row lies in the order of fragments: within its group the lanes' first 8 channels, then their
// second 8, ..., so that each load of a row takes 64 bytes that follow each other; within 8 the order of dequant_word.
__device__ inline int fragment_place(int n) {
  const int h = n >> 5 & 3, k = n >> 3 & 3, j = n & 7;
  return (n & ~127) | k << 5 | h << 3 | (j & 3) << 1 | j >> 2;
}

// Workgroups go through the tiles (16 gate and 16 up rows of a unit's expert), unit by unit, each a run of them. W waves
// share out the groups of channels: wave w has GW of them from group GW w on, whose part of the unit's tokens it keeps
// in registers (GW = 0: any number, w, w + W, ..., read again for each tile). Weights come straight into a ring of
// registers, R groups ahead, from tile to tile without a break: a tile's gate rows, then its up rows. Every kPark
// tiles, and where the unit ends, the waves' sums meet in LDS.
// PARTS = 2: the tokens' rows come from a transform, in two float16 parts, and take twice the registers and products (with
// sums of their own, group by group, for the lower parts).
// How many waves, and so how many groups to each, is a matter of registers: 16 waves on a CU leave each 128.
constexpr int kPark = 4;
template <int W, int GW, int PARTS, bool ONCE>
__global__ __launch_bounds__(64 * W, 4) void gate_up_kernel(const MoeCall c) {
  constexpr int R = GW == 1 ? 2 : GW == 3 ? 6 : 4;
  constexpr int S = GW ? 2 * GW : R;  // steps of a tile
  static_assert(S % R == 0, "a step's slot and its group are fixed");
  __shared__ f4 red[kPark][2][W][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), nl = lane & 15, h = lane >> 4;
  const int G = c.D / PARO_GROUP, per_unit = c.F / 16;
  const int total = *c.t.units * per_unit;
  const int begin = int(size_t(total) * blockIdx.x / gridDim.x), end = int(size_t(total) * (blockIdx.x + 1) / gridDim.x);
  if (begin == end) return;
  auto group = [&](int i) { return min(GW ? wave * GW + i : wave + W * i, G - 1); };  // past the last one that one again
  uint32_t wo = nl * 64 + h * 16;                                  // this lane's part of a group of 16 rows,
  uint32_t so = (nl * G + (GW ? group(GW == 1 ? 0 : GW == 2 ? h & 1 : min(h, GW - 1)) : 0)) * 2;  // and its scale and zero
  const size_t wup = size_t(c.F) * (c.D / 2), sup = size_t(c.F) * G * 2;  // from a gate row to its up row
  // the tile that is loaded: its unit, its place in it, its first gate row's addresses
  int lu = begin / per_unit, lt = begin - lu * per_unit, left = end - begin;
  const char *wp, *sp, *zp;
  auto aim = [&]() {
    const size_t row = size_t(__builtin_amdgcn_readfirstlane(c.t.unit[lu].expert)) * 2 * c.F + lt * 16;
    wp = reinterpret_cast<const char*>(c.gu_qw) + row * (c.D / 2);
    sp = reinterpret_cast<const char*>(c.gu_sc) + row * G * 2;
    zp = reinterpret_cast<const char*>(c.gu_zr) + row * G * 2;
  };
  aim();
  auto next_tile = [&]() {  // past the end the last tile again
    if (--left > 0) {
      wp += size_t(8) * c.D;
      sp += size_t(32) * G;
      zp += size_t(32) * G;
      if (++lt == per_unit) {
        lt = 0;
        ++lu;
        aim();
      }
    }
  };
  uint4 w[R];
  uint32_t scale[GW ? 2 : R], zero[GW ? 2 : R], sz[4];
  auto issue = [&](int q, int half, int i) {
    const int g = group(i);
    const size_t sa = (half ? sup : 0) + (GW ? 0 : uint32_t(g) * 2);
    if (GW == 0 || i == 0) load_scales(scale[GW ? half : q], zero[GW ? half : q], sp + sa, zp + sa, so);
    w[q] = load_weights<ONCE>(wp + (half ? wup : 0) + uint32_t(g) * 1024, wo);
  };
  auto spread = [&](int half) {
    const uint32_t v = scale[half] | zero[half] << 16;
    if constexpr (GW == 1) {
      sz[0] = v;
    } else if constexpr (GW == 2) {
      const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      sz[0] = r[0];
      sz[1] = r[1];
    } else {
      spread4(v, sz);
    }
  };
  // GW = 0: a step is a group's gate and up rows, in two slots of the ring, and a tile an even number of them
  const int gw = ((G + W - 1) / W + 1) / 2 * 2;
  int li = 0;
  auto issue_both = [&](int p) {
    issue(2 * p, 0, li);
    issue(2 * p + 1, 1, li);
    if (++li == gw) {
      li = 0;
      next_tile();
    }
  };
  if constexpr (GW > 0) {
#pragma unroll
    for (int q = 0; q < R; ++q) issue(q, q / GW, q % GW);
  } else {
    issue_both(0);
    issue_both(1);
  }
  __builtin_amdgcn_sched_barrier(0);

  Rows a[GW ? GW : 2][PARTS];
  int unit = begin / per_unit, tile = begin - unit * per_unit, first = 0, count = 0;
  uint32_t xo = 0;
  uint32_t mine = 0;  // of the token whose results this thread makes: its pair, and its row's power in the upper half
  // a group of the unit's tokens; past the last one zeros, so that its products are
  auto rows = [&](int q, int i) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) load_rows(a[q][p], c.x + size_t(p) * c.M * c.D + size_t(group(i)) * PARO_GROUP, xo);
  };
  auto settle = [&](int q, int i) {
    const bool in = (GW ? wave * GW + i : wave + W * i) < G;
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const u4 v = __builtin_bit_cast(u4, PARTS == 2 ? a[q][p].v[k] : decode_order(a[q][p].v[k]));
        a[q][p].v[k] = __builtin_bit_cast(h8, in ? v : u4{0u, 0u, 0u, 0u});
      }
  };
  auto tokens = [&]() {
    first = __builtin_amdgcn_readfirstlane(c.t.unit[unit].first);
    count = __builtin_amdgcn_readfirstlane(c.t.unit[unit].count);
    xo = uint32_t(c.t.slot[first + min(nl, count - 1)].token) * uint32_t(c.D) * 2 + h * 64;
    const MoeSlot s = c.t.slot[first + min(tid >> 4 & 15, count - 1)];
    mine = s.pair | uint32_t(c.power[s.token]) << 16;
    if constexpr (GW > 0) {
#pragma unroll
      for (int i = 0; i < GW; ++i) rows(i, i);
#pragma unroll
      for (int i = 0; i < GW; ++i) settle(i, i);
    } else {
      rows(0, 0);
      rows(1, 1);
    }
  };
  tokens();
  f4 acc[2] = {};
  int parked = 0;
  auto park = [&](int half) {
    red[parked][half][wave][lane] = acc[half];
    acc[half] = f4{0.f, 0.f, 0.f, 0.f};
  };
  for (int t = begin;;) {
    if constexpr (GW > 0) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        __builtin_amdgcn_sched_barrier(0);
        if (s % GW == 0) spread(s / GW);
        group_product<PARTS>(w[s % R], sz[s % GW], a[s % GW], acc[s / GW]);
        settled(acc[s / GW]);
        if (s % GW == GW - 1) park(s / GW);
        __builtin_amdgcn_sched_barrier(0);
        if (s + R == S) next_tile();
        issue(s % R, (s + R) % S / GW, (s + R) % GW);
      }
    } else {
      for (int i = 0; i < gw; i += 2) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          __builtin_amdgcn_sched_barrier(0);
          settle(p, i + p);
          group_product<PARTS>(w[2 * p], scale[2 * p] | zero[2 * p] << 16, a[p], acc[0]);
          group_product<PARTS>(w[2 * p + 1], scale[2 * p + 1] | zero[2 * p + 1] << 16, a[p], acc[1]);
          settled(acc[0]);
          settled(acc[1]);
          __builtin_amdgcn_sched_barrier(0);
          issue_both(p);
          rows(p, i + p + 2 < gw ? i + p + 2 : i + p + 2 - gw);
        }
      }
      park(0);
      park(1);
    }
    __builtin_amdgcn_sched_barrier(0);
    ++t;
    ++tile;
    ++parked;
    if (parked < kPark && tile < per_unit && t < end) continue;
    __syncthreads();
    static_assert(64 * W % 256 == 0, "a thread has one token");
    for (int o = tid; o < parked * 256; o += 64 * W) {
      const int col = o & 15, m = o >> 4 & 15, j = o >> 8, l = (m >> 2) * 16 + col, i = m & 3;
      if (m >= count) continue;
      float gate = 0, upv = 0;
#pragma unroll
      for (int v = 0; v < W; ++v) {
        gate += red[j][0][v][l][i];
        upv += red[j][1][v][l][i];
      }
      const int power = int(mine) >> 16;
      if constexpr (PARTS == 2) {
        gate *= power2(power);
        upv *= power2(power);
      }
      float v = gate / (1.0f + expf(-gate)) * upv;
      const size_t row = size_t(mine & 0xFFFFu) * c.F;
      const int n = (tile - parked + j) * 16 + col;
      if (c.a_fragments) {
        v *= power2(kLiftA - 2 * power);
        _Float16* const to = static_cast<_Float16*>(c.a) + row + fragment_place(n);
        *to = static_cast<_Float16>(v);
        to[size_t(c.M) * c.top_k * c.F] = __builtin_bit_cast(_Float16, rest16(v, static_cast<_Float16>(v)));
      } else
        static_cast<float*>(c.a)[row + n] = v;
    }
    if (t == end) break;
    parked = 0;
    if (tile == per_unit) {
      tile = 0;
      ++unit;
      tokens();
    }
    __syncthreads();  // the sums have been read
  }
}

struct DownArgs {
  MoeCall c;
  int splits;
};

// A workgroup has T times 16 columns of y and its share of the items, an item being four groups of a unit: the items in
// order are cut into splits * W equal runs, one for each wave. A wave keeps sums of its own for every token in LDS, to
// which it adds an expert's products times the tokens' weights where it leaves the expert. R groups are in flight.
// a is in two float16 parts (one would leave an error as large as y's own rounding, 3.2e-4 of a float16 y instead of
// 2.1e-4). A unit of up to 8 tokens has 8 rows of the matrix products to spare: they take the lower parts, at no cost in
// loads or products. A fuller unit, which only calls of more tokens have (PARTS = 2), loads them besides and takes them
// through products of their own (64 tokens, 8 of 64 experts, 4096 -> 1408: 57 us, 48 without). Those loads come in front of the
// group's others: the waits count as if they were not there, and so wait for no weights that are asked for later.
//
// What bounds it is what a CU takes in, some 38 KB a microsecond here (weights from HBM and a from the L2 cache; more
// groups in flight change nothing): a group of 16 rows of a, or of 8 in two parts, is four times the bytes of 16 columns'
// weights, so more columns to a workgroup cost less, as long as there is a workgroup for each CU.
template <int W, int T, int R, int PARTS, bool ONCE>
__global__ __launch_bounds__(64 * W, T == 4 || (T == 2 && PARTS == 2) ? 2 : 4) void down_kernel(const DownArgs args) {
  static_assert(R == 2 || R == 4, "a group's slot is fixed");
  extern __shared__ __attribute__((aligned(16))) char smem[];  // float [W][M][16 T], then the tables, then float [M]
  const MoeCall& c = args.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), nl = lane & 15, h = lane >> 4;
  const int pairs = c.M * c.top_k, tile = blockIdx.x / args.splits, split = blockIdx.x - tile * args.splits;
  float* const all = reinterpret_cast<float*>(smem);
  float* const sums = all + wave * c.M * 16 * T;
  MoeSlot* const slot = reinterpret_cast<MoeSlot*>(all + W * c.M * 16 * T);
  MoeUnit* const unit = reinterpret_cast<MoeUnit*>(slot + pairs);
  const int units = *c.t.units;
  float* const undo = reinterpret_cast<float*>(unit + units);  // [M]: what takes a's power of two off again
  for (int i = tid; i < c.M; i += 64 * W) undo[i] = power2(2 * c.power[i] - kLiftA);
  for (int i = tid; i < pairs; i += 64 * W) slot[i] = c.t.slot[i];  // (those past the last one are not used)
  for (int i = tid; i < units; i += 64 * W) unit[i] = c.t.unit[i];
  for (int i = lane; i < c.M * 16 * T; i += 64) sums[i] = 0;
  __syncthreads();
  const int G = c.F / PARO_GROUP, Q = (G + 3) / 4, total = units * Q, runs = args.splits * W, run = split * W + wave;
  const int begin = int(size_t(total) * run / runs), end = int(size_t(total) * (run + 1) / runs);
  uint32_t wo = nl * 64 + h * 16, so = 0, ao = 0;  // this lane's part of a group of 16 rows, its scale and zero, its row of a
  f4 acc[T] = {};
  uint4 w[R][T];
  Rows a[R][PARTS];
  uint32_t scale[T], zero[T], sz[T][4];
  // the item that is loaded next: its unit, four groups and addresses; and the one that is used next
  int lu = begin / Q, lq = begin - lu * Q, uu = lu, uq = lq, left = end - begin;
  bool lfull = false, ufull = false;  // their units have more than kTwoParts tokens
  const char *wp = nullptr, *sp = nullptr, *zp = nullptr;
  auto aim = [&]() {  // (no global access: the wait counts stay exact)
    const MoeUnit k = unit[lu];
    const int count = __builtin_amdgcn_readfirstlane(k.count);
    lfull = PARTS == 2 && count > kTwoParts;
    const int r = min(lfull ? nl : nl % kTwoParts, count - 1);
    ao = (uint32_t(slot[k.first + r].pair) + (!lfull && nl >= kTwoParts ? pairs : 0)) * uint32_t(c.F) * 2 + h * (c.a_fragments ? 16 : 64);
    const size_t row = size_t(__builtin_amdgcn_readfirstlane(k.expert)) * c.D + tile * 16 * T;
    wp = reinterpret_cast<const char*>(c.dn_qw) + row * (c.F / 2);
    sp = reinterpret_cast<const char*>(c.dn_sc) + row * G * 2;
    zp = reinterpret_cast<const char*>(c.dn_zr) + row * G * 2;
  };
  auto advance = [&]() {  // past the end the last item again
    if (--left > 0 && ++lq == Q) {
      lq = 0;
      ++lu;
      aim();
    }
  };
  auto load = [&](int q, int p) {  // the item's group p; past the last one that one again
    if (p == 0) {
      so = (nl * G + min(4 * lq + h, G - 1)) * 2;
#pragma unroll
      for (int t = 0; t < T; ++t) load_scales(scale[t], zero[t], sp + size_t(t) * 32 * G, zp + size_t(t) * 32 * G, so);
    }
    const uint32_t g = min(4 * lq + p, G - 1);
    if (PARTS == 2 && lfull) load_rows(a[q][PARTS - 1], c.a_down + (size_t(pairs) * c.F + g * PARO_GROUP), ao, c.a_fragments ? 64 : 16);
#pragma unroll
    for (int t = 0; t < T; ++t) w[q][t] = load_weights<ONCE>(wp + size_t(t) * 8 * c.F + g * 1024, wo);
    load_rows(a[q][0], c.a_down + g * PARO_GROUP, ao, c.a_fragments ? 64 : 16);
  };
  if (begin < end) {
    aim();
    ufull = lfull;
#pragma unroll
    for (int q = 0; q < R; ++q) load(q, q);
    for (int n = end - begin; n > 0; --n) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        __builtin_amdgcn_sched_barrier(0);
        if (p == 0) {
#pragma unroll
          for (int t = 0; t < T; ++t) spread4(scale[t] | zero[t] << 16, sz[t]);
        }
        if (p == 0 || 4 * uq + p < G) {  // uniform, as full is
          if (PARTS == 2 && ufull) {
#pragma unroll
            for (int t = 0; t < T; ++t) {
              group_product<PARTS>(w[p % R][t], sz[t][p], a[p % R], acc[t]);
              settled(acc[t]);
            }
          } else {
#pragma unroll
            for (int t = 0; t < T; ++t) {
              group_product(w[p % R][t], sz[t][p], a[p % R], acc[t]);
              settled(acc[t]);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (p + R == 4) advance();
        load(p % R, (p + R) % 4);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (++uq == Q || n == 1) {
        const MoeUnit k = unit[uu];
        if (!ufull) {  // lanes 32..63 have the lower parts' sums
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(kRestDown, __shfl_xor(acc[t][i], 32), acc[t][i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * h + i;
          if (r < k.count) {
            // (an expert has a token once: no two lanes meet)
            const MoeSlot o = slot[k.first + r];
            const float by = undo[o.token];
#pragma unroll
            for (int t = 0; t < T; ++t) {
              float& v = sums[(o.token * T + t) * 16 + nl];
              v = __builtin_fmaf(o.weight, acc[t][i] * by, v);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) acc[t] = f4{0.f, 0.f, 0.f, 0.f};
        uq = 0;
        ++uu;
        if (PARTS == 2 && n > 1) ufull = __builtin_amdgcn_readfirstlane(unit[uu].count) > kTwoParts;
      }
    }
  }
  __syncthreads();
  for (int o = tid; o < c.M * 16 * T; o += 64 * W) {
    const int m = o / (16 * T), n = o % (16 * T);
    float v = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) v += all[i * c.M * 16 * T + o];
    const size_t to = size_t(m) * c.D + tile * 16 * T + n;
    if (args.splits > 1)
      c.part[size_t(split) * c.M * c.D + to] = v;
    else if (c.ydtype == PARO_F32)
      static_cast<float*>(c.y)[to] = v;
    else
      static_cast<_Float16*>(c.y)[to] = static_cast<_Float16>(v);
  }
}

// y from the partial sums of the splits, in their order; 4 values a thread.
__global__ __launch_bounds__(256) void sum_kernel(const float* part, int splits, int total, void* y, int ydtype) {
  const int i = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f4*>(part + size_t(s) * total + i);
  if (ydtype == PARO_F32) {
    *reinterpret_cast<f4*>(static_cast<float*>(y) + i) = v;
  } else {
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<h4*>(static_cast<_Float16*>(y) + i) = __builtin_convertvector(v, h4);
  }
}

// The experts that a call reaches, where each choice of a token is as good as any other, and the units that those have.
double reached(int M, int E, int top_k) { return E * (1.0 - std::pow(1.0 - std::min(1.0, double(top_k) / E), M)); }
double expected_units(int M, int E, int top_k) {
  if (M <= 16) return reached(M, E, top_k);
  if (top_k >= E) return E * ((M + 15) / 16);
  const double p = double(top_k) / E;
  double sum = 0, chance = std::pow(1.0 - p, M);  // of an expert's having c tokens
  for (int c = 0; c <= M; ++c) {
    sum += chance * ((c + 15) / 16);
    chance *= p / (1.0 - p) * (M - c) / (c + 1);
  }
  return E * sum;
}

// From so many bytes of the reached experts' weights on they are loaded past the caches, and leave those to what is read
// again. Three sets of weights in turn, a layer with its loads in the caches and past them. Gate and up: 30 MB (8 tokens, 4
// of 16 experts, 2048 -> 1024) 30.1 and 30.7 us; 46 MB (4, 2 of 8, 4096 -> 2048) 31.9 and 32.6; 60 MB (8, 4 of 16, 2048 ->
// 2048) 39.9 and 39.0; 132 MB (32, 4 of 32, 4096 -> 1024) 66.2 and 60.2; 265 MB (32, 4 of 32, 4096 -> 2048) 106.4 and 100.0.
// Down: 21 to 92 MB within 1 % either way, 41 MB (13, 4 of 60, 1536 -> 1408, behind transforms) 62 and 65; 132 MB (32, 4 of
// 32, 4096 -> 2048) 106.4 and 104.1; 160 MB (4, 2 of 8, 4096 -> 14336) 103 and 100.
// Where experts have 16 tokens and more, most have several units, which read the same weights, and the caches keep them: 64
// tokens, 2 of 4 experts, 4096 -> 14336 (32 tokens to an expert) 242 us past the caches, 222 through them; 32 tokens (16 to
// an expert) 138 and 134; 24 tokens, 1 of 2 (12) 71 and 75; 64 tokens, 8 of 64, 4096 -> 1408 (8) 146 and 151.
constexpr double kOnceGateUp = 48e6, kOnceDown = 128e6;
bool weights_once(int M, int D, int F, int E, int top_k, double rows, double least) {  // rows: of weights, half a byte a channel
  return M * top_k < 16 * E && reached(M, E, top_k) * rows / 2 * F * D >= least;
}

// Workgroups: as many as the GPU holds at once (16 waves on a CU), and no more than there can be tiles.
template <int W, int GW, int PARTS>
hipError_t launch_gate_up(const MoeCall& c, bool once, hipStream_t st) {
  const long tiles = long(moe_units_max(c.M, c.E, c.top_k)) * (c.F / 16);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(std::min<long>(tiles, long(kCUs) * (16 / W)))), dim3(64 * W), 0, st, c);
    return hipGetLastError();
  };
  return once ? go(gate_up_kernel<W, GW, PARTS, true>) : go(gate_up_kernel<W, GW, PARTS, false>);
}

constexpr int kDownWaves = 8;
constexpr size_t down_lds(int T, int M, int units, int pairs) {
  return size_t(kDownWaves) * T * M * 64 + sizeof(MoeSlot) * pairs + sizeof(MoeUnit) * units + 4 * M;
}
static_assert(down_lds(4, PARO_MOE_MAX_M, PARO_MOE_MAX_E + PARO_MOE_MAX_M, PARO_MOE_MAX_M * PARO_MOE_MAX_K) <= 160 * 1024, "a CU's LDS");

}  // namespace

int moe_units_max(int M, int E, int top_k) { return std::min(E, M * top_k) + M * top_k / 16; }

// 16, 32 or 64 columns to a workgroup, and how many workgroups share them, by an estimate in microseconds: a CU's time for
// an item (four groups of a unit's rows), fitted to ten calls of 1 to 64 tokens at 27 cuts each, and the kernel that adds
// the parts. The shares are those that fill the GPU once, or one. Measured (with one part of a), a layer with 16 columns to a workgroup and no shares, with 32, 64 and
// as many shares as fill the GPU: 4 tokens, 2 of 8 experts, 4096 -> 14336 112, 107 and 106 us; 8 tokens, 4 of 16, 4096 ->
// 2048 48, 48 and 47; 64 tokens, 8 of 64, 4096 -> 1408 174, 150 and 142; one token, 8 of 64, 2048 -> 1024 21.5, 21.2 and 22.9.
MoeDownPlan moe_down_plan(int M, int D, int F, int E, int top_k) {
  constexpr double kItem[3] = {0.28, 0.39, 0.62}, kSum = 4.0;
  const double items = expected_units(M, E, top_k) * ((F / PARO_GROUP + 3) / 4);
  MoeDownPlan best{};
  double least = 1e30;
  for (int i = 0; i < 3; ++i) {
    const int columns = D / 16 >> i, rounds = (columns + kCUs - 1) / kCUs;
    const int shares = std::min({32, kCUs / columns, int(items / 3)});
    auto take = [&](int s, double us) {
      if (us < least) {
        least = us;
        best = MoeDownPlan{1 << i, s, M <= kTwoParts, false};
      }
    };
    take(1, rounds * items * kItem[i]);
    if (shares > 1) take(shares, items / shares * kItem[i] + kSum);
  }
  best.once = best.tiles == 4 && weights_once(M, D, F, E, top_k, 1, kOnceDown);  // (so much has wide columns, nearly always)
  return best;
}

// Waves, and groups of channels to each (0: any number), by the groups of a row and by the registers that the tokens' rows
// take: twice as many in two parts. (There, eight waves for 5 to 8 groups: half as many workgroups load the tokens; against
// four of two groups each, a layer of 50 tokens, 2 of 6 experts, 896 -> 2688 43 us against 47, of 64, 4 of 60, 1024 -> 1408
// 69 against 67.)
MoeGateUpPlan moe_gate_up_plan(int M, int D, int F, int E, int top_k, int parts) {
  const int G = D / PARO_GROUP;
  const bool once = weights_once(M, D, F, E, top_k, 2, kOnceGateUp);
  if (parts == 2) {
    if (G > 32) return {16, 0, once};
    return G <= 4 ? MoeGateUpPlan{4, 1, once} : G <= 8 ? MoeGateUpPlan{8, 1, once} : G <= 16 ? MoeGateUpPlan{8, 2, once} : MoeGateUpPlan{16, 2, once};
  }
  if (G > 64) return {16, 0, once};
  const int waves = G <= 16 ? 4 : G <= 32 ? 8 : 16;
  return {waves, std::max((G + waves - 1) / waves, waves > 4 ? 3 : 1), once};
}

hipError_t launch_moe_gate_up(const MoeCall& c, hipStream_t st) {
  const MoeGateUpPlan p = moe_gate_up_plan(c.M, c.D, c.F, c.E, c.top_k, c.x_parts ? 2 : 1);
  const auto is = [&](int waves, int groups) { return p.waves == waves && p.groups == groups; };
  if (c.x_parts) {
    if (is(4, 1)) return launch_gate_up<4, 1, 2>(c, p.once, st);
    if (is(8, 1)) return launch_gate_up<8, 1, 2>(c, p.once, st);
    if (is(8, 2)) return launch_gate_up<8, 2, 2>(c, p.once, st);
    if (is(16, 2)) return launch_gate_up<16, 2, 2>(c, p.once, st);
    return launch_gate_up<16, 0, 2>(c, p.once, st);
  }
  if (is(4, 1)) return launch_gate_up<4, 1, 1>(c, p.once, st);
  if (is(4, 2)) return launch_gate_up<4, 2, 1>(c, p.once, st);
  if (is(4, 3)) return launch_gate_up<4, 3, 1>(c, p.once, st);
  if (is(4, 4)) return launch_gate_up<4, 4, 1>(c, p.once, st);
  if (is(8, 3)) return launch_gate_up<8, 3, 1>(c, p.once, st);
  if (is(8, 4)) return launch_gate_up<8, 4, 1>(c, p.once, st);
  if (is(16, 3)) return launch_gate_up<16, 3, 1>(c, p.once, st);
  if (is(16, 4)) return launch_gate_up<16, 4, 1>(c, p.once, st);
  return launch_gate_up<16, 0, 1>(c, p.once, st);
}

hipError_t launch_moe_down(const MoeCall& c, hipStream_t st) {
  constexpr int W = kDownWaves;
  const MoeDownPlan p = moe_down_plan(c.M, c.D, c.F, c.E, c.top_k);
  const DownArgs a{c, p.splits};
  const size_t lds = down_lds(p.tiles, c.M, moe_units_max(c.M, c.E, c.top_k), c.M * c.top_k);
  auto go = [&](auto kernel) {
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, int(lds))) return e;
    hipLaunchKernelGGL(kernel, dim3(unsigned(c.D / 16 / p.tiles * p.splits)), dim3(64 * W), lds, st, a);
    return hipGetLastError();
  };
  if (hipError_t e = p.tiles == 1   ? p.few ? go(down_kernel<W, 1, 4, 1, false>) : go(down_kernel<W, 1, 2, 2, false>)
                     : p.tiles == 2 ? p.few ? go(down_kernel<W, 2, 2, 1, false>) : go(down_kernel<W, 2, 2, 2, false>)
                     : p.once       ? p.few ? go(down_kernel<W, 4, 2, 1, true>) : go(down_kernel<W, 4, 2, 2, true>)
                                    : p.few ? go(down_kernel<W, 4, 2, 1, false>) : go(down_kernel<W, 4, 2, 2, false>))
    return e;
  if (p.splits > 1) {
    const int total = c.M * c.D;
    hipLaunchKernelGGL(sum_kernel, dim3(unsigned((total / 4 + 255) / 256)), dim3(256), 0, st, c.part, p.splits, total, c.y, c.ydtype);
  }
  return hipGetLastError();
}

}  // namespace paro
