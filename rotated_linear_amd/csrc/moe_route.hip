// The router of a mixture-of-experts layer: logits, then the experts of each token with their weights.
//
// Logits are float64 sums of products that are exact in it: which expert a token takes hangs on the order of two
// logits, and a float32 sum turns close ones round. Bound by latency: one token, 64 experts, 2048 channels 2.5 us, little more
// than a launch, choice and tables 4.8, the round trips to LDS of one workgroup; 64 tokens, 64 experts, 4096 channels 5.8,
// choice 4.6, tables 4.7.
#include <algorithm>

#include "moe_tables.h"
#include "w4_device.h"

namespace paro {
namespace {

constexpr int kMaxM = PARO_MOE_MAX_M, kMaxK = PARO_MOE_MAX_K;
static_assert(PARO_MOE_MAX_E == 512, "a thread for each expert; select_kernel<2> has room for 512");
constexpr int kWaves = 8;

// Moves of a double between lanes without LDS, in its two halves.
template <class F>
__device__ inline double by_halves(double v, F move) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, uint64_t(move(uint32_t(b))) | uint64_t(move(uint32_t(b >> 32))) << 32);
}
// v plus what a data-parallel move brings; lanes without a source add 0.
template <int CTRL, int ROWS>
__device__ inline double plus_moved(double v) {
  return v + by_halves(v, [](uint32_t h) { return uint32_t(__builtin_amdgcn_update_dpp(0, int(h), CTRL, ROWS, 0xF, false)); });
}
// In lane 15 of each row of 16 lanes: the row's sum.
__device__ inline double row_sum(double v) {
  v = plus_moved<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8
  v = plus_moved<0x112, 0xF>(v);
  v = plus_moved<0x114, 0xF>(v);
  return plus_moved<0x118, 0xF>(v);
}
__device__ inline double lane_of(double v, int lane) {
  return by_halves(v, [lane](uint32_t h) { return uint32_t(__builtin_amdgcn_readlane(int(h), lane)); });
}
// In every lane: the wave's sum.
__device__ inline double wave_sum(double v) {
  v = row_sum(v);
  v = plus_moved<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = plus_moved<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return lane_of(v, 63);
}
// D = 32 (16): in the wave's first half (its even rows) a plus the other half's (the next row's) a, in the others b plus b.
template <int D>
__device__ inline double traded_sum(double a, double b) {
  const uint64_t x = __builtin_bit_cast(uint64_t, a), y = __builtin_bit_cast(uint64_t, b);
  uint64_t lo = 0, hi = 0;
#pragma unroll
  for (int s = 0; s < 64; s += 32) {
    const auto r = D == 32 ? __builtin_amdgcn_permlane32_swap(uint32_t(x >> s), uint32_t(y >> s), false, false)
                           : __builtin_amdgcn_permlane16_swap(uint32_t(x >> s), uint32_t(y >> s), false, false);
    lo |= uint64_t(uint32_t(r[0])) << s;
    hi |= uint64_t(uint32_t(r[1])) << s;
  }
  return __builtin_bit_cast(double, lo) + __builtin_bit_cast(double, hi);
}

// The power of a row of x (moe_internal.h), by all threads of a workgroup: 2^power is over its norm and at most twice it;
// 0 for a row of zeros, and for one that has no finite norm.
__device__ inline void row_power(const uint16_t* x, int D, int* power) {
  __shared__ double part[kWaves];
  const int tid = threadIdx.x;
  double v = 0;
  for (int c = tid; c < D / 8; c += 64 * kWaves) {
    const h8 w = *reinterpret_cast<const h8*>(x + c * 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) v = __builtin_fma(double(float(w[k])), double(float(w[k])), v);
  }
  v = wave_sum(v);
  if ((tid & 63) == 0) part[tid >> 6] = v;
  __syncthreads();
  if (tid == 0) {
    v = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += part[i];
    const int e = int(__builtin_bit_cast(uint64_t, v) >> 52);  // (exact squares: no subnormal sums)
    *power = e == 0 || e == 2047 ? 0 : ((e - 1023) >> 1) + 1;
  }
}

// A workgroup has MT tokens and ET experts; its threads take 8 channels at a time. With r.power there are MT more to each
// row of the grid, for the powers of its tokens.
template <bool F32, int MT, int ET>
__global__ __launch_bounds__(64 * kWaves) void logits_kernel(const MoeRoute r) {
  constexpr int V = MT * ET;
  __shared__ double part[kWaves][V];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e0 = blockIdx.x * ET, m0 = blockIdx.y * MT;
  const int tiles = (r.E + ET - 1) / ET;
  if (int(blockIdx.x) >= tiles) {
    const int m = m0 + blockIdx.x - tiles;
    if (m < r.M) row_power(r.x + size_t(m) * r.D, r.D, r.power + m);
    return;
  }
  double acc[V] = {};
  for (int c = tid; c < r.D / 8; c += 64 * kWaves) {
    float w[ET][8];
#pragma unroll
    for (int i = 0; i < ET; ++i) {
      const size_t row = size_t(min(e0 + i, r.E - 1)) * r.D + c * 8;
      if constexpr (F32) {
        const float* const p = static_cast<const float*>(r.router) + row;
        const f4 lo = *reinterpret_cast<const f4*>(p), hi = *reinterpret_cast<const f4*>(p + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[i][k] = k < 4 ? lo[k] : hi[k - 4];
      } else {
        const h8 v = *reinterpret_cast<const h8*>(static_cast<const uint16_t*>(r.router) + row);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[i][k] = float(v[k]);
      }
    }
    h8 x[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = *reinterpret_cast<const h8*>(r.x + size_t(min(m0 + j, r.M - 1)) * r.D + c * 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < ET; ++i) acc[j * ET + i] = __builtin_fma(double(float(x[j][k])), double(w[i][k]), acc[j * ET + i]);
    }
  }
  // The wave's sums. While there are several, halves of the wave (then its rows of 16 lanes) trade them, so that each
  // goes on with half of them; what is left is summed over the row, or over the wave.
  if constexpr (V == 1) {
    const double v = wave_sum(acc[0]);
    if (lane == 0) part[wave][0] = v;
  } else {
    constexpr int H = V / 2, Q = V / 4;
#pragma unroll
    for (int i = 0; i < H; ++i) acc[i] = traded_sum<32>(acc[i], acc[H + i]);  // lanes 32..63: sums H + i
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const double v = row_sum(traded_sum<16>(acc[i], acc[Q + i]));  // odd rows: sums Q + i
      if ((lane & 15) == 15) part[wave][(lane >> 5) * H + (lane >> 4 & 1) * Q + i] = v;
    }
  }
  __syncthreads();
  if (tid < V) {
    const int m = m0 + tid / ET, e = e0 + tid % ET;
    double v = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += part[i][tid];
    if (m < r.M && e < r.E) r.logits[size_t(m) * r.E + e] = v;
  }
}

// A workgroup has a token. An expert's rank is how many others go before it: the larger logits, the equal ones of a
// lower index; the first top_k ranks are the token's choices. No rank waits for another, where top_k searches for
// the largest one would go through the wave one after the other. PARTS threads share the comparisons of an expert.
template <int PARTS>
__global__ __launch_bounds__(1024) void select_kernel(const MoeRoute r) {
  constexpr int kExperts = 1024 / PARTS;
  __shared__ double key[kExperts], part[16], chosen[kMaxK];
  __shared__ int id[kMaxK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = blockIdx.x, e = tid / PARTS;
  const double logit = e < r.E ? r.logits[size_t(m) * r.E + e] : 0.0;
  const double mine = logit == logit ? logit : -__builtin_inf();  // a NaN ranks as minus infinity
  if (tid % PARTS == 0) key[e] = mine;
  __syncthreads();
  int rank = 0;
#pragma unroll 4
  for (int o = tid % PARTS; o < r.E; o += PARTS) {
    const double other = key[o];
    rank += other > mine || (other == mine && o < e);
  }
#pragma unroll
  for (int d = 1; d < PARTS; d *= 2) rank += __shfl_xor(rank, d);
  if (tid % PARTS == 0 && e < r.E && rank < r.top_k) {
    id[rank] = e;
    chosen[rank] = logit;
  }
  __syncthreads();
  double sum = 0, top = 0;
  if (!r.sigmoid) {
    top = key[id[0]];
    if (wave < (r.E * PARTS + 63) / 64) sum = wave_sum(e < r.E && tid % PARTS == 0 ? exp(logit - top) : 0.0);
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += part[i];
  }
  if (tid < 64) {
    const double v = lane < r.top_k ? chosen[lane] : 0.0;
    const double w = r.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / sum;
    double all = 0;
    for (int j = 0; j < r.top_k; ++j) all += lane_of(w, j);
    if (lane < r.top_k) {
      r.ids[m * r.top_k + lane] = id[lane];
      r.weights[m * r.top_k + lane] = float(r.renormalize ? w / all : w);
    }
  }
}

// The same in one workgroup, a thread to each (token, expert) pair, for up to kOneGroup of them; and, with TABLES, the
// tables of the experts' products: a launch less. While some waves work out the weights, others count.
constexpr int kOneGroup = 1024;
template <bool TABLES>
__global__ __launch_bounds__(kOneGroup) void select_one_kernel(const MoeRoute r, const MoeTables t) {
  // Logits as whole numbers of the same order, in two halves, each token's upper halves from a multiple of four on, with
  // zeros behind them (no logit's): four are compared at a time, and the lower ones only where upper ones are equal.
  __shared__ __attribute__((aligned(16))) uint32_t upper[kOneGroup + 3 * kMaxM];
  __shared__ uint32_t lower[kOneGroup];
  __shared__ double share[kOneGroup];
  __shared__ TableWork work;
  __shared__ int ids[kMaxM * kMaxK];
  __shared__ double chosen[kMaxM * kMaxK];
  __shared__ float weights[kMaxM * kMaxK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = tid / r.E, e = tid - m * r.E, pairs = r.M * r.top_k;
  const bool live = m < r.M;
  const double logit = live ? r.logits[tid] : 0.0;
  const double mine = logit == logit ? logit + 0.0 : -__builtin_inf();  // a NaN ranks as minus infinity, -0 as 0
  const uint64_t bits = __builtin_bit_cast(uint64_t, mine), key = bits ^ (bits >> 63 ? ~0ull : 1ull << 63);
  const uint32_t high = uint32_t(key >> 32), low = uint32_t(key);
  const int stride = (r.E + 3) & ~3;
  const uint32_t* const row = upper + m * stride;
  if (live) {
    upper[m * stride + e] = high;
    lower[tid] = low;
    if (e == 0)
      for (int o = r.E; o < stride; ++o) upper[m * stride + o] = 0;
  }
  if (TABLES && tid < PARO_MOE_MAX_E) work.mask[tid] = 0;
  __syncthreads();
  if (live) {
    int rank = 0, equal = 0;
#pragma unroll 4
    for (int o = 0; o < r.E; o += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + o);
      rank += (v.x > high) + (v.y > high) + (v.z > high) + (v.w > high);
      equal += (v.x == high) + (v.y == high) + (v.z == high) + (v.w == high);
    }
    if (equal > 1)
      for (int o = 0; o < r.E; ++o) {
        const uint32_t other = lower[tid - e + o];
        rank += row[o] == high && (other > low || (other == low && o < e));
      }
    if (rank < r.top_k) {
      ids[m * r.top_k + rank] = e;
      chosen[m * r.top_k + rank] = logit;
      if (TABLES) atomicOr(&work.mask[e], 1ull << m);  // (in any order the same)
    }
  }
  __syncthreads();
  if (live && !r.sigmoid) share[tid] = exp(logit - chosen[m * r.top_k]);
  __syncthreads();
  TablePlace place{};
  if (TABLES && tid < PARO_MOE_MAX_E) {
    place = tables_count(work);
  } else {
    constexpr int kFirst = TABLES ? PARO_MOE_MAX_E / 64 : 0;
    for (int at = wave - kFirst; at < r.M; at += kOneGroup / 64 - kFirst) {  // a wave for each token
      double sum = 0;
      if (!r.sigmoid) {
        for (int o = lane; o < r.E; o += 64) sum += share[at * r.E + o];
        sum = wave_sum(sum);
      }
      const int p = at * r.top_k + lane;
      double w = 0;
      if (lane < r.top_k) w = r.sigmoid ? 1.0 / (1.0 + exp(-chosen[p])) : share[at * r.E + ids[p]] / sum;
      double all = 0;
      for (int j = 0; j < r.top_k; ++j) all += lane_of(w, j);
      if (lane < r.top_k) weights[p] = float(r.renormalize ? w / all : w);
    }
  }
  __syncthreads();
  if (TABLES && tid < PARO_MOE_MAX_E) tables_units(work, place, t);
  for (int p = tid; p < pairs; p += kOneGroup) {
    r.ids[p] = ids[p];
    r.weights[p] = weights[p];
  }
  if constexpr (TABLES) {
    __syncthreads();
    tables_slots(work, r.M, r.E, r.top_k, ids, weights, t);
  }
}

// One workgroup makes the tables; with more, each of the others has the power of a row of x.
static_assert(PARO_MOE_MAX_E == 64 * kWaves, "row_power's threads");
__global__ __launch_bounds__(PARO_MOE_MAX_E) void group_kernel(int M, int D, int E, int top_k, const uint16_t* x, const int32_t* given_ids,
                                                               const float* given_weights, const MoeTables t, int* power) {
  if (blockIdx.x > 0) {
    row_power(x + size_t(blockIdx.x - 1) * D, D, power + blockIdx.x - 1);
    return;
  }
  __shared__ TableWork work;
  __shared__ int ids[kMaxM * kMaxK];
  __shared__ float weights[kMaxM * kMaxK];
  const int tid = threadIdx.x;
  constexpr int kEach = kMaxM * kMaxK / PARO_MOE_MAX_E;
  int id[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int p = tid + i * PARO_MOE_MAX_E;
    id[i] = -1;
    if (p < M * top_k) {
      ids[p] = id[i] = given_ids[p];
      weights[p] = given_weights[p];
    }
  }
  work.mask[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (uint32_t(id[i]) < uint32_t(E)) atomicOr(&work.mask[id[i]], 1ull << ((tid + i * PARO_MOE_MAX_E) / top_k));  // (in any order the same)
  __syncthreads();
  const TablePlace place = tables_count(work);
  __syncthreads();
  tables_units(work, place, t);
  __syncthreads();
  tables_slots(work, M, E, top_k, ids, weights, t);
}

template <int MT, int ET>
hipError_t launch_logits(const MoeRoute& r, hipStream_t st) {
  const dim3 grid(unsigned((r.E + ET - 1) / ET + (r.power ? MT : 0)), unsigned((r.M + MT - 1) / MT));
  if (r.router_f32)
    hipLaunchKernelGGL((logits_kernel<true, MT, ET>), grid, dim3(64 * kWaves), 0, st, r);
  else
    hipLaunchKernelGGL((logits_kernel<false, MT, ET>), grid, dim3(64 * kWaves), 0, st, r);
  return hipGetLastError();
}

}  // namespace

// A single token: a workgroup for each expert. Few pairs of tokens and experts: as many workgroups as tiles of 4 by 1
// give; many: tiles of 4 by 4, which read half as much.
hipError_t launch_moe_logits(const MoeRoute& r, hipStream_t st) {
  if (r.M == 1) return launch_logits<1, 1>(r, st);
  return r.M * r.E <= 2048 ? launch_logits<4, 1>(r, st) : launch_logits<4, 4>(r, st);
}

// t: the tables too, or nullptr.
hipError_t launch_moe_select(const MoeRoute& r, const MoeTables* t, hipStream_t st) {
  if (r.M * r.E <= kOneGroup) {
    if (t)
      hipLaunchKernelGGL(select_one_kernel<true>, dim3(1), dim3(1024), 0, st, r, *t);
    else
      hipLaunchKernelGGL(select_one_kernel<false>, dim3(1), dim3(1024), 0, st, r, MoeTables{});
    return hipGetLastError();
  }
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(unsigned(r.M)), dim3(1024), 0, st, r);
    return hipGetLastError();
  };
  if (hipError_t e = r.E <= 64 ? go(select_kernel<16>) : r.E <= 256 ? go(select_kernel<4>) : go(select_kernel<2>)) return e;
  return t ? launch_moe_group(r.M, r.D, r.E, r.top_k, nullptr, r.ids, r.weights, *t, nullptr, st) : hipSuccess;
}

hipError_t launch_moe_group(int M, int D, int E, int top_k, const uint16_t* x, const int32_t* ids, const float* weights, const MoeTables& t,
                            int* power, hipStream_t st) {
  hipLaunchKernelGGL(group_kernel, dim3(x ? 1 + M : 1), dim3(PARO_MOE_MAX_E), 0, st, M, D, E, top_k, x, ids, weights, t, power);
  return hipGetLastError();
}

}  // namespace paro
