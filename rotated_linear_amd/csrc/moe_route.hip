// The router of a mixture-of-experts layer: logits, the experts of each token, and the tables that the experts'
// products go by.
//
// Logits are float64 sums of products that are exact in it: which expert a token takes hangs on the order of two
// logits, and a float32 sum turns close ones round.
#include <algorithm>

#include "moe_internal.h"
#include "w4_device.h"

namespace paro {
namespace {

constexpr int kMaxM = PARO_MOE_MAX_M, kMaxE = PARO_MOE_MAX_E, kMaxK = PARO_MOE_MAX_K;
constexpr int kTile = 4;  // a workgroup has 4 tokens and 4 experts

template <bool F32>
__global__ __launch_bounds__(256) void logits_kernel(const MoeRoute r) {
  __shared__ double part[4][kTile * kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e0 = blockIdx.x * kTile, m0 = blockIdx.y * kTile;
  double acc[kTile][kTile] = {};
  for (int c = tid; c < r.D / 8; c += 256) {
    double w[kTile][8];
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
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
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const h8 v = *reinterpret_cast<const h8*>(r.x + size_t(min(m0 + j, r.M - 1)) * r.D + c * 8);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double x = float(v[k]);
#pragma unroll
        for (int i = 0; i < kTile; ++i) acc[j][i] = __builtin_fma(x, w[i][k], acc[j][i]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kTile; ++j)
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      double v = acc[j][i];
#pragma unroll
      for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
      if (lane == 0) part[wave][j * kTile + i] = v;
    }
  __syncthreads();
  if (tid < kTile * kTile) {
    const int m = m0 + tid / kTile, e = e0 + tid % kTile;
    if (m < r.M && e < r.E) r.logits[size_t(m) * r.E + e] = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
  }
}

struct Shared {
  unsigned long long mask[kMaxE];  // an expert's tokens
  int first[kMaxE];                // its first slot
  int ids[kMaxM * kMaxK];
  float weights[kMaxM * kMaxK];
};

// The tables from s.ids and s.weights (all threads of the workgroup).
__device__ inline void make_tables(Shared& s, int M, int E, int top_k, const MoeTables& t) {
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int e = tid; e < kMaxE; e += nt) s.mask[e] = 0;
  __syncthreads();
  for (int p = tid; p < M * top_k; p += nt) {
    const int e = s.ids[p];
    if (e >= 0 && e < E) atomicOr(&s.mask[e], 1ull << (p / top_k));  // (an or: the same in any order)
  }
  __syncthreads();
  if (tid < 64) {  // a lane has 8 experts in a row
    constexpr int kEach = kMaxE / 64;
    int slots = 0, active = 0;
    for (int i = 0; i < kEach; ++i) {
      const int n = __popcll(s.mask[tid * kEach + i]);
      slots += n;
      active += n > 0;
    }
    int slot = slots, at = active;
    for (int d = 1; d < 64; d <<= 1) {
      const int a = __shfl_up(slot, d), b = __shfl_up(at, d);
      if (tid >= d) {
        slot += a;
        at += b;
      }
    }
    if (tid == 63) *t.active_count = at;
    slot -= slots;
    at -= active;
    for (int i = 0; i < kEach; ++i) {
      const int e = tid * kEach + i, n = __popcll(s.mask[e]);
      s.first[e] = slot;
      if (n) t.active[at++] = MoeActive{e, slot, n};
      slot += n;
    }
  }
  __syncthreads();
  for (int p = tid; p < M * top_k; p += nt) {
    const int e = s.ids[p], m = p / top_k;
    if (e < 0 || e >= E) continue;
    float w = 0;
    bool again = false;
    for (int j = 0; j < top_k; ++j)
      if (s.ids[m * top_k + j] == e) {
        again |= m * top_k + j < p;
        w += s.weights[m * top_k + j];
      }
    if (again) continue;
    const int slot = s.first[e] + __popcll(s.mask[e] & ((1ull << m) - 1));
    t.slot_token[slot] = m;
    t.slot_weight[slot] = w;
  }
}

__global__ __launch_bounds__(1024) void group_kernel(int M, int E, int top_k, const int32_t* ids, const float* weights, const MoeTables t) {
  __shared__ Shared s;
  for (int p = threadIdx.x; p < M * top_k; p += blockDim.x) {
    s.ids[p] = ids[p];
    s.weights[p] = weights[p];
  }
  make_tables(s, M, E, top_k, t);  // (its first barrier comes before any use of them)
}

// A wave takes a token: its logits, kMaxE / 64 to a lane, and top_k times the largest that is left.
template <bool TABLES>
__global__ __launch_bounds__(1024) void select_kernel(const MoeRoute r, const MoeTables t) {
  __shared__ Shared s;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kEach = kMaxE / 64;
  for (int m = wave; m < r.M; m += 16) {
    const double* const row = r.logits + size_t(m) * r.E;
    double v[kEach];
    double top = -__builtin_inf();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = lane + i * 64;
      v[i] = e < r.E ? row[e] : -__builtin_inf();
      top = v[i] > top ? v[i] : top;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const double o = __shfl_xor(top, d);
      top = o > top ? o : top;
    }
    double sum = 0;
    if (!r.sigmoid) {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (lane + i * 64 < r.E) sum += exp(v[i] - top);
#pragma unroll
      for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    }
    uint32_t taken = 0;
    double mine = 0, chosen = 0;  // lane j holds the j-th weight
    int id = 0;
    for (int j = 0; j < r.top_k; ++j) {
      double best = 0;
      int at = kMaxE;  // none yet
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int e = lane + i * 64;
        if (e < r.E && !(taken >> i & 1)) {
          const double key = v[i] == v[i] ? v[i] : -__builtin_inf();
          if (at == kMaxE || key > best) {
            best = key;
            at = e;
          }
        }
      }
#pragma unroll
      for (int d = 32; d; d >>= 1) {
        const double o = __shfl_xor(best, d);
        const int oe = __shfl_xor(at, d);
        if (oe != kMaxE && (at == kMaxE || o > best || (o == best && oe < at))) {
          best = o;
          at = oe;
        }
      }
      // the logit itself (a NaN stays one)
      double logit = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (lane == (at & 63) && i == at / 64) {
          logit = v[i];
          taken |= 1u << i;
        }
      logit = __shfl(logit, at & 63);
      const double w = r.sigmoid ? 1.0 / (1.0 + exp(-logit)) : exp(logit - top) / sum;
      chosen += w;
      if (lane == j) {
        mine = w;
        id = at;
      }
    }
    if (lane < r.top_k) {
      const float w = float(r.renormalize ? mine / chosen : mine);
      const int p = m * r.top_k + lane;
      r.ids[p] = id;
      r.weights[p] = w;
      if constexpr (TABLES) {
        s.ids[p] = id;
        s.weights[p] = w;
      }
    }
  }
  if constexpr (TABLES) make_tables(s, r.M, r.E, r.top_k, t);
}

}  // namespace

hipError_t launch_moe_logits(const MoeRoute& r, hipStream_t st) {
  const dim3 grid(unsigned((r.E + kTile - 1) / kTile), unsigned((r.M + kTile - 1) / kTile));
  if (r.router_f32)
    hipLaunchKernelGGL(logits_kernel<true>, grid, dim3(256), 0, st, r);
  else
    hipLaunchKernelGGL(logits_kernel<false>, grid, dim3(256), 0, st, r);
  return hipGetLastError();
}

hipError_t launch_moe_select(const MoeRoute& r, const MoeTables* t, hipStream_t st) {
  if (t)
    hipLaunchKernelGGL(select_kernel<true>, dim3(1), dim3(1024), 0, st, r, *t);
  else
    hipLaunchKernelGGL(select_kernel<false>, dim3(1), dim3(1024), 0, st, r, MoeTables{});
  return hipGetLastError();
}

hipError_t launch_moe_group(int M, int E, int top_k, const int32_t* ids, const float* weights, const MoeTables& t, hipStream_t st) {
  hipLaunchKernelGGL(group_kernel, dim3(1), dim3(1024), 0, st, M, E, top_k, ids, weights, t);
  return hipGetLastError();
}

}  // namespace paro
