// Which tokens go to which experts, made by one workgroup from the ids.
#pragma once

#include "moe_internal.h"

namespace paro {

struct TableWork {
  unsigned long long mask[PARO_MOE_MAX_E];  // an expert's tokens
  int first[PARO_MOE_MAX_E];                // its first slot
  int slots[8], units[8];                   // of 64 experts each
};

// All threads of the workgroup (512 at least); ids and weights [M][top_k] in LDS.
__device__ inline void make_tables(TableWork& s, int M, int E, int top_k, const int* ids, const float* weights, const MoeTables& t) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, wave = tid >> 6, pairs = M * top_k;
  __syncthreads();
  if (tid < PARO_MOE_MAX_E) s.mask[tid] = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += nt)
    if (uint32_t(ids[p]) < uint32_t(E)) atomicOr(&s.mask[ids[p]], 1ull << (p / top_k));  // (in any order the same)
  __syncthreads();
  int n = 0, slot = 0, unit = 0;  // of the thread's expert, then what lies before it in its 64
  if (tid < PARO_MOE_MAX_E) {
    n = int(__popcll(s.mask[tid]));
    slot = n;
    unit = (n + 15) / 16;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int a = __shfl_up(slot, d), b = __shfl_up(unit, d);
      if (lane >= d) {
        slot += a;
        unit += b;
      }
    }
    if (lane == 63) {
      s.slots[wave] = slot;
      s.units[wave] = unit;
    }
    slot -= n;
    unit -= (n + 15) / 16;
  }
  __syncthreads();
  if (tid < PARO_MOE_MAX_E) {
    int all = unit;
    for (int w = 0; w < PARO_MOE_MAX_E / 64; ++w) {
      if (w < wave) {
        slot += s.slots[w];
        unit += s.units[w];
      }
      all = w == 0 ? s.units[0] : all + s.units[w];
    }
    s.first[tid] = slot;
    for (int f = 0; f < n; f += 16) t.unit[unit++] = MoeUnit{tid, slot + f, min(16, n - f)};
    if (tid == 0) *t.units = all;
  }
  __syncthreads();
  for (int p = tid; p < pairs; p += nt) {
    const int e = ids[p], m = p / top_k;
    if (uint32_t(e) >= uint32_t(E)) continue;
    float w = 0;
    bool again = false;
    for (int q = m * top_k; q < (m + 1) * top_k; ++q)  // an expert named twice counts twice
      if (ids[q] == e) {
        again |= q < p;
        w += weights[q];
      }
    if (again) continue;
    const int at = s.first[e] + int(__popcll(s.mask[e] & ((1ull << m) - 1)));
    t.slot[at] = MoeSlot{uint16_t(p), uint16_t(m), w};
  }
}

}  // namespace paro
