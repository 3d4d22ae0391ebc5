// Which tokens go to which experts, made by one workgroup from masks of the experts' tokens, in three steps with a
// barrier of all its threads before each.
#pragma once

#include "moe_internal.h"

namespace paro {

struct TableWork {
  unsigned long long mask[PARO_MOE_MAX_E];  // an expert's tokens
  int first[PARO_MOE_MAX_E];                // its first slot
  uint32_t totals[PARO_MOE_MAX_E / 64];     // of 64 experts each: slots, and units in the upper half
};

// Threads 0..511, one for each expert: what it and those before it in its 64 have.
struct TablePlace {
  int count;
  uint32_t before;  // slots, and units in the upper half
};
template <int CTRL, int ROWS>
__device__ inline uint32_t up(uint32_t v) {  // what a data-parallel move brings, 0 to lanes without a source
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false));
}
__device__ inline TablePlace tables_count(TableWork& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  TablePlace p;
  p.count = int(__popcll(s.mask[tid]));
  const uint32_t own = uint32_t(p.count) | uint32_t((p.count + 15) / 16) << 16;
  uint32_t sum = own;
  sum += up<0x111, 0xF>(sum);  // row_shr:1, 2, 4, 8: sums up to the lane within its row of 16
  sum += up<0x112, 0xF>(sum);
  sum += up<0x114, 0xF>(sum);
  sum += up<0x118, 0xF>(sum);
  sum += up<0x142, 0xA>(sum);  // row_bcast:15 into rows 1 and 3
  sum += up<0x143, 0xC>(sum);  // row_bcast:31 into rows 2 and 3
  if (lane == 63) s.totals[wave] = sum;
  p.before = sum - own;
  return p;
}
// The same threads: units, and the experts' first slots.
__device__ inline void tables_units(TableWork& s, const TablePlace& p, const MoeTables& t) {
  const int tid = threadIdx.x, wave = tid >> 6;
  uint32_t before = p.before, all = 0;
#pragma unroll
  for (int w = 0; w < PARO_MOE_MAX_E / 64; ++w) {
    if (w < wave) before += s.totals[w];
    all += s.totals[w];
  }
  const int slot = int(before & 0xFFFFu);
  int unit = int(before >> 16);
  s.first[tid] = slot;
  for (int f = 0; f < p.count; f += 16) t.unit[unit++] = MoeUnit{tid, slot + f, min(16, p.count - f)};
  if (tid == 0) *t.units = int(all >> 16);
}
// All threads: the slots.
__device__ inline void tables_slots(const TableWork& s, int M, int E, int top_k, const int* ids, const float* weights, const MoeTables& t) {
  for (int p = threadIdx.x; p < M * top_k; p += blockDim.x) {
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
