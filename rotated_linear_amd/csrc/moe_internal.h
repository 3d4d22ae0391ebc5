// Internal declarations of the mixture-of-experts calls (include/paro_block.h).
#pragma once

#include "paro_block.h"
#include "paro_internal.h"

namespace paro {

// Which tokens go to which experts. Slots are the (expert, token) pairs in the order of the experts, then the tokens;
// a token that names an expert twice has one slot with both weights. A unit is up to 16 slots of one expert.
struct MoeUnit {
  int expert, first, count;  // its slots are first .. first + count - 1
};
struct MoeSlot {
  uint16_t pair, token;  // the first (token, choice) pair, whose row of a the slot has
  float weight;
};
struct MoeTables {
  int* units;  // how many
  MoeUnit* unit;
  MoeSlot* slot;
};
// The rows of a matrix product are 16: a unit of up to 8 tokens has room for both parts of its rows of a, and a call of
// up to 8 tokens has no other units.
constexpr int kTwoParts = 8;
// What is held in two float16 parts (w4_device.h) is held times a power of two, by the token's row of x: x' times
// 2^-power, a times 2^(kLiftA - 2 power), where 2^power is over the row's norm and at most twice it. So neither leaves
// float16's range, whatever the scale of x: where rows of gate and up have norms g and u, |a| <= g u |x|^2, and a is past
// the range from 2^12 |x|^2 on at the earliest; while a typical a, some |x|^2 / (2 D) where g = u = 1, is held as 2^-10
// for D = 1024.
constexpr int kLiftA = 4;
int moe_units_max(int M, int E, int top_k);

struct MoeCall {
  int M, D, F, E, top_k;
  const uint16_t* x;  // [M][D], as the experts see it
  bool x_parts;  // a transform's rows: 8-channel words as [0,4,1,5,2,6,3,7], and [M][D] more, their lower parts
  bool a_fragments;     // a is float16 in the order of fragments; else, with a transform behind it, float32 as it is, and
                        // a_down float16 in the nibble order. Behind float16 rows [M top_k][F] of a as many more,
                        // their lower parts
  const uint8_t* gu_qw;
  const uint16_t* gu_sc;
  const uint16_t* gu_zr;
  const uint8_t* dn_qw;
  const uint16_t* dn_sc;
  const uint16_t* dn_zr;
  void* a;                 // [M top_k][F], what the gate and up products make: the rows of the pairs that have an expert
  const uint16_t* a_down;  // the same as the down product sees it
  float* part;             // [splits][M][D], where the down product is split
  MoeTables t;
  const int* power;  // [M], of the tokens' rows
  void* y;
  int ydtype;
};

struct MoeRoute {
  int M, D, E, top_k;
  const uint16_t* x;
  const void* router;
  bool router_f32;
  bool sigmoid, renormalize;
  double* logits;  // [M][E]
  int32_t* ids;
  float* weights;
  int* power;  // [M], of the rows of x; nullptr: not wanted
};

hipError_t launch_moe_logits(const MoeRoute& r, hipStream_t st);
// Ids and weights from the logits, and with t the tables too.
hipError_t launch_moe_select(const MoeRoute& r, const MoeTables* t, hipStream_t st);
// The tables from given ids and weights, and where x is not nullptr the rows' powers.
hipError_t launch_moe_group(int M, int D, int E, int top_k, const uint16_t* x, const int32_t* ids, const float* weights, const MoeTables& t,
                            int* power, hipStream_t st);
struct MoeGateUpPlan {
  int waves, groups;  // of a workgroup, and of a wave (0: any number)
  bool once;          // weights past the caches
};
MoeGateUpPlan moe_gate_up_plan(int M, int D, int F, int E, int top_k, int parts);  // parts: of x'
hipError_t launch_moe_gate_up(const MoeCall& c, hipStream_t st);
struct MoeDownPlan {
  int tiles, splits;  // 16-column tiles of a workgroup, and the workgroups that share them
  bool few;           // no unit has more than kTwoParts tokens
  bool once;          // weights past the caches
};
MoeDownPlan moe_down_plan(int M, int D, int F, int E, int top_k);
hipError_t launch_moe_down(const MoeCall& c, hipStream_t st);

}  // namespace paro

// For tests, and in no header of the library: the kernel of a call's gate and up product, and how its down product is cut.
extern "C" void paro_internal_moe_gate_up_plan(int M, int D, int F, int E, int top_k, int parts, int* waves, int* groups, int* once);
extern "C" void paro_internal_moe_down_plan(int M, int D, int F, int E, int top_k, int* tiles, int* splits);
extern "C" void paro_internal_moe_down_kernel(int M, int D, int F, int E, int top_k, int* tiles, int* few, int* once);
