// Internal declarations of the mixture-of-experts calls (include/paro_block.h).
#pragma once

#include "paro_block.h"
#include "paro_internal.h"

namespace paro {

// Which tokens go to which experts, made on the GPU from the ids. Slots are the (expert, token) pairs in the order
// of experts, then tokens; a token that names an expert twice has one slot with both weights.
struct MoeActive {
  int expert, first, count;  // its slots are first .. first + count - 1
};
struct MoeTables {
  int* active_count;
  MoeActive* active;   // the experts that have tokens, in their order
  int* slot_token;     // [slots]
  float* slot_weight;  // [slots]
};

struct MoeCall {
  int M, D, F, E, top_k;
  const uint16_t* x;  // [M][D], as the experts see it
  const uint8_t* gu_qw;
  const uint16_t* gu_sc;
  const uint16_t* gu_zr;
  const uint8_t* dn_qw;
  const uint16_t* dn_sc;
  const uint16_t* dn_zr;
  uint16_t* a;             // [slots][F], what the gate and up products make
  const uint16_t* a_down;  // the same as the down product sees it
  void* y;
  int ydtype;
  MoeTables t;
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
};

hipError_t launch_moe_logits(const MoeRoute& r, hipStream_t st);
// Ids and weights from the logits, and with t the tables too.
hipError_t launch_moe_select(const MoeRoute& r, const MoeTables* t, hipStream_t st);
// The tables from given ids and weights.
hipError_t launch_moe_group(int M, int E, int top_k, const int32_t* ids, const float* weights, const MoeTables& t, hipStream_t st);
hipError_t launch_moe_gate_up(const MoeCall& c, hipStream_t st);
hipError_t launch_moe_down(const MoeCall& c, hipStream_t st);

}  // namespace paro
