// Argument checks of the calls in paro_w8a8.h and paro_block.h.
#pragma once

#include "paro_block.h"
#include "paro_internal.h"

namespace paro {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  const void* p;
  size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
// Every output apart from every input and every other output.
template <size_t NO, size_t NI>
bool any_overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (size_t o = 0; o < NO; ++o) {
    for (size_t i = 0; i < NI; ++i)
      if (overlap(outs[o], ins[i])) return true;
    for (size_t k = o + 1; k < NO; ++k)
      if (overlap(outs[o], outs[k])) return true;
  }
  return false;
}

inline bool good_ptr(const void* p) { return p && aligned16(p); }
inline bool good_D(int D) { return D >= PARO_GROUP && D <= PARO_MAX_D && D % PARO_GROUP == 0; }
inline bool row_dtype(int t) { return t == PARO_F16 || t == PARO_BF16; }
inline bool out_dtype(int t) { return row_dtype(t) || t == PARO_F32; }
inline size_t dtype_bytes(int t) { return t == PARO_F32 ? 4 : 2; }
inline paro_status from_hip(hipError_t e) { return e == hipSuccess ? PARO_OK : PARO_EHIP; }
inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// The transform of a call (r may be NULL); *out is filled either way.
inline paro_status check_rot(const paro_rotation* r, int D, DevRot* out, Span* desc) {
  *out = DevRot{0, D, nullptr, nullptr, nullptr};
  *desc = Span{nullptr, 0};
  if (!r) return PARO_OK;
  if (r->D != D || r->K < 0 || r->K > PARO_MAX_K) return PARO_ESHAPE;
  if (!good_ptr(r->dev)) return PARO_EINVAL;
  *out = dev_rot(*r);
  *desc = Span{r->dev, desc_layout(r->K, r->D).total};
  return PARO_OK;
}

}  // namespace paro
