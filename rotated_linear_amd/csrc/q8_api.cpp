// Host side of the 8-bit path (include/paro_w8a8.h): argument checks and dispatch. Every error
// path returns before anything is enqueued on the stream.
#include <limits.h>
#include <math.h>

#include "q8_internal.h"

using namespace paro;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
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

// The byte offsets of a gated call's 2 F scales stay below 2^32.
constexpr int kMaxGatedF = (1 << 29) - 1;
// Rows of x and of y's columns: rounded up to a tile they still are ints.
constexpr int kMaxProductRows = INT_MAX - 511;
bool good_rows(int M, int N, bool gated) {
  return M >= 0 && N >= 0 && M <= kMaxProductRows && N <= (gated ? kMaxGatedF : kMaxProductRows);
}

bool good_ptr(const void* p) { return p && aligned16(p); }
bool good_D(int D) { return D >= PARO_GROUP && D <= PARO_MAX_D && D % PARO_GROUP == 0; }
bool row_dtype(int t) { return t == PARO_F16 || t == PARO_BF16; }
bool out_dtype(int t) { return row_dtype(t) || t == PARO_F32; }
size_t dtype_bytes(int t) { return t == PARO_F32 ? 4 : 2; }
paro_status from_hip(hipError_t e) { return e == hipSuccess ? PARO_OK : PARO_EHIP; }
hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

// The kernel of an 8-bit product: a function of its shape only.
enum class Kernel { kStream, kColumn, kTiled };
struct Plan {
  Kernel kernel;
  GemmPlanQ8 tiled;
};
Plan plan(int M, int D, int N, bool gated) {
  if (w8a8_stream_takes(M, N)) return Plan{Kernel::kStream, {}};
  const GemmPlanQ8 t = plan_gemm_w8a8(M, D, N, gated);
  return w8a8_column_us(M, D, N, gated) <= t.us ? Plan{Kernel::kColumn, {}} : Plan{Kernel::kTiled, t};
}

// The transform of a call (r may be NULL); *out is filled either way.
paro_status check_rot(const paro_rotation* r, int D, DevRot* out, Span* desc) {
  *out = DevRot{0, D, nullptr, nullptr, nullptr};
  *desc = Span{nullptr, 0};
  if (!r) return PARO_OK;
  if (r->D != D || r->K < 0 || r->K > PARO_MAX_K) return PARO_ESHAPE;
  if (!good_ptr(r->dev)) return PARO_EINVAL;
  *out = dev_rot(*r);
  *desc = Span{r->dev, desc_layout(r->K, r->D).total};
  return PARO_OK;
}

paro_status norm(int M, int D, int dtype, const void* x, const void* residual, const void* gamma, float eps,
                 void* residual_out, void* y, bool q8, int8_t* q, float* scales, void* stream) {
  if (M < 0 || !row_dtype(dtype)) return PARO_EINVAL;
  if (!(eps >= 0x1p-126f) || !isfinite(eps)) return PARO_EINVAL;
  if (!good_D(D)) return PARO_ESHAPE;
  if (M == 0) return PARO_OK;
  if (!good_ptr(x) || !good_ptr(gamma) || (residual == nullptr) != (residual_out == nullptr)) return PARO_EINVAL;
  if (!aligned16(residual) || !aligned16(residual_out)) return PARO_EINVAL;
  if (q8 ? !good_ptr(q) || !good_ptr(scales) : !good_ptr(y)) return PARO_EINVAL;
  const size_t n = size_t(M) * D;
  // residual and residual_out may be the same rows (each row is read before it is written), not shifted ones
  const Span outs[] = {{residual_out, 2 * n}, {y, 2 * n}, {q, n}, {scales, size_t(M) * 4}};
  const Span ins[] = {{x, 2 * n}, {gamma, size_t(D) * 2}, {residual_out == residual ? nullptr : residual, 2 * n}};
  if (any_overlap(outs, ins)) return PARO_EINVAL;
  return from_hip(launch_rmsnorm(NormArgs{M, D, dtype, x, residual, gamma, eps, residual_out, y, q, scales},
                                 as_stream(stream)));
}

// forced: the plan to take instead of the shape's own, or nullptr.
paro_status linear(const Plan* forced, int M, int D, int N, bool gated, const int8_t* x, const float* xs, const int8_t* w, const float* wsc,
                   void* y, int ydtype, void* ws, size_t ws_bytes, void* stream) {
  if (!good_rows(M, N, gated) || !out_dtype(ydtype)) return PARO_EINVAL;
  if (!good_D(D)) return PARO_ESHAPE;
  if (M == 0 || N == 0) return PARO_OK;
  if (!good_ptr(x) || !good_ptr(xs) || !good_ptr(w) || !good_ptr(wsc) || !good_ptr(y)) return PARO_EINVAL;
  const size_t rows = size_t(N) * (gated ? 2 : 1);
  const Plan p = forced ? *forced : plan(M, D, N, gated);
  const size_t need = p.tiled.part_bytes;
  if (need && (!ws || ws_bytes < need)) return PARO_EWORKSPACE;
  if (need && !aligned16(ws)) return PARO_EINVAL;
  const Span outs[] = {{y, size_t(M) * N * dtype_bytes(ydtype)}, {need ? ws : nullptr, need}};
  const Span ins[] = {{x, size_t(M) * D}, {xs, size_t(M) * 4}, {w, rows * D}, {wsc, rows * 4}};
  if (any_overlap(outs, ins)) return PARO_EINVAL;
  const W8A8Call c{M, D, N, gated, x, xs, w, wsc, y, ydtype};
  const hipStream_t st = as_stream(stream);
  return from_hip(p.kernel == Kernel::kStream   ? launch_w8a8_stream(c, st)
                  : p.kernel == Kernel::kColumn ? launch_w8a8_column(c, st)
                                                : launch_w8a8_gemm(c, p.tiled, static_cast<int*>(ws), st));
}

}  // namespace

extern "C" {

paro_status paro_rmsnorm_q8(int M, int D, int dtype, const void* x, const void* residual, const void* gamma, float eps,
                            void* residual_out, int8_t* q, float* scales, void* stream) {
  return norm(M, D, dtype, x, residual, gamma, eps, residual_out, nullptr, true, q, scales, stream);
}

paro_status paro_rmsnorm(int M, int D, int dtype, const void* x, const void* residual, const void* gamma, float eps,
                         void* residual_out, void* y, void* stream) {
  return norm(M, D, dtype, x, residual, gamma, eps, residual_out, y, false, nullptr, nullptr, stream);
}

paro_status paro_quantize_q8(const paro_rotation* r, int M, int D, int dtype, const void* x, int8_t* q, float* scales,
                             void* stream) {
  if (M < 0 || !row_dtype(dtype)) return PARO_EINVAL;
  if (!good_D(D)) return PARO_ESHAPE;
  DevRot R;
  Span desc;
  if (paro_status e = check_rot(r, D, &R, &desc)) return e;
  if (M == 0) return PARO_OK;
  if (!good_ptr(x) || !good_ptr(q) || !good_ptr(scales)) return PARO_EINVAL;
  const size_t n = size_t(M) * D;
  const Span outs[] = {{q, n}, {scales, size_t(M) * 4}};
  const Span ins[] = {{x, 2 * n}, desc};
  if (any_overlap(outs, ins)) return PARO_EINVAL;
  return from_hip(r ? launch_rotate_q8(R, M, dtype, x, q, scales, as_stream(stream))
                    : launch_quantize_q8(M, D, dtype, x, q, scales, as_stream(stream)));
}

paro_status paro_dequantize_q8(int M, int D, const int8_t* q, const float* scales, void* x, int dtype, void* stream) {
  if (M < 0 || !out_dtype(dtype)) return PARO_EINVAL;
  if (!good_D(D)) return PARO_ESHAPE;
  if (M == 0) return PARO_OK;
  if (!good_ptr(x) || !good_ptr(q) || !good_ptr(scales)) return PARO_EINVAL;
  const size_t n = size_t(M) * D;
  const Span outs[] = {{x, n * dtype_bytes(dtype)}};
  const Span ins[] = {{q, n}, {scales, size_t(M) * 4}};
  if (any_overlap(outs, ins)) return PARO_EINVAL;
  return from_hip(launch_dequantize_q8(M, D, q, scales, x, dtype, as_stream(stream)));
}

paro_status paro_pack_weights_q8(const paro_rotation* r, int N, int D, int dtype, const void* W, int8_t* qweight,
                                 float* scales, void* stream) {
  if (N < 0 || !row_dtype(dtype)) return PARO_EINVAL;
  if (!good_D(D)) return PARO_ESHAPE;
  DevRot R;
  Span desc;
  if (paro_status e = check_rot(r, D, &R, &desc)) return e;
  if (N == 0) return PARO_OK;
  if (!good_ptr(W) || !good_ptr(qweight) || !good_ptr(scales)) return PARO_EINVAL;
  const size_t n = size_t(N) * D;
  const Span outs[] = {{qweight, n}, {scales, size_t(N) * 4}};
  const Span ins[] = {{W, 2 * n}, desc};
  if (any_overlap(outs, ins)) return PARO_EINVAL;
  return from_hip(launch_pack_q8(R, N, dtype, W, qweight, scales, as_stream(stream)));
}

size_t paro_w8a8_workspace_bytes(int M, int D, int N) {
  return M > 0 && N > 0 && good_rows(M, N, false) && good_D(D) ? plan(M, D, N, false).tiled.part_bytes : 0;
}

size_t paro_w8a8_gated_workspace_bytes(int M, int D, int F) {
  return M > 0 && F > 0 && good_rows(M, F, true) && good_D(D) ? plan(M, D, F, true).tiled.part_bytes : 0;
}

paro_status paro_w8a8_linear(int M, int D, int N, const int8_t* x, const float* xscales, const int8_t* qweight,
                             const float* wscales, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream) {
  return linear(nullptr, M, D, N, false, x, xscales, qweight, wscales, y, ydtype, ws, ws_bytes, stream);
}

paro_status paro_w8a8_gated_linear(int M, int D, int F, const int8_t* x, const float* xscales, const int8_t* qweight,
                                   const float* wscales, void* y, int ydtype, void* ws, size_t ws_bytes,
                                   void* stream) {
  return linear(nullptr, M, D, F, true, x, xscales, qweight, wscales, y, ydtype, ws, ws_bytes, stream);
}

void paro_internal_w8a8_plan(int M, int D, int N, int gated, int* kernel, int* tile, int* splits) {
  const Plan p = plan(M, D, N, gated != 0);
  *kernel = int(p.kernel);
  *tile = p.kernel == Kernel::kTiled ? p.tiled.tile : -1;
  *splits = p.kernel == Kernel::kTiled ? p.tiled.splits : 1;
}

int paro_internal_w8a8_tiling(int tile, int* bm, int* bn, int* workgroups) {
  if (tile < 0 || tile >= kTilingsQ8) return 0;
  const TilingQ8 t = tiling_w8a8(tile);
  *bm = t.bm;
  *bn = t.bn;
  *workgroups = t.workgroups;
  return 1;
}

size_t paro_internal_w8a8_tiled_workspace_bytes(int M, int N, int gated, int splits) {
  return part_bytes_w8a8(M, N, gated != 0, splits);
}

paro_status paro_internal_w8a8_tiled(int tile, int splits, int gated, int M, int D, int N, const int8_t* x, const float* xscales,
                                     const int8_t* qweight, const float* wscales, void* y, int ydtype, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (tile < 0 || tile >= kTilingsQ8 || splits < 1 || splits > D / PARO_GROUP) return PARO_EINVAL;
  const Plan p{Kernel::kTiled, {tile, splits, part_bytes_w8a8(M, N, gated != 0, splits), 0}};
  return linear(&p, M, D, N, gated != 0, x, xscales, qweight, wscales, y, ydtype, ws, ws_bytes, stream);
}

}  // extern "C"
