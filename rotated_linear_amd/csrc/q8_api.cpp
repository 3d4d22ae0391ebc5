// Host side of the 8-bit path (include/paro_w8a8.h): argument checks and dispatch. Every error
// path returns before anything is enqueued on the stream.
#include <limits.h>
#include <math.h>

#include "host_checks.h"
#include "q8_internal.h"

using namespace paro;

namespace {

// The byte offsets of a gated call's 2 F scales stay below 2^32.
constexpr int kMaxGatedF = (1 << 29) - 1;
// Rows of x and of y's columns: rounded up to a tile they still are ints.
constexpr int kMaxProductRows = INT_MAX - 511;
bool good_rows(int M, int N, bool gated) {
  return M >= 0 && N >= 0 && M <= kMaxProductRows && N <= (gated ? kMaxGatedF : kMaxProductRows);
}

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
  return from_hip(launch_rmsnorm(NormArgs{M, D, dtype, x, residual, gamma, eps, residual_out, y, q, scales, nullptr, nullptr, 1, 1.0f},
                                 as_stream(stream)));
}

paro_status block_norm(int M, int D, int dtype, const void* x, const void* post_gamma, const void* gate, int gate_rows,
                       const void* residual, float residual_scale, const void* gamma, float eps, void* residual_out, void* y, bool q8,
                       int8_t* q, float* scales, void* stream) {
  if (M < 0 || !row_dtype(dtype) || (gate && gate_rows < 1)) return PARO_EINVAL;
  if (!(eps >= 0x1p-126f) || !isfinite(eps) || !isfinite(residual_scale)) return PARO_EINVAL;
  if (!good_D(D)) return PARO_ESHAPE;
  if (M == 0) return PARO_OK;
  if (!good_ptr(x) || !good_ptr(gamma) || !good_ptr(residual) || !good_ptr(residual_out)) return PARO_EINVAL;
  if (!aligned16(post_gamma) || !aligned16(gate)) return PARO_EINVAL;
  if (q8 ? !good_ptr(q) || !good_ptr(scales) : !good_ptr(y)) return PARO_EINVAL;
  const size_t n = size_t(M) * D, gates = gate ? (size_t(M) + gate_rows - 1) / gate_rows : 0;
  // residual and residual_out may be the same rows (each row is read before it is written), not shifted ones
  const Span outs[] = {{residual_out, 2 * n}, {y, 2 * n}, {q, n}, {scales, size_t(M) * 4}};
  const Span ins[] = {{x, 2 * n}, {gamma, size_t(D) * 2}, {post_gamma, size_t(D) * 2}, {gate, gates * D * 2},
                      {residual_out == residual ? nullptr : residual, 2 * n}};
  if (any_overlap(outs, ins)) return PARO_EINVAL;
  return from_hip(launch_block_norm(NormArgs{M, D, dtype, x, residual, gamma, eps, residual_out, y, q, scales, post_gamma, gate,
                                             uint32_t(gate ? gate_rows : 1), residual_scale},
                                    as_stream(stream)));
}

// What an epilogue adds to a product: any of the three.
struct Epilogue {
  const void* bias;
  int act;
  const void* residual;
};

// forced: the plan to take instead of the shape's own, or nullptr.
paro_status linear(const Plan* forced, int M, int D, int N, bool gated, const int8_t* x, const float* xs, const int8_t* w, const float* wsc,
                   void* y, int ydtype, void* ws, size_t ws_bytes, void* stream, const Epilogue* ep = nullptr) {
  if (ep && (ep->act < PARO_ACT_NONE || ep->act > PARO_ACT_GELU_TANH)) return PARO_EINVAL;
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
  W8A8Call c{M, D, N, gated, x, xs, w, wsc, y, ydtype, false, PARO_ACT_NONE, nullptr, nullptr};
  if (ep) {
    if (!aligned16(ep->bias) || !aligned16(ep->residual)) return PARO_EINVAL;
    // the residual may be y itself (each element is read by the thread that writes it)
    const Span more[] = {{ep->bias, size_t(N) * dtype_bytes(ydtype)}, {ep->residual == y ? nullptr : ep->residual, outs[0].bytes}};
    if (any_overlap(outs, more)) return PARO_EINVAL;
    c.bias = ep->bias;
    c.act = ep->act;
    c.residual = ep->residual;
    c.epilogue = c.bias || c.residual || c.act != PARO_ACT_NONE;
  }
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

paro_status paro_block_norm_q8(int M, int D, int dtype, const void* x, const void* post_gamma, const void* gate, int gate_rows,
                               const void* residual, float residual_scale, const void* gamma, float eps, void* residual_out,
                               int8_t* q, float* scales, void* stream) {
  return block_norm(M, D, dtype, x, post_gamma, gate, gate_rows, residual, residual_scale, gamma, eps, residual_out, nullptr, true, q,
                    scales, stream);
}

paro_status paro_block_norm(int M, int D, int dtype, const void* x, const void* post_gamma, const void* gate, int gate_rows,
                            const void* residual, float residual_scale, const void* gamma, float eps, void* residual_out, void* y,
                            void* stream) {
  return block_norm(M, D, dtype, x, post_gamma, gate, gate_rows, residual, residual_scale, gamma, eps, residual_out, y, false, nullptr,
                    nullptr, stream);
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

paro_status paro_w8a8_linear_epilogue(int M, int D, int N, const int8_t* x, const float* xscales, const int8_t* qweight,
                                      const float* wscales, const void* bias, int activation, const void* residual, void* y,
                                      int ydtype, void* ws, size_t ws_bytes, void* stream) {
  const Epilogue ep{bias, activation, residual};
  return linear(nullptr, M, D, N, false, x, xscales, qweight, wscales, y, ydtype, ws, ws_bytes, stream, &ep);
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

paro_status paro_internal_w8a8_tiled_epilogue(int tile, int splits, int M, int D, int N, const int8_t* x, const float* xscales,
                                              const int8_t* qweight, const float* wscales, const void* bias, int activation,
                                              const void* residual, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream) {
  if (tile < 0 || tile >= kTilingsQ8 || splits < 1 || splits > D / PARO_GROUP) return PARO_EINVAL;
  const Plan p{Kernel::kTiled, {tile, splits, part_bytes_w8a8(M, N, false, splits), 0}};
  const Epilogue ep{bias, activation, residual};
  return linear(&p, M, D, N, false, x, xscales, qweight, wscales, y, ydtype, ws, ws_bytes, stream, &ep);
}

}  // extern "C"
