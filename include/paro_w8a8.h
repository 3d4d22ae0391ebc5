/*
 * paro_w8a8.h -- C ABI of libparo's 8-bit path on MI355X (gfx950): activations and weights as
 * 8-bit integers with one scale per token and one per output channel (W8A8), next to the W4A16
 * path of paro.h, whose transform (paro_rotation), status codes and conventions it shares.
 *
 * What an 8-bit linear layer is here: the rows of x (after the channel-pair rotations of paro.h,
 * which spread the outlier channels that make 8-bit activations inaccurate, or as they are) and
 * the rows of W each become integers -127..127 times one float32 scale, and
 *     y[m][n] = xs[m] * ws[n] * sum_k xq[m][k] * wq[n][k]
 * with the sum exact in 32-bit integers (at most PARO_MAX_D * 128 * 128 = 2^28).
 *
 * Conventions, beside those of paro.h (caller owns every buffer, asynchronous on `stream`, every
 * argument checked on the host before anything is enqueued, 16-byte aligned device pointers, no
 * output overlapping another operand)
 *   - Shapes: rows of D channels, D % 128 == 0, 128 <= D <= PARO_MAX_D (PARO_ESHAPE), every array
 *     row-major and contiguous. M, N, F >= 0; a zero size enqueues nothing and succeeds. Rows
 *     past M (N, F) are neither read nor written.
 *   - Types: `dtype` is PARO_F16 or PARO_BF16 for rows that are read; outputs of the linears and
 *     of paro_dequantize_q8 may be PARO_F32 too. Codes are int8, scales float32.
 *   - Row quantiser (every call that writes q and scales): with a = the largest |v| of the row
 *     and c = max(a, 2^-100): scale = c / 127 and code = rint(v * 127 / c), ties to even, so a
 *     zero row has codes 0 and a positive scale. Arithmetic is float32 (float64 where stated)
 *     except for rounding of the result. A row with an infinity or a NaN has scale NaN and codes
 *     0, so everything computed from that row, and nothing else, is NaN.
 *   - Forward only: these are the calls of a served model, and none has a backward pass.
 *   - Results do not depend on the other rows of a call, on the workspace or on its previous
 *     contents, and are the same bits every time.
 */
#ifndef PARO_W8A8_H
#define PARO_W8A8_H

#include "paro.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Third element type, beside PARO_F16 and PARO_F32 of paro_dtype; taken by the calls below only. */
#define PARO_BF16 2

/*
 * paro_rmsnorm_q8 -- residual addition, root-mean-square norm and row quantiser in one pass:
 *     h = dtype(x + residual)         (h = x with residual == NULL)
 *     n = (h * gamma) / sqrt(mean(h^2) + eps)
 *     residual_out = h;  (q, scales) = the row quantiser on n
 * x, residual, residual_out dtype [M][D], gamma dtype [D]; q int8 [M][D], scales float32 [M]. The
 * addition is float32 rounded once; the norm is that of the rounded h, the row that the next
 * layers see. The mean of squares is float64 (no overflow for bfloat16 rows), 1 / sqrt rounded
 * once to float32; bfloat16 rows where h * gamma or 1 / sqrt leave float32's range, though n may not,
 * have n in float64, rounded once. eps must be finite and at least 2^-126. residual and residual_out go together
 * (both or neither NULL, else PARO_EINVAL) and may be the same pointer: the stream is then updated
 * in place. x may not be residual_out.
 */
paro_status paro_rmsnorm_q8(int M, int D, int dtype, const void* x, const void* residual, const void* gamma,
                            float eps, void* residual_out, int8_t* q, float* scales, void* stream);

/*
 * paro_rmsnorm -- the same norm with y = dtype(n) [M][D] as its output: rows for paro_quantize_q8
 * behind a transform, and, in float16 only, for paro_rotate and the W4A16 linears. Arguments as in
 * paro_rmsnorm_q8.
 */
paro_status paro_rmsnorm(int M, int D, int dtype, const void* x, const void* residual, const void* gamma, float eps,
                         void* residual_out, void* y, void* stream);

/*
 * paro_quantize_q8 -- rows of x in 8 bits: the row quantiser on v = x (r == NULL), or on
 * v = G_K ... G_1 x / s, the activation-side transform of paro_rotate in float32 with no rounding
 * to 16 bits in between (then D must equal r->D, else PARO_ESHAPE). x dtype [M][D]; q int8 [M][D],
 * scales float32 [M].
 */
paro_status paro_quantize_q8(const paro_rotation* r, int M, int D, int dtype, const void* x, int8_t* q, float* scales,
                             void* stream);

/* paro_dequantize_q8 -- reads rows back: x[m][k] = dtype(q[m][k] * scales[m]), rounded once;
 * dtype PARO_F16, PARO_BF16 or PARO_F32. */
paro_status paro_dequantize_q8(int M, int D, const int8_t* q, const float* scales, void* x, int dtype, void* stream);

/*
 * paro_pack_weights_q8 -- build-time weights in 8 bits: the row quantiser in float64 on each row of
 * W (r == NULL), or on the row with the transform folded in (the K stages of r, then times s, as
 * paro_pack_weights folds it), so that transform(x) . W'^T = x . W^T. Every product and sum of
 * the fold is float64 with no fused multiply-add, v * 127 / c is held to twice that precision, and scale
 * is rounded once to float32 (past its range, which no s of ordinary size takes a row to, an infinity). W dtype [N][D]; qweight int8 [N][D] row-major (row n is weight row n),
 * scales float32 [N].
 */
paro_status paro_pack_weights_q8(const paro_rotation* r, int N, int D, int dtype, const void* W, int8_t* qweight,
                                 float* scales, void* stream);

/* Workspace bytes that paro_w8a8_linear needs at (M, D, N): room for the 32-bit partial sums of a
 * reduction that is split to fill the GPU; 0 for calls that do not split and for bad sizes. */
size_t paro_w8a8_workspace_bytes(int M, int D, int N);

/*
 * paro_w8a8_linear -- y[m][n] = (sum_k x[m][k] * qweight[n][k]) * xscales[m] * wscales[n]: the
 * integer sum is exact, then float32, rounded once to ydtype (PARO_F16, PARO_BF16 or PARO_F32).
 * x int8 [M][D], xscales float32 [M], qweight int8 [N][D], wscales float32 [N], y [M][N]. ws holds
 * at least paro_w8a8_workspace_bytes(M, D, N) bytes (else PARO_EWORKSPACE; NULL where that is 0)
 * and overlaps no operand. Two calls that may run at the same time need two workspaces. M and N are
 * at most 2^31 - 512 (PARO_EINVAL). The products are taken in the order written: a sum times xscales[m]
 * that passes float32 is an infinity, whatever wscales[n].
 */
paro_status paro_w8a8_linear(int M, int D, int N, const int8_t* x, const float* xscales, const int8_t* qweight,
                             const float* wscales, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream);

/* Workspace bytes that paro_w8a8_gated_linear needs at (M, D, F). */
size_t paro_w8a8_gated_workspace_bytes(int M, int D, int F);

/*
 * paro_w8a8_gated_linear -- both projections of a gated feed-forward block, the activation and the
 * product in one: with g and u the linears of qweight's first and last F rows,
 *     y[m][f] = silu(g[m][f]) * u[m][f],  silu(g) = g / (1 + exp(-g))
 * in float32, rounded once to ydtype. A float32 y has the activation to float32's last digits; a
 * 16-bit y to its own, and where 1 / (1 + exp(-g)) is under 2^-126 (g below -87.3) that may count as
 * 0. qweight int8 [2F][D] (gate rows 0..F-1, then up rows; F below 2^29), wscales float32 [2F], y
 * [M][F]; the rest as in paro_w8a8_linear.
 */
paro_status paro_w8a8_gated_linear(int M, int D, int F, const int8_t* x, const float* xscales, const int8_t* qweight,
                                   const float* wscales, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PARO_W8A8_H */
