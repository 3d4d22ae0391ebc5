/*
 * paro_block.h -- C ABI of what surrounds the products of a decoder block on MI355X (gfx950), beside the linears of
 * paro.h (W4A16) and the 8-bit path of paro_w8a8.h, whose status codes, types and conventions it shares:
 *
 *   - the W8A8 product with bias, activation and residual in its epilogue;
 *   - the norms after one block and before the next, with the gate and the residual scale between them;
 *   - a mixture-of-experts layer on INT4 weights for a few tokens, and its router.
 *
 * As there: the caller owns every buffer, every call is asynchronous on `stream` and enqueues kernels only (so it
 * may be captured into a graph), arguments are checked on the host before anything is enqueued, device pointers are
 * 16-byte aligned, no output overlaps another operand (exceptions are named), zero sizes enqueue nothing and
 * succeed, results are the same bits every time and do not depend on a workspace's previous contents, and none of
 * the calls has a backward pass. Two calls that may run at the same time need two workspaces.
 */
#ifndef PARO_BLOCK_H
#define PARO_BLOCK_H

#include "paro_w8a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of paro_w8a8_linear_epilogue, in float32:
 *   RELU max(v, 0), RELU2 max(v, 0)^2, SILU v / (1 + exp(-v)), GELU v (1 + erf(v / sqrt(2))) / 2,
 *   GELU_TANH v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2.
 * A NaN gives a NaN, and so does minus infinity with the last three (it is multiplied by a factor of 0). */
typedef enum {
  PARO_ACT_NONE = 0,
  PARO_ACT_RELU = 1,
  PARO_ACT_RELU2 = 2,
  PARO_ACT_SILU = 3,
  PARO_ACT_GELU = 4,
  PARO_ACT_GELU_TANH = 5
} paro_activation;

/*
 * paro_w8a8_linear_epilogue -- paro_w8a8_linear with
 *     y[m][n] = act(sum * xscales[m] * wscales[n] + bias[n]) + residual[m][n],
 * float32 steps in this order, rounded once to ydtype. bias ydtype [N] or NULL, residual ydtype [M][N] or NULL;
 * activation a paro_activation. residual may be y itself: the stream is then updated in place. A float32 y has its
 * activation to float32's last digits (relative to the activation's argument, whose rounding the exponential of a
 * large one multiplies), a 16-bit y to its own, where a factor of v under 2^-126 may count as 0. The workspace is
 * that of paro_w8a8_linear: paro_w8a8_workspace_bytes(M, D, N). The rest as there.
 */
paro_status paro_w8a8_linear_epilogue(int M, int D, int N, const int8_t* x, const float* xscales, const int8_t* qweight,
                                      const float* wscales, const void* bias, int activation, const void* residual, void* y,
                                      int ydtype, void* ws, size_t ws_bytes, void* stream);

/*
 * paro_block_norm_q8 -- from the output x of one block and the residual stream to the rows of the next, one pass:
 *     p = (x / sqrt(mean(x^2) + eps)) * post_gamma      (p = x with post_gamma == NULL)
 *     h = dtype(residual_scale * residual + gate[m / gate_rows] * p)    (no gate: gate == NULL)
 *     n = (h * gamma) / sqrt(mean(h^2) + eps)
 *     residual_out = h;  (q, scales) = the row quantiser of paro_w8a8.h on n
 * x, residual, residual_out dtype [M][D]; gamma, post_gamma dtype [D]; gate dtype [ceil(M / gate_rows)][D], row m
 * with the gate's row m / gate_rows (gate_rows >= 1: 1 for a gate per row, M or more for one gate, a sequence's length
 * in a padded batch; not read without a gate). residual_scale is finite. The second norm and the quantiser are those of
 * paro_rmsnorm_q8, word for word. Of the first part, each product is float32 in the order written and the sum one fused
 * multiply-add (a plain sum where residual_scale is 1); its mean of squares is float64, and x / sqrt keeps float32's
 * digits over bfloat16's whole range. residual and residual_out may be the same pointer; x may not be residual_out.
 */
paro_status paro_block_norm_q8(int M, int D, int dtype, const void* x, const void* post_gamma, const void* gate, int gate_rows,
                               const void* residual, float residual_scale, const void* gamma, float eps, void* residual_out,
                               int8_t* q, float* scales, void* stream);

/* paro_block_norm -- the same with y = dtype(n) [M][D], as paro_rmsnorm beside paro_rmsnorm_q8. */
paro_status paro_block_norm(int M, int D, int dtype, const void* x, const void* post_gamma, const void* gate, int gate_rows,
                            const void* residual, float residual_scale, const void* gamma, float eps, void* residual_out, void* y,
                            void* stream);

/* Limits of the mixture-of-experts calls (PARO_EINVAL past them): tokens of a call, experts, experts of a token. */
#define PARO_MOE_MAX_M 64
#define PARO_MOE_MAX_E 512
#define PARO_MOE_MAX_K 16

/* How a token's weights come from its router logits. */
typedef enum { PARO_MOE_SOFTMAX = 0, PARO_MOE_SIGMOID = 1 } paro_moe_scoring;

/*
 * paro_moe_route -- the router: for each token the top_k experts with the largest logits x . router^T, the largest
 * first and the lower index first among equals, and their weights: the softmax over all E logits or the logit's
 * sigmoid, with renormalize != 0 divided by their sum over the top_k. Logits are float64 sums of exact products,
 * weights float64 until one rounding. x float16 [M][D]; router float16 or float32 (router_dtype) [E][D]; ids int32
 * [M][top_k]; weights float32 [M][top_k]. 1 <= top_k <= E. A NaN logit ranks as minus infinity does; a row with a NaN
 * logit has NaN weights under softmax, and under sigmoid those of the chosen logits. D as in paro.h. ws holds at least
 * paro_moe_route_workspace_bytes(M, E) bytes (else PARO_EWORKSPACE).
 */
size_t paro_moe_route_workspace_bytes(int M, int E);
paro_status paro_moe_route(int M, int D, int E, int top_k, const void* x, const void* router, int router_dtype, int scoring,
                           int renormalize, int32_t* ids, float* weights, void* ws, size_t ws_bytes, void* stream);

/* INT4 weights of E experts as paro_pack_weights packs E * N rows (N a multiple of 16, so that every expert's blocks
 * are whole): qweight E * N * D/2 bytes, scales and zeros float16 [E * N][D/128]. */
typedef struct {
  const uint8_t* qweight;
  const void* scales;
  const void* zeros;
} paro_w4_experts;

/*
 * paro_moe_w4a16 -- the experts of a few tokens, ids and weights given:
 *     y[m] = sum over j of weights[m][j] * down_e(a),  e = ids[m][j],
 *     a = silu(gate_e x'[m]) * (up_e x'[m]),
 * each product as in paro_w4a16_linear (products of float16 values exact, float32 sums). a is rounded to two float16
 * parts times a power of two by the norm |x[m]| of the token's row. They leave 2^-22 of it, or 2^-38 |x[m]|^2 where that
 * is more; past 2^11 |x[m]|^2, where no a gets if the norms of gate's and up's rows multiply to less than 2^11, it may be
 * an infinity. y is rounded once to ydtype (PARO_F16 or PARO_F32). An id outside 0..E-1 takes no expert (its weight is not
 * read into the sum): a hole in a padded batch, or an expert on another GPU; a token without experts has y = 0. An id that
 * a token names twice counts twice.
 * x float16 [M][D]; ids int32 [M][top_k], weights float32 [M][top_k], 1 <= top_k <= PARO_MOE_MAX_K (with ids given it
 * may pass E); gate_up [E][2 F][D] (gate rows, then up rows), down [E][D][F]. With rot_x (D channels), x' is the
 * transform of x in float32, rounded to two such parts (which leave 2^-22 of it, or 2^-35 |x[m]|; past 2^15 |x[m]| it may
 * be an infinity), else x; with rot_a (F channels), a is the transform of silu(gate) * up, in float32 until its rounding.
 * Both are shared by all experts, whose weights are packed with them. D and F as D in paro.h. A row of x with a NaN or an
 * infinity reaches no other row of y; an expert that no token names is not read. How many tokens share an expert may
 * change the last bits of the float32 sums. ws holds at least paro_moe_workspace_bytes(M, D, F, E, top_k) bytes (else
 * PARO_EWORKSPACE), which are enough with transforms and without.
 */
size_t paro_moe_workspace_bytes(int M, int D, int F, int E, int top_k);
paro_status paro_moe_w4a16(int M, int D, int F, int E, int top_k, const void* x, const int32_t* ids, const float* weights,
                           const paro_rotation* rot_x, const paro_rotation* rot_a, const paro_w4_experts* gate_up,
                           const paro_w4_experts* down, void* y, int ydtype, void* ws, size_t ws_bytes, void* stream);

/* paro_moe_layer_w4a16 -- the whole layer: paro_moe_route on x, then paro_moe_w4a16 with its ids and weights, which
 * the call also writes. The router sees x itself. Workspace as in paro_moe_w4a16. */
paro_status paro_moe_layer_w4a16(int M, int D, int F, int E, int top_k, const void* x, const void* router, int router_dtype,
                                 int scoring, int renormalize, const paro_rotation* rot_x, const paro_rotation* rot_a,
                                 const paro_w4_experts* gate_up, const paro_w4_experts* down, void* y, int ydtype, int32_t* ids,
                                 float* weights, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PARO_BLOCK_H */
