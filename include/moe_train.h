/*
 * moe_train.h - training an expert layer: the router, the bf16 products and the
 * gradients of dispatch, products and combine (libmoe.so).
 *
 * moe.h takes token rows to the experts and back; these calls do the rest of a
 * training step of the same layer, on bf16 rows in the same layout:
 *
 *   forward    moe_router_topk, moe_dispatch_send, moe_expert_linear (gate and
 *              up, then down), moe_combine_send, moe_combine_recv
 *   backward   moe_combine_backward, moe_expert_linear_backward_weight and
 *              _input for either product, moe_dispatch_backward,
 *              moe_router_topk_backward
 *
 * Conventions as in moe.h: device pointers owned by the caller, no device
 * allocation, no host synchronisation, `stream` is a cudaStream_t, argument
 * errors are found on the host (MOE_EINVAL) before anything is enqueued,
 * MOE_ECUDA if a launch fails.  Tensors are row-major and contiguous, and must
 * not overlap unless a call says so.  Products, sums and statistics are held in
 * float32 and rounded once on the way out; the same call gives the same bits
 * each time.  None of these calls needs a moe_ctx, and several may run at once
 * on different streams.
 */
#ifndef MOE_TRAIN_H_
#define MOE_TRAIN_H_

#include <stddef.h>
#include <stdint.h>

#include "moe.h"
#include "moe_ffn.h" /* MOE_TYPE_BF16, MOE_TYPE_F32 */

#ifdef __cplusplus
extern "C" {
#endif

/* How a router's logits become scores. */
#define MOE_SCORE_SOFTMAX 0 /* p = exp(z) / sum over all experts of exp(z) */
#define MOE_SCORE_SIGMOID 1 /* p = 1 / (1 + exp(-z)) */

/* The experts of each token and their weights, in the form that
 * moe_dispatch_send and moe_combine_recv take:
 *   topk_idx[t, :]  the top_k experts with the largest p + bias, the largest
 *                   first, of equal ones the lower index first;
 *   topk_w[t, k]    scale * p[topk_idx[t, k]], with `normalize` divided by the
 *                   sum of p over the token's choices.
 * The choice is that of exact arithmetic: logits are compared as they are
 * without a bias, sums closer than float32 can tell apart in 64 bits with one.
 * A logit of -inf is a score of zero; where all of a token's choices have that,
 * its weights are 0.  Of a token with a NaN or +inf among its logits the weights
 * are undefined, its indices differ and are in range all the same.
 *   logits       device bf16 or float32 (logits_type MOE_TYPE_*) [num_tokens, num_experts]
 *   bias         device float32 [num_experts], finite, or NULL; only with
 *                MOE_SCORE_SIGMOID.  It takes part in the choice alone
 *   num_experts  1..MOE_MAX_EXPERTS;  top_k  1..min(num_experts, MOE_MAX_TOP_K)
 *   scale        finite
 *   topk_idx     device int32 [num_tokens, top_k]
 *   topk_w       device float32 [num_tokens, top_k]
 * Pointers are aligned to their elements.  num_tokens == 0 is allowed. */
int moe_router_topk(const void* logits, int logits_type, const float* bias, int64_t num_tokens, int32_t num_experts,
                    int32_t top_k, int score, int normalize, float scale, int32_t* topk_idx, float* topk_w,
                    void* stream);

/* Gradient of moe_router_topk's weights by the logits, the choice held fixed:
 *   d_logits[t, e] = sum over k of d_topk_w[t, k] * d topk_w[t, k] / d z[t, e]
 * for every expert (zero for those that no weight of the token depends on).
 * logits, num_*, top_k, score, normalize and scale as given to moe_router_topk,
 * topk_idx as it wrote it: an index outside [0, num_experts) is left out.
 *   d_topk_w  device float32 [num_tokens, top_k], e.g. of moe_combine_backward
 *   d_logits  device [num_tokens, num_experts], of the logits' type */
int moe_router_topk_backward(const void* logits, int logits_type, const int32_t* topk_idx, const float* d_topk_w,
                             int64_t num_tokens, int32_t num_experts, int32_t top_k, int score, int normalize,
                             float scale, void* d_logits, void* stream);

/* Gradient of moe_combine_recv:
 *   d_expert_y[slot_row[t, k], :] = bf16( topk_w[t, k] * d_out[t, :] )
 *   d_topk_w[t, k] = sum over h of d_out[t, h] * expert_y[slot_row[t, k], h]
 *   d_out       device bf16 [num_tokens, hidden], hidden % 8 == 0
 *   expert_y    device bf16 [rows, hidden]: what the combine read; NULL exactly
 *               when d_topk_w is
 *   topk_w      device float32 [num_tokens, top_k], top_k 1..MOE_MAX_TOP_K
 *   slot_row    device int32 [num_tokens, top_k], of the dispatch's layout.  A
 *               row outside [0, rows) (after a routing error: -1) is neither
 *               read nor written, its d_topk_w is 0; a row that two
 *               slots name (no dispatch makes that) may hold either's gradient
 *   rows        rows of expert_y and d_expert_y, < 2^31
 *   d_expert_y  device bf16 [rows, hidden], rows that no slot names are left
 *               untouched.  May be expert_y itself
 *   d_topk_w    device float32 [num_tokens, top_k], or NULL
 * d_out, expert_y and d_expert_y are 16-byte aligned.  num_tokens == 0 is allowed. */
int moe_combine_backward(const void* d_out, const void* expert_y, const float* topk_w, const int32_t* slot_row,
                         int64_t num_tokens, int32_t hidden, int32_t top_k, int64_t rows, void* d_expert_y,
                         float* d_topk_w, void* stream);

/* Gradient of moe_dispatch_send:
 *   d_x[t, :] = bf16( sum over k of d_expert_x[slot_row[t, k], :], then + add[t, :] )
 * in float32, k ascending.
 *   d_expert_x  device bf16 [rows, hidden], hidden % 8 == 0
 *   slot_row    device int32 [num_tokens, top_k]; rows outside [0, rows) add nothing
 *   add         device bf16 [num_tokens, hidden]: the gradient of x that came by
 *               other ways (the router, a skip connection), or NULL
 *   d_x         device bf16 [num_tokens, hidden]; may be add itself
 * d_expert_x, add and d_x are 16-byte aligned.  num_tokens == 0 is allowed. */
int moe_dispatch_backward(const void* d_expert_x, const int32_t* slot_row, const void* add, int64_t num_tokens,
                          int32_t hidden, int32_t top_k, int64_t rows, void* d_x, void* stream);

/* Activations of the expert products. */
#define MOE_ACT_NONE 0
#define MOE_ACT_RELU 1
#define MOE_ACT_GELU 2   /* v * (1 + erf(v / sqrt 2)) / 2 */
#define MOE_ACT_SILU 3   /* v / (1 + exp(-v)) */
#define MOE_ACT_SWIGLU 4 /* SiLU(gate) * up: gate is the first half of v, up the second */

/* The experts' product on grouped rows (or one dense product), bf16 operands:
 *   v[i, j]   = sum over c of a[i, c] * w[e, j, c]  + bias[e, j]
 *   out[i, :] = act(v[i, :]) + residual[i, :],   pre[i, :] = bf16(v[i, :])
 * for the rows i in [expert_offsets[e], expert_offsets[e+1]) of expert e.
 *   a               device bf16 [rows, k], k % 8 == 0
 *   w               device bf16 [num_experts, n, k], n % 8 == 0; with
 *                   MOE_ACT_SWIGLU n % 16 == 0: n/2 gate rows, then n/2 up rows
 *   expert_offsets  device int32 [num_experts + 1], non-decreasing; read on the
 *                   device, values outside [0, rows] are taken as the nearest
 *                   inside.  Rows that no expert owns are left untouched.
 *                   NULL (num_experts 1 only): all rows
 *   bias            device [num_experts, n], bf16 or float32 (bias_type), or NULL
 *   activation      MOE_ACT_*
 *   residual        device bf16 [rows, n_out], n_out = n, with MOE_ACT_SWIGLU
 *                   n / 2; or NULL.  May be out itself if out is bf16
 *   pre             device bf16 [rows, n], or NULL: what the gradient through
 *                   the activation needs
 *   out             device bf16 or float32 (out_type) [rows, n_out]
 *   status          device int32 [1], or NULL; set to MOE_ETIMEDOUT from MOE_OK
 *                   if a bounded wait inside the kernel gives up (the outputs
 *                   are then incomplete), otherwise not touched
 * a, w, bias, residual, pre and out are 16-byte aligned.  rows == 0 is allowed;
 * rows < 2^31 - 256, n and k <= 2^30, num_experts <= MOE_MAX_EXPERTS. */
int moe_expert_linear(const void* a, int64_t rows, int32_t k, const void* w, int32_t n, int32_t num_experts,
                      const int32_t* expert_offsets, const void* bias, int bias_type, int activation,
                      const void* residual, void* pre, void* out, int out_type, int32_t* status, void* stream);

/* Gradient of a product by its rows, and on through the activation that made
 * those rows (activation and pre are the earlier product's, the one that wrote
 * this product's rows):
 *   g[i, c]  = sum over j of dy[i, j] * w[e, j, c]
 *   dx[i, :] = bf16( g[i, :] * act'(pre[i, :]) );   MOE_ACT_NONE: bf16(g)
 *   MOE_ACT_SWIGLU: dx [rows, 2k] = (g * up * SiLU'(gate), g * SiLU(gate))
 *   dy    device bf16 [rows, n], n % 8 == 0
 *   w     device bf16 [num_experts, n, k], k % 8 == 0
 *   pre   device bf16 [rows, k], MOE_ACT_SWIGLU [rows, 2k]; NULL exactly with
 *         MOE_ACT_NONE
 *   dx    device bf16 [rows, k], MOE_ACT_SWIGLU [rows, 2k]; may be pre itself
 * The derivative of RELU at 0 is 0.  Everything else as for moe_expert_linear. */
int moe_expert_linear_backward_input(const void* dy, int64_t rows, int32_t n, const void* w, int32_t k,
                                     int32_t num_experts, const int32_t* expert_offsets, int activation,
                                     const void* pre, void* dx, int32_t* status, void* stream);

/* Gradient of a product by its weights and its bias:
 *   dw[e, j, c] = sum over the rows i of expert e of dy[i, j] * a[i, c]
 *   db[e, j]    = sum over the rows i of expert e of dy[i, j]
 * (0 for an expert without rows), or, with `accumulate`, added to what dw and db
 * hold: in float32, rounded once.
 *   dy   device bf16 [rows, n], n % 8 == 0: the gradient of v, after an
 *        activation that is moe_expert_linear_backward_input's output
 *   a    device bf16 [rows, k], k % 8 == 0
 *   dw   device bf16 or float32 (dw_type) [num_experts, n, k]
 *   db   device float32 [num_experts, n], or NULL
 * dy, a, dw and db are 16-byte aligned.  rows == 0 is allowed (dw and db are
 * then zeroed, or with `accumulate` left).  Everything else as for
 * moe_expert_linear. */
int moe_expert_linear_backward_weight(const void* dy, int64_t rows, int32_t n, const void* a, int32_t k,
                                      int32_t num_experts, const int32_t* expert_offsets, void* dw, int dw_type,
                                      float* db, int accumulate, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H_ */
