/*
 * moe_ffn.h - the feed-forward operators around dispatch and combine (libmoe.so).
 *
 * A user of moe.h has token rows before the dispatch and expert rows between
 * dispatch and combine.  These calls do that work on the same payload as
 * moe_dispatch_send_fp8 / moe_dispatch_send_quantized: E4M3 codes with one
 * float32 scale for each block of MOE_FP8_BLOCK consecutive elements of a row,
 * weights with one float32 scale for each MOE_FP8_BLOCK x MOE_FP8_BLOCK block.
 *
 *   moe_add_rms_norm_fp8  x + residual -> RMS norm -> codes and scales
 *   moe_expert_glu_fp8    expert rows -> SiLU(gate) * up -> codes and scales
 *   moe_expert_gemm_fp8   expert rows -> one product, bf16 or float32 rows
 *   moe_decode_layer_fp8  a few tokens through dispatch, both products and
 *                         combine at once
 *
 * Quantisation of a block with largest magnitude amax, in float32:
 *   scale = max(amax, 2^-100) / 448 (1 for an all-zero block), inv = 1 / scale,
 *   q = E4M3(v * inv), round to nearest even, saturating.
 * For blocks that hold a bf16 value of at least 2^-100 this is the rule of
 * moe_dispatch_send_fp8; below, the floor keeps 1 / scale finite.  Here v is not
 * a value in memory but the result of a computation, and each call takes v * inv
 * with as few roundings as it can: moe_add_rms_norm_fp8 as (s * weight) * (448 /
 * amax(s * weight)), without the block's common factor.  So a code whose v lies
 * within float32 error of the middle between two codes may be either of them.
 * A row that holds an infinity or a NaN has no defined outputs, nor has a row of
 * moe_add_rms_norm_fp8 whose sum of squares overflows float32, whose mean(s^2) +
 * eps is not a normal float32, or where the largest s * weight of a block is
 * neither zero nor a normal float32; other rows are not touched by it.
 *
 * Conventions as in moe.h: device pointers owned by the caller, no device
 * allocation, no host synchronisation, `stream` is a cudaStream_t, argument
 * errors are found on the host (MOE_EINVAL) before anything is enqueued,
 * MOE_ECUDA if a launch fails.  Tensors are row-major and contiguous, and
 * must not overlap unless a call says so.  None of these calls needs a moe_ctx.
 */
#ifndef MOE_FFN_H_
#define MOE_FFN_H_

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of arguments that may have more than one. */
#define MOE_TYPE_BF16 0
#define MOE_TYPE_F32 1

/* Largest row of moe_add_rms_norm_fp8. */
#define MOE_NORM_MAX_HIDDEN 65536

/* Residual addition, root-mean-square norm and quantisation of token rows:
 *   s = x + residual (float32; s = x without a residual)
 *   v = s / sqrt(mean(s^2) + eps) * weight, float32
 *   residual_out = bf16(s), y = bf16(v), (xq, x_scales) = v quantised
 * The norm and the codes are taken from the float32 s and v, not from their
 * roundings to bf16.  xq and x_scales are what moe_dispatch_send_quantized
 * takes (it needs hidden % 512 == 0); y is what a router reads.
 *   x             device bf16 [num_tokens, hidden], hidden % MOE_FP8_BLOCK == 0
 *   residual      device bf16 [num_tokens, hidden], or NULL
 *   weight        device [hidden], bf16 or float32 (weight_type MOE_TYPE_*)
 *   eps           finite, > 0
 *   residual_out  device bf16 [num_tokens, hidden]; NULL exactly when residual
 *                 is.  May be x or residual itself (updated in place).
 *   y             device bf16 [num_tokens, hidden], or NULL; may be x itself
 *                 unless residual_out is
 *   xq            device E4M3 bytes [num_tokens, hidden]
 *   x_scales      device float32 [num_tokens, hidden / MOE_FP8_BLOCK]
 * All but x_scales (4 bytes) are 16-byte aligned.  num_tokens == 0 is allowed. */
int moe_add_rms_norm_fp8(const void* x, const void* residual, const void* weight, int weight_type,
                         int64_t num_tokens, int32_t hidden, float eps, void* residual_out, void* y, void* xq,
                         float* x_scales, void* stream);

/* The experts' product on grouped rows (or one dense product):
 *   out[i, j] = sum over blocks b of k:  a_scales[i, b] * w_scales[e, j / 128, b]
 *               * sum over c in block b of  a[i, c] * w[e, j, c]
 * for the rows i in [expert_offsets[e], expert_offsets[e+1]) of expert e,
 * accumulated in float32 and rounded once.  With expert_offsets of
 * moe_dispatch_recv this turns dispatched rows into the expert_y that
 * moe_combine_send takes.
 *   a               device E4M3 [rows, k], k % 16 == 0, k <= 2^31 - 128
 *   a_scales        device float32 [rows, ceil(k / 128)]
 *   w               device E4M3 [num_experts, n, k], n % 8 == 0,
 *                   num_experts * n <= 2^31 - 256
 *   w_scales        device float32 [num_experts, ceil(n / 128), ceil(k / 128)]
 *   expert_offsets  device int32 [num_experts + 1], non-decreasing; read on the
 *                   device, values outside [0, rows] are taken as the nearest
 *                   inside.  Rows that no expert owns are left untouched.
 *                   NULL (num_experts 1 only): all rows.
 *   out             device bf16 or float32 (out_type MOE_TYPE_*) [rows, n]
 *   status          device int32 [1], or NULL; set to MOE_ETIMEDOUT from MOE_OK
 *                   if a bounded wait inside the kernel gives up (the outputs
 *                   are then incomplete), otherwise not touched.  The only
 *                   sign of it: with NULL nothing tells
 * a, w and out are 16-byte aligned.  rows == 0 is allowed; rows < 2^31 - 128. */
int moe_expert_gemm_fp8(const void* a, const float* a_scales, int64_t rows, int32_t k, const void* w,
                        const float* w_scales, int32_t n, int32_t num_experts, const int32_t* expert_offsets,
                        void* out, int out_type, int32_t* status, void* stream);

/* The experts' gated product with its activation and quantisation:
 *   gate = a . w13[e, 0..inter), up = a . w13[e, inter..2 inter), each as in
 *   moe_expert_gemm_fp8, left in float32;
 *   h = gate / (1 + exp(-gate)) * up;  (hq, h_scales) = h quantised,
 * which is what moe_expert_gemm_fp8 takes for the second product.  For gates
 * below about -87.3, where 1 + exp(-gate) passes 2^126, h is 0 (its size is less
 * than 2^-119 of up).
 *   a, a_scales     device E4M3 [rows, hidden] and its scales, hidden % 16 == 0,
 *                   hidden <= 2^31 - 128
 *   w13             device E4M3 [num_experts, 2 * inter, hidden]: gate rows,
 *                   then up rows; inter % 128 == 0, num_experts * 2 * inter <= 2^31 - 256
 *   w13_scales      device float32 [num_experts, 2 * inter / 128, ceil(hidden / 128)]
 *   hq, h_scales    device E4M3 [rows, inter], float32 [rows, inter / 128]
 * Everything else as for moe_expert_gemm_fp8. */
int moe_expert_glu_fp8(const void* a, const float* a_scales, int64_t rows, int32_t hidden, const void* w13,
                       const float* w13_scales, int32_t inter, int32_t num_experts, const int32_t* expert_offsets,
                       void* hq, float* h_scales, int32_t* status, void* stream);

/* Largest number of tokens of moe_decode_layer_fp8. */
#define MOE_DECODE_MAX_TOKENS 64

/* Device workspace (bytes, a multiple of 256) of moe_decode_layer_fp8: the
 * quantised h of every (token, choice).  Its contents need no initialisation.
 * MOE_EINVAL for a configuration the call does not take. */
int moe_decode_workspace_bytes(const moe_config* cfg, int32_t inter, size_t* bytes);

/* A whole expert layer for a few tokens, in two kernels and without a grouped
 * copy of the rows:
 *   h[t,k] = SiLU(gate) * up of token t by expert e = topk_idx[t,k], quantised
 *            (as moe_expert_glu_fp8);
 *   out[t] = bf16( sum_k topk_w[t,k] * (w2[e] . h[t,k]) ), products and sum in
 *            float32, rounded once.
 * The same layer through moe_dispatch_send_quantized, moe_expert_glu_fp8,
 * moe_expert_gemm_fp8 and moe_combine_recv differs in that expert_y is rounded
 * to bf16 there.  The chosen experts' weights are read once.
 *   cfg          num_tokens <= MOE_DECODE_MAX_TOKENS, hidden % 128 == 0, else as
 *                for moe_ctx_create (num_ranks plays no part beyond its checks)
 *   inter        inner size of an expert, a multiple of 128; E * 2 * inter and
 *                E * hidden < 2^31
 *   xq, x_scales device E4M3 [T, hidden] and float32 [T, hidden / 128], as
 *                moe_add_rms_norm_fp8 writes them
 *   topk_idx     device int32 [T, K];  topk_w  device float32 [T, K]
 *   w13          device E4M3 [E, 2 * inter, hidden]: gate rows, then up rows
 *   w13_scales   device float32 [E, 2 * inter / 128, hidden / 128]
 *   w2           device E4M3 [E, hidden, inter]
 *   w2_scales    device float32 [E, hidden / 128, inter / 128]
 *   out          device bf16 [T, hidden]
 *   status       device int32 [1], written: MOE_OK, MOE_EROUTE if an index is
 *                out of range or repeated within a token (out is then untouched),
 *                or MOE_ETIMEDOUT if a bounded wait gave up (out is incomplete)
 *   workspace    device, at least moe_decode_workspace_bytes, 256-byte aligned;
 *                calls that may overlap need one each.  A call is two launches:
 *                host threads that share a stream and a workspace may not be
 *                inside this call at the same time
 * xq, w13, w2 and out are 16-byte aligned.  num_tokens == 0 does nothing. */
int moe_decode_layer_fp8(const moe_config* cfg, int32_t inter, const void* xq, const float* x_scales,
                         const int32_t* topk_idx, const float* topk_w, const void* w13, const float* w13_scales,
                         const void* w2, const float* w2_scales, void* out, int32_t* status, void* workspace,
                         size_t workspace_bytes, void* stream);

/* For tests of failure detection: in later calls of this process every CTA of a
 * product kernel leaves out its operand load number `load` (from 0), as if the
 * copy never arrived.  The wait for it runs out after its limit (2 s), and the
 * call reports MOE_ETIMEDOUT.  -1 (the default): none.  MOE_EINVAL below -1. */
int moe_ffn_test_drop_load(int32_t load);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_H_ */
