/*
 * wna16_moe_block.h -- C ABI of the operators around the routed experts on
 * GB300 (sm_103a): what a transformer layer runs before, beside and after
 * wna16_moe_forward (wna16_moe.h; same library, same conventions: device
 * pointers owned by the caller, asynchronous on `stream`, host-side validation
 * only, wna16_moe_last_error for the message, WNA16_OK and nothing launched
 * for an empty batch).
 *
 *   wna16_moe_add_rmsnorm_q8   residual addition + RMS norm; its rows in 16 bits
 *                              (router, routed experts) and in 8 bits (shared expert)
 *   wna16_moe_route_scored     expert choice: sigmoid or softmax scores, a bias used
 *                              for the choice only, groups, top-k, weights
 *   wna16_moe_linear_q8        product of 8-bit integers with a scale per token and
 *                              per output channel (the shared expert's layers)
 *   wna16_moe_swiglu_q8        the clamped SwiGLU between them, in 8 bits
 *   wna16_moe_quantize_q8, wna16_moe_dequantize_q8   rows to 8 bits and back
 *
 * 8-bit rows (q, scales).  A row of K values, or each run of group_size values
 * of it (group_size 0: the whole row), is held as one fp32 scale and K codes:
 *   m = max |y|,  scale = m / Q,  code = round(y * (Q / m)),  value = code * scale
 * with Q = 127 and codes -127..127 rounded to nearest, ties to even
 * (WNA16_Q8_INT8), or Q = 448 and codes in e4m3 (WNA16_Q8_E4M3).  The quotient and
 * the product are fp32: a value that near to a half step may get either code.  m below
 * 2^-100 gives scale 0 and codes 0.  A row (run) that holds a NaN or an
 * infinity gets a scale that is not finite and codes 0, so that all its values
 * read back as NaN.
 *   q       int8 or e4m3 [T, K], contiguous
 *   scales  fp32 [T, K / group_size] ([T, 1] for group_size 0), contiguous
 * group_size: 0, 32, 64, 128 or 256; a group divides K.
 *
 * Inputs may be rows of a wider tensor: ld* is the distance between rows in
 * elements (>= the row's length).  Any length and alignment is taken; rows
 * whose length is a multiple of 8 and which start on 16-byte boundaries are
 * read 16 bytes at a time.
 */
#ifndef WNA16_MOE_BLOCK_H
#define WNA16_MOE_BLOCK_H

#include "wna16_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { WNA16_TYPE_BF16 = 0, WNA16_TYPE_FP16 = 1, WNA16_TYPE_FP32 = 2 } wna16_type;
typedef enum { WNA16_Q8_INT8 = 0, WNA16_Q8_E4M3 = 1 } wna16_q8_type;
typedef enum { WNA16_SCORE_SIGMOID = 0, WNA16_SCORE_SOFTMAX = 1 } wna16_score;
typedef enum { WNA16_GROUP_TOP2 = 0, WNA16_GROUP_MAX = 1 } wna16_group_score;

/* h = x + residual (fp32, not rounded before its use below; residual NULL: h = x)
 *   residual_out = h rounded to `type`                         (NULL: not written)
 *   y = h / sqrt(mean_k h^2 + eps) * weight                    (fp32)
 *   norm_out = y rounded to `type`                             (NULL: not written)
 *   (q, scales) = y in 8 bits                                  (both NULL: not written)
 * x, residual, residual_out, norm_out of `type`, [T, K]; residual_out and
 * norm_out contiguous; weight [K] of `weight_type` (`type` or fp32).  At least
 * one of norm_out and q.  residual_out may be x or residual itself (same
 * pointer and ld = K); outputs must not overlap inputs otherwise.
 * 1 <= K <= 32768; eps >= 0.
 * The sum of h^2 is an fp32 one: where it passes 3.4e38 (values above 1e18) y is 0, and
 * where the mean and eps are both below 2^-126 (eps 0: values below 1e-19) y loses bits
 * and, where they are 0, is not finite.
 * Rows (runs) with |h weight| below 2^-119 are stored in 8 bits as zeros. */
WNA16_API int wna16_moe_add_rmsnorm_q8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                       const void* weight, int weight_type, int64_t T, int64_t K, int type, float eps,
                                       int q_type, int group_size, void* q, float* scales, void* residual_out,
                                       void* norm_out, void* stream);

/* h = silu(min(g, L)) * clamp(u, -L, L), g = gu[t][0..N), u = gu[t][N..2N);
 * (q, scales) = h in 8 bits.  L = swiglu_limit > 0 (+inf: no clamp), as in
 * wna16_moe_forward; NaN passes through the clamps.  The sigmoid below g = -87 is 0.
 * 1 <= N <= 32768. */
WNA16_API int wna16_moe_swiglu_q8(const void* gu, int64_t ldg, int64_t T, int64_t N, int type, float swiglu_limit,
                                  int q_type, int group_size, void* q, float* scales, void* stream);

/* (q, scales) = x in 8 bits: x [T, K] of `type` (weights: one scale per output channel). */
WNA16_API int wna16_moe_quantize_q8(const void* x, int64_t ldx, int64_t T, int64_t K, int type, int q_type,
                                    int group_size, void* q, float* scales, void* stream);

/* out = code * scale, rounded to `type`, [T, K] contiguous. */
WNA16_API int wna16_moe_dequantize_q8(const void* q, const float* scales, int64_t T, int64_t K, int q_type,
                                      int group_size, int type, void* out, void* stream);

/* Expert choice.  Per token, with s_e = sigmoid(z_e) or softmax(z)_e and
 * c_e = s_e + bias_e (bias NULL: c = s):
 *   1. the experts are `groups` runs of E / groups; a group's score is the sum
 *      of its two largest c (WNA16_GROUP_TOP2) or its largest (WNA16_GROUP_MAX);
 *      the topk_groups best groups stay
 *   2. topk_ids = the topk experts of largest c in them, descending
 *   3. topk_weights = s of the chosen (without the bias), divided by their sum
 *      if `renormalize` (sum 0: weights 0), times `scale`
 * Equal values go to the lower index, in both choices.  The choice is that of
 * exact scores: without a bias the experts' order is the logits' order; else it
 * is made on 32-bit scores, and again on 64-bit ones for a token in which two
 * neighbours in the order are closer than the 32-bit error.
 * A logit of -inf (a masked expert) or NaN scores 0, and so does one below -709
 * (sigmoid) or 709 below the token's largest (softmax); a token without any other
 * gets the lowest experts (by bias) with weights 0.  Softmax: logits of +inf share the whole weight.  A bias of +inf counts
 * as fp32's largest number, one of -inf or NaN as its lowest.
 *   logits        fp32, bf16 or fp16 device [T, E], rows ld apart
 *   bias          fp32 device [E] or NULL
 *   topk_ids      int32 device [T, topk] (written)
 *   topk_weights  fp32 device [T, topk] (written)
 * E <= 1024; groups <= 32 divides E; topk <= min(32, topk_groups * E / groups). */
WNA16_API int wna16_moe_route_scored(const void* logits, int64_t ld, const float* bias, int64_t T, int64_t E, int type,
                                     int score, int groups, int topk_groups, int group_score, int topk,
                                     int renormalize, float scale, int32_t* topk_ids, float* topk_weights,
                                     void* stream);

/* out[t][n] = (sum_k xq[t][k] * wq[n][k]) * x_scales[t] * w_scales[n]
 *             (+ bias[n]) (+ addend[t][n])
 *   xq int8 [T, K], wq int8 [N, K], x_scales fp32 [T], w_scales fp32 [N],
 *   bias fp32 [N] or NULL, addend [T, N] of `type` or NULL (may be out),
 *   out [T, N] of `type`; all contiguous
 * K a multiple of 16, at most 65536; xq and wq 16-byte aligned.  The sums are
 * 32-bit integers for up to 32 tokens, and for more where the weights have few
 * channels (an estimate of time decides).  Other calls have fp32 sums of exact
 * products on the tensor cores, which are the same integers while no partial sum
 * passes 2^24 (always for K <= 1024).  Beyond that bits are dropped on the way: with
 * S = sum_k |xq[t][k] wq[n][k]| the sum is off by 2^-20 S per 16 k at most.  That
 * is an absolute error; where large products cancel it can pass the sum itself.
 * (Measured at 65536 k, products of 1023 after half as many of 16129: 8e-4 of the
 * sum.)  Workspace (256-byte aligned): its first
 * word is the status word of wna16_moe_read_status, the size is below.  It is 0
 * for up to 32 tokens; a workspace of at least 4 bytes gets the status word all
 * the same.  It may be NULL: the status word is then not readable; an output
 * whose sums are missing after a device timeout is NaN either way. */
WNA16_API int wna16_moe_linear_q8(const int8_t* xq, const float* x_scales, const int8_t* wq, const float* w_scales,
                                  const float* bias, const void* addend, int64_t T, int64_t K, int64_t N, int type,
                                  void* out, void* workspace, size_t workspace_bytes, void* stream);
WNA16_API size_t wna16_moe_linear_q8_workspace_size(int64_t T, int64_t K, int64_t N);

#ifdef __cplusplus
}
#endif

#endif /* WNA16_MOE_BLOCK_H */
