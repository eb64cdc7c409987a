/*
 * wna16_moe_f8.h -- C ABI of routed experts in 8-bit floats on GB300 (sm_103a):
 * tokens to rows in expert order and back, and products of 8-bit floats with a
 * scale per block of 128 (wna16_moe.h and wna16_moe_block.h: same library, same
 * conventions: device pointers owned by the caller, asynchronous on `stream`,
 * host-side validation only, wna16_moe_last_error for the message, WNA16_OK and
 * nothing launched for an empty batch).
 *
 *   wna16_moe_sort_tokens         a token's row, copied to the rows of its experts
 *   wna16_moe_unsort_tokens       every token's rows back, weighted and added up
 *   wna16_moe_unsort_tokens_grad  the gradient of that
 *   wna16_moe_linear_f8           e4m3 rows times one e4m3 weight
 *   wna16_moe_grouped_linear_f8   e4m3 rows in expert order times their experts' weights
 *   wna16_moe_quantize_blocks_f8  weights to e4m3 with a scale per block of 128 x 128
 *
 * A layer of routed experts with such weights, on 8-bit rows (q, scales) of
 * wna16_moe_add_rmsnorm_q8 (WNA16_Q8_E4M3, group_size 128):
 *   sort_tokens(q, scales) -> grouped_linear_f8 (gate/up) -> wna16_moe_swiglu_q8
 *   (WNA16_Q8_E4M3, 128) -> grouped_linear_f8 (down) -> unsort_tokens
 */
#ifndef WNA16_MOE_F8_H
#define WNA16_MOE_F8_H

#include "wna16_moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A type beside wna16_type's, for rows that are copied only: 8-bit codes. */
enum { WNA16_TYPE_Q8 = 3 };

/* Tokens to rows in the order of their experts.  Slot f = t * topk + j of token t
 * has expert e = topk_ids[f] - expert_begin.  Slots with e in [0, E) get rows in
 * the order of (e, f); the others (other ranges of experts, padding) are left out.
 *   offsets[e]  first row of expert e, int32 [E + 1]; offsets[E]: the rows in use
 *   inv[f]      row of slot f, int32 [T, topk]; -1 if it is left out
 *   rows[inv[f]]       = x[t]          [T * topk, K] of `type`, contiguous
 *   row_scales[inv[f]] = x_scales[t]   fp32 [T * topk, groups] (with x_scales)
 * Rows from offsets[E] on are left as they were.  x [T, K] of `type` (wna16_type or
 * WNA16_TYPE_Q8), rows ldx elements apart; x_scales fp32 [T, groups], contiguous, or
 * NULL.  x and rows NULL (then x_scales too): offsets and inv only.
 * An empty batch gets offsets of 0.
 * 1 <= E <= 1024, 1 <= topk <= 1024, T * topk < 2^31; K up to 2^26.
 * The gradient of rows with respect to x is wna16_moe_unsort_tokens without weights.  */
WNA16_API int wna16_moe_sort_tokens(const void* x, int64_t ldx, const float* x_scales, int64_t groups, int64_t T,
                                    int64_t K, int type, const int32_t* topk_ids, int topk, int64_t E,
                                    int64_t expert_begin, void* rows, float* row_scales, int32_t* offsets,
                                    int32_t* inv, void* stream);

/* out[t] = sum_j weights[t][j] * y[inv[t][j]] (+ addend[t]), in fp32, j ascending, the addend last.
 * Slots whose inv is outside [0, R) are left out (a token without any gets the addend, or zeros).
 *   y [R, K], out [T, K], addend [T, K] (or NULL; may be out) of `type`, contiguous
 *   inv int32 [T, topk], weights fp32 [T, topk] or NULL (all 1)
 * 1 <= topk <= 1024, T * topk and R < 2^31, K up to 2^26.  */
WNA16_API int wna16_moe_unsort_tokens(const void* y, int64_t R, const int32_t* inv, const float* weights,
                                      const void* addend, int64_t T, int64_t K, int topk, int type, void* out,
                                      void* stream);

/* The gradient of unsort_tokens at dout [T, K]:
 *   dy[inv[t][j]] = weights[t][j] * dout[t]              [R, K] of `type`
 *   dweights[t][j] = sum_k dout[t][k] * y[inv[t][j]][k]  fp32 [T, topk], in fp32; 0 for slots left out
 * (the addend's gradient is dout).  Rows of dy that no slot has are left as they were;
 * no two slots may have the same row.  weights NULL: all 1.  y and dweights both or neither;
 * dy may be NULL with them.  */
WNA16_API int wna16_moe_unsort_tokens_grad(const void* dout, const int32_t* inv, const void* y, const float* weights,
                                           int64_t T, int64_t K, int topk, int64_t R, int type, void* dy,
                                           float* dweights, void* stream);

/* out[t][n] = sum_b x_scales[t][b] * w_scales[n / 128][b] * (sum over the 128 k of block b of xq[t][k] * wq[n][k])
 *             (+ bias[n]) (+ addend[t][n])
 *   xq e4m3 [T, K], x_scales fp32 [T, K / 128]    (rows of WNA16_Q8_E4M3, group_size 128)
 *   wq e4m3 [N, K], w_scales fp32 [ceil(N / 128), K / 128]
 *   bias fp32 [N] or NULL, addend [T, N] of `type` or NULL (may be out), out [T, N] of `type`; all contiguous
 * K a multiple of 128, at most 65536; xq and wq 16-byte aligned.  A block's sum is an fp32
 * one of the tensor cores; it is multiplied by the fp32 product of its two scales and added
 * in fp32, in an order that the sizes fix (up to 8 parts of the blocks, b ascending in each, then
 * the parts).  Another number of rows may have another order.
 * A product of two scales outside fp32's range is 0 or infinite.  Rows whose scale is not
 * finite (see wna16_moe_block.h) give NaN.
 * The gradient with respect to the rows' values is the same product of dout's 8-bit rows
 * with the transposed weight (wna16_moe_quantize_blocks_f8 takes either order of strides).
 * Workspace: its first word gets the status word of wna16_moe_read_status (4-byte
 * aligned, at least 4 bytes); NULL: the status is not readable.  Outputs whose sums are
 * missing after a device timeout are NaN either way.  */
WNA16_API int wna16_moe_linear_f8(const void* xq, const float* x_scales, const void* wq, const float* w_scales,
                                  const float* bias, const void* addend, int64_t T, int64_t K, int64_t N, int type,
                                  void* out, void* workspace, size_t workspace_bytes, void* stream);

/* The same for R rows in expert order: rows offsets[e] .. offsets[e + 1] - 1 with weight e.
 *   wq e4m3 [E, N, K], w_scales fp32 [E, ceil(N / 128), K / 128], offsets int32 device [E + 1]
 * Rows of `out` before offsets[0] and from offsets[E] on are left as they were.  Offsets are read on
 * the device: one below its predecessor or above R counts as the nearest that is not, and
 * sets the status word to WNA16_ERR_BAD_ROUTING.  1 <= E <= 1024, E * N < 2^31.  */
WNA16_API int wna16_moe_grouped_linear_f8(const void* xq, const float* x_scales, const void* wq,
                                          const float* w_scales, const int32_t* offsets, int64_t E, int64_t R,
                                          int64_t K, int64_t N, int type, void* out, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* Per block of 128 x 128 of each of E weights [N, K] (the last rows' blocks may be lower):
 *   m = max |w|,  scale = m / 448,  code = e4m3(w * (448 / m)),  value = code * scale
 * with the rules of wna16_moe_block.h for m below 2^-100 and for values that are not finite.
 *   w of `type`; element (e, n, k) at e * stride_e + n * stride_n + k * stride_k, where
 *     stride_k is 1 and stride_n at least K, or stride_n is 1 (a transposed weight) and stride_k at least N;
 *     stride_e at least a weight's extent, (N - 1) * stride_n + (K - 1) * stride_k + 1 (E > 1)
 *   q e4m3 [E, N, K], scales fp32 [E, ceil(N / 128), K / 128], contiguous
 * K a multiple of 128.  */
WNA16_API int wna16_moe_quantize_blocks_f8(const void* w, int64_t E, int64_t N, int64_t K, int64_t stride_e,
                                           int64_t stride_n, int64_t stride_k, int type, void* q, float* scales,
                                           void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WNA16_MOE_F8_H */
