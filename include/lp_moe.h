/*
 * lp_moe.h - what a mixture-of-experts layer needs around its grouped products
 * on AMD Instinct MI355X (gfx950): the router's gate, tokens sorted by expert
 * and back with weights applied, the gradients of both, and forwards of few
 * rows from 4-bit weights.
 *
 * Included with lp.h, whose conventions (device pointers, ownership, streams,
 * status codes, row-major tensors) hold here too.  A layer is
 *
 *   lp_moe_gate          logits -> the k experts and weights of every token
 *   lp_moe_sort          experts -> offsets (the grouped products' groups), the row of
 *                        every (token, slot) pair, the pair of every row
 *   lp_moe_gather        tokens -> rows in the experts' order (bf16), or
 *   lp_moe_gather_quant  the same straight into FP8, both copies
 *   lp_grouped_fwd ...   the experts
 *   lp_moe_combine       rows -> tokens, by the weights
 *
 * and backwards lp_moe_combine_bwd (or lp_moe_gather_quant with the weights, for
 * FP8 gradients), the grouped products, lp_moe_combine without weights, and
 * lp_moe_gate_bwd.
 *
 * Sizes: T tokens, k slots each (1 <= k <= 64), M = T k < 2^30 pairs and rows;
 * 1 to 1024 experts; cols a multiple of 8 below 2^22; M cols < 2^34
 * (LP_ERR_SHAPE otherwise).  Pair (t, j) is number t k + j.  bf16 tensors and
 * codes are 16-byte aligned, int32 and fp32 arrays and logits 4-byte aligned.
 * Every array is dense.  Indices are read on the device; one outside its range
 * stands for nothing (below) and never makes a kernel leave its buffers.
 * None of these calls uses atomics on memory: two calls on the same inputs give
 * the same bits.
 */
#ifndef LP_MOE_H
#define LP_MOE_H

#include "lp.h"
#include "lp_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * lp_moe_gate - every token's k experts and their weights.
 *
 * logits   device [T][E], dtype LP_DTYPE_F32 or LP_DTYPE_BF16; k <= E.
 * chosen   device int32 [T][k]: the experts of the k largest logits, largest
 *          first, of equal ones the lowest index.  -inf is never chosen: slots
 *          that nothing is left for hold -1.
 * weights  device fp32 [T][k]: p_e of each chosen e, p = softmax(logits[t]);
 *          with renorm != 0 divided by their sum over the k slots.  0 where
 *          chosen is -1.
 * A NaN is chosen as +inf is; a row that holds either has NaN weights.
 * Sums and exponentials in fp32.
 */
lp_status lp_moe_gate(const void* logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t topk, int32_t renorm,
                      float* weights, int32_t* chosen, void* stream);

/*
 * lp_moe_gate_bwd - the gradient of the logits.
 *
 * grad_weights  device fp32 [T][k].
 * logits, renorm, weights, chosen: those of lp_moe_gate and what it wrote.
 * grad_logits   device [T][E], in the logits' dtype, with w, g and e of the slots
 *               whose expert is in 0 .. E-1 (the others have no gradient):
 *               renorm: w_j (g_j - sum w g) for the chosen, 0 for the others;
 *               else p_i (sum of g_j over slots with e_j = i, minus sum w g).
 */
lp_status lp_moe_gate_bwd(const float* grad_weights, const void* logits, int32_t dtype, int64_t tokens, int64_t experts,
                          int64_t topk, int32_t renorm, const float* weights, const int32_t* chosen, void* grad_logits,
                          void* stream);

/*
 * lp_moe_sort - the pairs sorted by expert, pairs of one expert in their order.
 *
 * experts  device int32 [pairs]: expert of each pair; outside 0 .. groups-1 the
 *          pair is nobody's (padding, an expert of another GPU).
 * offsets  device int32 [groups]: cumulative end rows, as the grouped products take
 *          them.
 * rows     device int32 [pairs]: the pair's row, -1 for a pair of nobody's.
 * order    device int32 [pairs]: the pair of each row; entries at or past
 *          offsets[groups-1] are left unwritten.
 * workspace  device memory of lp_moe_sort_workspace bytes, 16-byte aligned (NULL
 *          when that is 0); its contents are unspecified before and after, and
 *          calls that may overlap must not share it.  LP_ERR_SHAPE when it is too
 *          small.
 */
lp_status lp_moe_sort_workspace(int64_t pairs, int64_t groups, size_t* bytes);
lp_status lp_moe_sort(const int32_t* experts, int64_t pairs, int64_t groups, int32_t* offsets, int32_t* rows,
                      int32_t* order, void* workspace, size_t workspace_bytes, void* stream);

/*
 * lp_moe_gather - every token's row copied to the rows of its pairs.
 *
 * x     device bf16 [T][cols].
 * rows  device int32 [T][k]; a pair whose row is outside 0 .. M-1 is skipped.
 * y     device bf16 [M][cols]; rows of no pair are left unwritten.
 */
lp_status lp_moe_gather(const void* x, int64_t tokens, int64_t topk, int64_t cols, const int32_t* rows, void* y,
                        void* stream);

/*
 * lp_moe_gather_quant - the rows quantized to LP_FP8_R128 along both axes, without
 * the bf16 rows in between.
 *
 * Row r has the value v = x[order[r] / k], or with weights
 * v = bf16(fp32(weights[order[r]] * x[order[r] / k])), a row whose pair is outside
 * 0 .. M-1 that of zeros.  Writes what lp_r128_quant_dual(v, 1, M, cols, offsets,
 * groups, ...) writes, bit for bit, and leaves unwritten what that leaves
 * unwritten; its rules on sizes hold (cols % 16).  weights: device fp32 [M] by
 * pair, or NULL.
 */
lp_status lp_moe_gather_quant(const void* x, int64_t tokens, int64_t topk, int64_t cols, const int32_t* order,
                              const float* weights, const int32_t* offsets, int64_t groups, void* codes_cols,
                              void* scales_cols, void* codes_rows, void* scales_rows, void* stream);

/*
 * lp_moe_combine - out[t] = sum over j of weights[t][j] * y[rows[t][j]].
 *
 * y        device bf16 [M][cols].
 * rows     device int32 [T][k]; a pair whose row is outside 0 .. M-1 adds nothing.
 * weights  device fp32 [T][k], or NULL for 1 (the gradient of lp_moe_gather).
 * out      device bf16 [T][cols]: fp32 sums in slot order, rounded once; zeros for
 *          a token without a row.
 */
lp_status lp_moe_combine(const void* y, int64_t tokens, int64_t topk, int64_t cols, const int32_t* rows,
                         const float* weights, void* out, void* stream);

/*
 * lp_moe_combine_bwd - the gradients of lp_moe_combine.
 *
 * grad          device bf16 [T][cols], the gradient of out.
 * grad_y        device bf16 [M][cols], or NULL: weights[t][j] * grad[t] at row
 *               rows[t][j]; rows of no pair are left unwritten.  weights NULL: 1.
 * grad_weights  device fp32 [T][k], or NULL: the products grad[t] . y[row] summed in
 *               fp32; 0 for a pair without a row.  y may be NULL without it.
 */
lp_status lp_moe_combine_bwd(const void* grad, const void* y, int64_t tokens, int64_t topk, int64_t cols,
                             const int32_t* rows, const float* weights, void* grad_y, float* grad_weights, void* stream);

/*
 * lp_linear_fwd_w4, lp_grouped_fwd_w4 - y = x @ W^T of a bf16 x and a weight in 4
 * bits, made for few rows: the weight is streamed once.
 *
 * x  device bf16 [M][K], K = w->cols, 16-byte aligned.
 * w  LP_MXFP4 or LP_NVFP4 (scale_axis -1) [N][K], or [groups][N][K]; K % 32 == 0,
 *    N % 16 == 0.
 * y  device bf16 [M][N]; lp_grouped_fwd_w4 leaves rows at or past the last offset
 *    unwritten.  offsets as for lp_grouped_fwd.
 * The product of x with the decoded weight (lp.h: an element is
 * bf16(fp32(code * S))), summed in fp32 on the bf16 MFMA: what lp_dequant of w
 * and lp_linear_fwd (lp_grouped_fwd) compute, up to the order of the sums.  A NaN
 * scale gives NaN in its column of y.  Sizes and errors as for lp_linear_fwd and
 * lp_grouped_fwd; LP_ERR_FORMAT for another weight.
 */
lp_status lp_linear_fwd_w4(const void* x_bf16, int64_t M, const lp_qtensor* w, void* y, void* stream);
lp_status lp_grouped_fwd_w4(const void* x_bf16, int64_t M, const lp_qtensor* w, const int32_t* offsets, int64_t groups,
                            void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LP_MOE_H */
