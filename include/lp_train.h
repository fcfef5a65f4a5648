/*
 * lp_train.h - training with block-scaled FP8 operands on AMD Instinct MI355X
 * (gfx950): quantization to E4M3 with fp32 scales per 128 elements, forwards
 * that quantize their own input, and the AdamW step.
 *
 * Included with lp.h, whose conventions (device pointers, ownership, streams,
 * status codes, alignment, row-major tensors) hold here too.  The products
 * themselves are those of lp.h, with these operands:
 *
 *   y      = lp_linear_fwd / lp_grouped_fwd    x LP_FP8_R128 (axis -1), w LP_FP8_B128
 *   grad_X = lp_linear_bwd / lp_grouped_bwd    grad_out LP_FP8_R128 (axis -1), w LP_FP8_B128
 *   grad_W = lp_linear_bwd / lp_grouped_bwd    grad_out and x LP_FP8_R128 (axis -2)
 *
 * lp_linear_bwd_workspace reports a size for a dense product of few output tiles
 * over a long contraction, and lp_linear_bwd_ws then splits it; of these
 * operands' workspace nothing need be zero before the call, its first 4 KiB
 * are left alone, the rest is overwritten.
 *
 * Quantization rule, shared by every function here.  A set of values (a run
 * of 128 along an axis, cut at the tensor's edge, or a 128 x 128 block) with
 * largest magnitude a gets
 *     s = fp32(max(a, 2^-64) / 448)           (fp32 division, nearest even)
 *     code = E4M3(fp32(v / s))                (nearest even, saturating at 448)
 * A set that holds a NaN or an infinity gets s = NaN and the code 0x7F with
 * each element's sign.  Bit-exact.
 *
 * Sizes of the quantizers: cols % 16 == 0, fewer than 2^34 elements, and fewer
 * than 2^23 tiles of 128 x 128 (axis -1: 2^24 of 16 x 512), partial ones and
 * one spare per batch entry or group counted (LP_ERR_SHAPE otherwise).
 */
#ifndef LP_TRAIN_H
#define LP_TRAIN_H

#include "lp.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * lp_r128_quant - bf16 to LP_FP8_R128 along one axis.
 *
 * src_bf16  device bf16 [batch][rows][cols]; cols % 16 == 0, rows arbitrary.
 * axis      -1: runs along cols; scales fp32 [batch][ceil(cols/128)][rows].
 *           -2: runs along rows; scales fp32 [batch][ceil(rows/128)][cols].
 * offsets   NULL, or (axis -2, batch 1 only: LP_ERR_FORMAT otherwise) device
 *           int32 [groups], cumulative end rows as for lp_grouped_bwd, read
 *           on the device and clamped as there.  Runs then restart at every
 *           group's first row: group g, starting at row o, has the run
 *           indices o / 128 + g, o / 128 + g + 1, ..., its last run cut at the
 *           group's end; scales are [rows / 128 + groups][cols].  Run indices
 *           that no group has, and rows at or past the last offset, are left
 *           unwritten.  1 <= groups <= 1024.
 * codes     device bytes [batch][rows][cols].
 */
lp_status lp_r128_quant(const void* src_bf16, int64_t batch, int64_t rows, int64_t cols, int32_t axis,
                        const int32_t* offsets, int64_t groups, void* codes, void* scales, void* stream);

/*
 * lp_r128_quant_dual - both copies of one tensor from one read.
 *
 * codes_cols, scales_cols  what lp_r128_quant(axis -1) writes.
 * codes_rows, scales_rows  what lp_r128_quant(axis -2, offsets) writes.
 * With offsets (batch 1 only), rows at or past the last offset are left
 * unwritten in both copies.
 */
lp_status lp_r128_quant_dual(const void* src_bf16, int64_t batch, int64_t rows, int64_t cols, const int32_t* offsets,
                             int64_t groups, void* codes_cols, void* scales_cols, void* codes_rows, void* scales_rows,
                             void* stream);

/*
 * lp_b128_quant - bf16 to LP_FP8_B128: one fp32 scale per 128 x 128 block,
 * scales [batch][ceil(rows/128)][ceil(cols/128)]; cols % 16 == 0.
 */
lp_status lp_b128_quant(const void* src_bf16, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                        void* stream);

/*
 * lp_linear_fwd_dyn, lp_grouped_fwd_dyn - the forward y = x @ W^T from a bf16
 * x, quantized as part of the call.
 *
 * Computes what lp_r128_quant(x, axis -1) followed by lp_linear_fwd (or
 * lp_grouped_fwd) computes, up to fp32 summation order.
 *
 * x         device bf16 [M][K], K = w->cols.
 * w         LP_FP8_B128 [N][K] (lp_grouped_fwd_dyn: [groups][N][K]).
 * x_codes   device bytes [M][K] and
 * x_scales  device fp32 [ceil(K/128)][M]: caller-owned scratch, not to be
 *           shared by calls that may overlap; its contents afterwards are
 *           unspecified.  lp_linear_fwd_dyn of M <= 4 rows with M * 128 *
 *           ceil(K/128) <= 65536 quantizes x inside the product and needs none
 *           (both may be NULL).
 * y         device bf16 [M][N]; lp_grouped_fwd_dyn leaves rows at or past
 *           the last offset unwritten.
 * Errors as lp_r128_quant and lp_linear_fwd / lp_grouped_fwd, found before
 * anything is enqueued.
 */
lp_status lp_linear_fwd_dyn(const void* x_bf16, int64_t M, const lp_qtensor* w, void* x_codes, void* x_scales, void* y,
                            void* stream);
lp_status lp_grouped_fwd_dyn(const void* x_bf16, int64_t M, const lp_qtensor* w, const int32_t* offsets,
                             int64_t groups, void* x_codes, void* x_scales, void* y, void* stream);

/*
 * lp_adamw_plan, lp_adamw - one AdamW step (decoupled weight decay) over many
 * tensors, in one launch.
 *
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
 *   p = (1 - lr wd) p - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *
 * with lr = lr * lr_scale and wd = weight_decay of the tensor.  Each operation
 * is rounded to fp32 by itself; the factors that depend on the step only are
 * computed in double, then rounded.  An fp32 or bf16 parameter, an fp32 or
 * bf16 gradient; one combination per plan.
 *
 * lp_adamw_plan writes the table that lp_adamw reads: which tensors, and which
 * part of them each workgroup takes.  It runs on the host and touches no GPU.
 * The caller copies the table to device memory once and keeps it (and the
 * tensors) as long as it steps with it, or replays a graph that captured a step
 * with it; a plan is made anew when a tensor moves.
 *
 * tensors      HOST array of `count`, not kept.  Pointers need the alignment of
 *              their element only; tensors whose pointers are all aligned to
 *              four elements (param, grad, exp_avg, exp_avg_sq, param_copy) take
 *              wider accesses.  Tensors of one plan must not overlap.
 * state_dtype  LP_STATE_F32: exp_avg and exp_avg_sq are fp32 [n].
 *              LP_STATE_E4M3: exp_avg holds E4M3 codes of m, exp_avg_sq those
 *              of sqrt(v), bytes [n], in runs of 128 consecutive elements by
 *              the quantization rule above, with fp32 scales
 *              [ceil(n/128)] each; a positive sqrt(v) never becomes 0 (at
 *              least code 1).  All-zero codes and scales are the initial state.
 * table        HOST buffer, 8-byte aligned, or NULL to ask for its size only.
 * table_bytes  in: the buffer's size; out: the bytes needed.
 * chunks       out: the number of workgroups, an argument of lp_adamw.
 * Errors: LP_ERR_SHAPE for count < 0, n < 0 or n >= 2^34, a negative or
 * non-finite lr_scale or weight_decay, 2^24 chunks or more (a chunk is 4096
 * elements of one tensor), or a buffer too small; LP_ERR_FORMAT for an unknown
 * dtype, or a param_copy beside a bf16 parameter; LP_ERR_NULL, LP_ERR_ALIGN as
 * usual.
 *
 * lp_adamw     table is the DEVICE copy (8-byte aligned); count, chunks and the
 *              dtypes those of its plan.  grad_scale: device fp32, or NULL for 1
 *              (loss scaling, clipping).  step: 1 for the first.
 * Errors: LP_ERR_SHAPE for step < 1, betas outside [0, 1), a negative or
 * non-finite lr or eps, count < 0, chunks outside [0, 2^24); LP_ERR_FORMAT,
 * LP_ERR_NULL, LP_ERR_ALIGN.
 */
enum { LP_STATE_F32 = 0, LP_STATE_E4M3 = 1 };
enum { LP_DTYPE_F32 = 0, LP_DTYPE_BF16 = 1 };

typedef struct {
  void* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scales;       /* LP_STATE_E4M3 only */
  float* exp_avg_sq_scales;    /* LP_STATE_E4M3 only */
  void* param_copy;            /* bf16 [n] that receives the new fp32 parameter rounded, or NULL */
  int64_t n;
  float lr_scale;
  float weight_decay;
} lp_adamw_tensor;

lp_status lp_adamw_plan(const lp_adamw_tensor* tensors, int64_t count, int32_t param_dtype, int32_t grad_dtype,
                        int32_t state_dtype, void* table, size_t* table_bytes, int64_t* chunks);
lp_status lp_adamw(const void* table, int64_t count, int64_t chunks, int32_t param_dtype, int32_t grad_dtype,
                   int32_t state_dtype, double lr, double beta1, double beta2, double eps, int64_t step,
                   const float* grad_scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LP_TRAIN_H */
