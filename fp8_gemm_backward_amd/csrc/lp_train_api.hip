// C-ABI entry points of lp_train.h: argument checking, then the launches.
// Every rule checked here is stated next to the entry point in the header.
#include <math.h>
#include <stdint.h>

#include "lp_internal.hpp"

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 34;
constexpr int64_t kMaxChunks = (int64_t)1 << 24;   // workgroups of 256 threads: a launch has fewer than 2^32 threads

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
lp_status hip_status(hipError_t e) { return e == hipSuccess ? LP_OK : LP_ERR_HIP; }

// Sizes and offsets of a quantizer call; by_rows: tiles of 16 rows x 512
// columns (axis -1), else of 128 x 128.
lp_status check_quant(int64_t batch, int64_t rows, int64_t cols, bool by_rows, const int32_t* offsets,
                      int64_t groups) {
  constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;
  if (batch < 0 || rows < 0 || cols < 0 || batch > kMaxDim || rows > kMaxDim || cols > kMaxDim) return LP_ERR_SHAPE;
  if (cols % 16) return LP_ERR_SHAPE;
  if (rows * cols != 0 && batch > (kMaxElems - 1) / (rows * cols)) return LP_ERR_SHAPE;
  if (batch * rows > kMaxDim) return LP_ERR_SHAPE;               // rows are counted in 32 bits
  if (offsets != nullptr) {
    if (groups < 1 || groups > 1024) return LP_ERR_SHAPE;
    if (batch != 1) return LP_ERR_FORMAT;
    if (rows >= (int64_t)1 << 30) return LP_ERR_SHAPE;
    if (!aligned(offsets, 4)) return LP_ERR_ALIGN;
  }
  // One workgroup of 256 threads per tile (512 for 128 x 128); a launch has fewer
  // than 2^32 threads.
  const int64_t tiles = by_rows ? (batch * rows / 16 + 1) * (cols / 512 + 1)
                                : batch * (rows / 128 + (offsets ? groups : 1)) * (cols / 128 + 1);
  return tiles >= (int64_t)1 << (by_rows ? 24 : 23) ? LP_ERR_SHAPE : LP_OK;
}

lp_status check_buffers(int64_t n, const void* const* ptrs, int count) {
  if (n == 0) return LP_OK;
  for (int i = 0; i < count; ++i)
    if (ptrs[i] == nullptr) return LP_ERR_NULL;
  for (int i = 0; i < count; ++i)
    if (!aligned(ptrs[i], 16)) return LP_ERR_ALIGN;
  return LP_OK;
}

lp_status fwd_dyn(const void* x, int64_t M, const lp_qtensor* w, const int32_t* offsets, int64_t groups, void* x_codes,
                  void* x_scales, void* y, void* stream) {
  if (w == nullptr) return LP_ERR_NULL;
  if (w->fmt != LP_FP8_B128) return LP_ERR_FORMAT;
  lp_status st = check_quant(1, M, w->cols, true, nullptr, 0);
  if (st != LP_OK) return st;
  const bool fused = lp::fwd_dyn_fuses(M, w->cols, groups != 0);
  if (fused) x_codes = x_scales = const_cast<void*>(x);          // not touched: stand-ins for the checks
  const void* ptrs[] = {x, x_codes, x_scales};
  if ((st = check_buffers(M * w->cols, ptrs, 3)) != LP_OK) return st;
  const lp_qtensor xq{LP_FP8_R128, -1, 1, M, w->cols, x_codes, x_scales, nullptr};
  if ((st = lp::check_forward(&xq, w, y, groups)) != LP_OK) return st;
  if (groups != 0) {
    if (offsets == nullptr) return LP_ERR_NULL;
    if (!aligned(offsets, 4)) return LP_ERR_ALIGN;
  }
  if (M * w->rows == 0) return LP_OK;
  return hip_status(lp::launch_fwd_dyn(x, xq, *w, offsets, (int32_t)(groups ? groups : 1), x_codes, x_scales, y,
                                       static_cast<hipStream_t>(stream)));
}

bool bad_factor(double v) { return !(v >= 0.0) || isinf(v); }

lp_status check_dtypes(int32_t param, int32_t grad, int32_t state) {
  for (int32_t d : {param, grad})
    if (d != LP_DTYPE_F32 && d != LP_DTYPE_BF16) return LP_ERR_FORMAT;
  return state == LP_STATE_F32 || state == LP_STATE_E4M3 ? LP_OK : LP_ERR_FORMAT;
}

}  // namespace

extern "C" {

lp_status lp_r128_quant(const void* src, int64_t batch, int64_t rows, int64_t cols, int32_t axis,
                        const int32_t* offsets, int64_t groups, void* codes, void* scales, void* stream) {
  if (axis != -1 && axis != -2) return LP_ERR_FORMAT;
  if (axis == -1 && offsets != nullptr) return LP_ERR_FORMAT;
  lp_status st = check_quant(batch, rows, cols, axis == -1, offsets, groups);
  if (st != LP_OK) return st;
  const void* ptrs[] = {src, codes, scales};
  if ((st = check_buffers(batch * rows * cols, ptrs, 3)) != LP_OK) return st;
  if (batch * rows * cols == 0) return LP_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return hip_status(axis == -1 ? lp::launch_r128_cols(src, batch, rows, cols, codes, scales, s)
                               : lp::launch_r128_tiles(src, batch, rows, cols, offsets, groups, nullptr, nullptr,
                                                       codes, scales, s));
}

lp_status lp_r128_quant_dual(const void* src, int64_t batch, int64_t rows, int64_t cols, const int32_t* offsets,
                             int64_t groups, void* codes_cols, void* scales_cols, void* codes_rows, void* scales_rows,
                             void* stream) {
  lp_status st = check_quant(batch, rows, cols, false, offsets, groups);
  if (st != LP_OK) return st;
  const void* ptrs[] = {src, codes_cols, scales_cols, codes_rows, scales_rows};
  if ((st = check_buffers(batch * rows * cols, ptrs, 5)) != LP_OK) return st;
  if (batch * rows * cols == 0) return LP_OK;
  return hip_status(lp::launch_r128_tiles(src, batch, rows, cols, offsets, groups, codes_cols, scales_cols, codes_rows,
                                          scales_rows, static_cast<hipStream_t>(stream)));
}

lp_status lp_b128_quant(const void* src, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                        void* stream) {
  lp_status st = check_quant(batch, rows, cols, false, nullptr, 0);
  if (st != LP_OK) return st;
  const void* ptrs[] = {src, codes, scales};
  if ((st = check_buffers(batch * rows * cols, ptrs, 3)) != LP_OK) return st;
  if (batch * rows * cols == 0) return LP_OK;
  return hip_status(lp::launch_r128_tiles(src, batch, rows, cols, nullptr, 0, codes, scales, nullptr, nullptr,
                                          static_cast<hipStream_t>(stream)));
}

lp_status lp_linear_fwd_dyn(const void* x, int64_t M, const lp_qtensor* w, void* x_codes, void* x_scales, void* y,
                            void* stream) {
  return fwd_dyn(x, M, w, nullptr, 0, x_codes, x_scales, y, stream);
}

lp_status lp_grouped_fwd_dyn(const void* x, int64_t M, const lp_qtensor* w, const int32_t* offsets, int64_t groups,
                             void* x_codes, void* x_scales, void* y, void* stream) {
  if (groups < 1 || groups > 1024) return LP_ERR_SHAPE;
  return fwd_dyn(x, M, w, offsets, groups, x_codes, x_scales, y, stream);
}

lp_status lp_adamw_plan(const lp_adamw_tensor* tensors, int64_t count, int32_t param_dtype, int32_t grad_dtype,
                        int32_t state_dtype, void* table, size_t* table_bytes, int64_t* chunks) {
  if (count < 0 || count >= kMaxChunks) return LP_ERR_SHAPE;
  lp_status st = check_dtypes(param_dtype, grad_dtype, state_dtype);
  if (st != LP_OK) return st;
  if (table_bytes == nullptr || chunks == nullptr || (count > 0 && tensors == nullptr)) return LP_ERR_NULL;
  const bool bits8 = state_dtype == LP_STATE_E4M3, bp = param_dtype == LP_DTYPE_BF16, bg = grad_dtype == LP_DTYPE_BF16;
  for (int64_t k = 0; k < count; ++k) {
    const lp_adamw_tensor& t = tensors[k];
    if (t.n < 0 || t.n >= kMaxElems || bad_factor(t.lr_scale) || bad_factor(t.weight_decay)) return LP_ERR_SHAPE;
    if (bp && t.param_copy != nullptr) return LP_ERR_FORMAT;
    if (t.n == 0) continue;
    if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr) return LP_ERR_NULL;
    if (bits8 && (t.exp_avg_scales == nullptr || t.exp_avg_sq_scales == nullptr)) return LP_ERR_NULL;
    if (!aligned(t.param, bp ? 2 : 4) || !aligned(t.grad, bg ? 2 : 4) || !aligned(t.param_copy, 2)) return LP_ERR_ALIGN;
    if (!bits8 && (!aligned(t.exp_avg, 4) || !aligned(t.exp_avg_sq, 4))) return LP_ERR_ALIGN;
    if (bits8 && (!aligned(t.exp_avg_scales, 4) || !aligned(t.exp_avg_sq_scales, 4))) return LP_ERR_ALIGN;
  }
  const int64_t n = lp::adamw_chunks(tensors, count);
  if (n >= kMaxChunks) return LP_ERR_SHAPE;
  const size_t need = lp::adamw_table_bytes(count, n), have = *table_bytes;
  *table_bytes = need;
  *chunks = n;
  if (table == nullptr) return LP_OK;
  if (!aligned(table, 8)) return LP_ERR_ALIGN;
  if (have < need) return LP_ERR_SHAPE;
  lp::adamw_fill(tensors, count, bp, bg, bits8, table);
  return LP_OK;
}

lp_status lp_adamw(const void* table, int64_t count, int64_t chunks, int32_t param_dtype, int32_t grad_dtype,
                   int32_t state_dtype, double lr, double beta1, double beta2, double eps, int64_t step,
                   const float* grad_scale, void* stream) {
  if (count < 0 || chunks < 0 || chunks >= kMaxChunks || step < 1 || bad_factor(lr) || bad_factor(eps)) return LP_ERR_SHAPE;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0)) return LP_ERR_SHAPE;
  lp_status st = check_dtypes(param_dtype, grad_dtype, state_dtype);
  if (st != LP_OK) return st;
  if (chunks > 0 && table == nullptr) return LP_ERR_NULL;
  if (!aligned(table, 8) || !aligned(grad_scale, 4)) return LP_ERR_ALIGN;
  if (chunks == 0) return LP_OK;
  const lp::AdamwCall c{table, count, chunks, param_dtype == LP_DTYPE_BF16, grad_dtype == LP_DTYPE_BF16,
                        state_dtype == LP_STATE_E4M3, lr, beta1, beta2, eps, step, grad_scale};
  return hip_status(lp::launch_adamw(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
