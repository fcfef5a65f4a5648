// C-ABI entry points of lp_moe.h: argument checking, then the launches.
// Every rule checked here is stated next to the entry point in the header.
#include <stdint.h>

#include "lp_internal.hpp"

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 34;
constexpr int64_t kMaxPairs = (int64_t)1 << 30;
constexpr int64_t kMaxCols = (int64_t)1 << 22;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
lp_status hip_status(hipError_t e) { return e == hipSuccess ? LP_OK : LP_ERR_HIP; }

lp_status check_pairs(int64_t tokens, int64_t topk) {
  if (topk < 1 || topk > 64 || tokens < 0 || tokens >= kMaxPairs || tokens * topk >= kMaxPairs) return LP_ERR_SHAPE;
  return LP_OK;
}

lp_status check_rows(int64_t tokens, int64_t topk, int64_t cols) {
  const lp_status st = check_pairs(tokens, topk);
  if (st != LP_OK) return st;
  if (cols < 0 || cols >= kMaxCols || cols % 8 || tokens * topk * cols >= kMaxElems) return LP_ERR_SHAPE;
  return LP_OK;
}

lp_status check_gate(int32_t dtype, int64_t tokens, int64_t experts, int64_t topk) {
  if (dtype != LP_DTYPE_F32 && dtype != LP_DTYPE_BF16) return LP_ERR_FORMAT;
  const lp_status st = check_pairs(tokens, topk);
  if (st != LP_OK) return st;
  if (experts < 1 || experts > 1024 || topk > experts || tokens * experts >= kMaxElems) return LP_ERR_SHAPE;
  return LP_OK;
}

// Required pointers of one alignment.
lp_status check_buffers(const void* const* ptrs, int count, uintptr_t align) {
  for (int i = 0; i < count; ++i)
    if (ptrs[i] == nullptr) return LP_ERR_NULL;
  for (int i = 0; i < count; ++i)
    if (!aligned(ptrs[i], align)) return LP_ERR_ALIGN;
  return LP_OK;
}

lp_status fwd_w4(const void* x, int64_t M, const lp_qtensor* w, const int32_t* offsets, int64_t groups, void* y,
                 void* stream) {
  if (w == nullptr) return LP_ERR_NULL;
  if (M < 0) return LP_ERR_SHAPE;
  const lp_qtensor xq{LP_BF16, -1, 1, M, w->cols, x, nullptr, nullptr};
  const lp_status st = lp::check_forward(&xq, w, y, groups, true);
  if (st != LP_OK) return st;
  if (groups != 0) {
    if (offsets == nullptr) return LP_ERR_NULL;
    if (!aligned(offsets, 4)) return LP_ERR_ALIGN;
  }
  if (M * w->rows == 0) return LP_OK;
  if (w->fmt == LP_NVFP4 && w->tensor_scale == nullptr) return LP_ERR_NULL;   // read also when K is 0
  return hip_status(lp::launch_fwd_w4(xq, *w, offsets, (int32_t)(groups ? groups : 1), y, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

lp_status lp_moe_gate(const void* logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t topk, int32_t renorm,
                      float* weights, int32_t* chosen, void* stream) {
  lp_status st = check_gate(dtype, tokens, experts, topk);
  if (st != LP_OK) return st;
  if (tokens == 0) return LP_OK;
  const void* ptrs[] = {logits, weights, chosen};
  if ((st = check_buffers(ptrs, 3, 4)) != LP_OK) return st;
  return hip_status(lp::launch_moe_gate(logits, dtype == LP_DTYPE_BF16, tokens, (int32_t)experts, (int32_t)topk, renorm != 0,
                                        weights, chosen, static_cast<hipStream_t>(stream)));
}

lp_status lp_moe_gate_bwd(const float* grad_weights, const void* logits, int32_t dtype, int64_t tokens, int64_t experts,
                          int64_t topk, int32_t renorm, const float* weights, const int32_t* chosen, void* grad_logits,
                          void* stream) {
  lp_status st = check_gate(dtype, tokens, experts, topk);
  if (st != LP_OK) return st;
  if (tokens == 0) return LP_OK;
  const void* ptrs[] = {grad_weights, logits, weights, chosen, grad_logits};
  if ((st = check_buffers(ptrs, 5, 4)) != LP_OK) return st;
  return hip_status(lp::launch_moe_gate_bwd(grad_weights, logits, dtype == LP_DTYPE_BF16, tokens, (int32_t)experts,
                                            (int32_t)topk, renorm != 0, weights, chosen, grad_logits,
                                            static_cast<hipStream_t>(stream)));
}

lp_status lp_moe_sort_workspace(int64_t pairs, int64_t groups, size_t* bytes) {
  if (bytes == nullptr) return LP_ERR_NULL;
  *bytes = 0;
  if (pairs < 0 || pairs >= kMaxPairs || groups < 1 || groups > 1024) return LP_ERR_SHAPE;
  *bytes = lp::moe_sort_workspace(pairs, groups);
  return LP_OK;
}

lp_status lp_moe_sort(const int32_t* experts, int64_t pairs, int64_t groups, int32_t* offsets, int32_t* rows,
                      int32_t* order, void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  lp_status st = lp_moe_sort_workspace(pairs, groups, &need);
  if (st != LP_OK) return st;
  if (offsets == nullptr) return LP_ERR_NULL;
  if (!aligned(offsets, 4)) return LP_ERR_ALIGN;
  const void* ptrs[] = {experts, rows, order};
  if (pairs > 0 && (st = check_buffers(ptrs, 3, 4)) != LP_OK) return st;
  if (need > 0) {
    if (workspace == nullptr) return LP_ERR_NULL;
    if (!aligned(workspace, 16)) return LP_ERR_ALIGN;
    if (workspace_bytes < need) return LP_ERR_SHAPE;
  }
  return hip_status(lp::launch_moe_sort(experts, pairs, (int32_t)groups, offsets, rows, order, workspace,
                                        static_cast<hipStream_t>(stream)));
}

lp_status lp_moe_gather(const void* x, int64_t tokens, int64_t topk, int64_t cols, const int32_t* rows, void* y,
                        void* stream) {
  lp_status st = check_rows(tokens, topk, cols);
  if (st != LP_OK) return st;
  if (tokens * cols == 0) return LP_OK;
  const void* ptrs[] = {x, y};
  const void* small[] = {rows};
  if ((st = check_buffers(ptrs, 2, 16)) != LP_OK || (st = check_buffers(small, 1, 4)) != LP_OK) return st;
  return hip_status(lp::launch_moe_gather(x, tokens, topk, cols, rows, y, static_cast<hipStream_t>(stream)));
}

lp_status lp_moe_gather_quant(const void* x, int64_t tokens, int64_t topk, int64_t cols, const int32_t* order,
                              const float* weights, const int32_t* offsets, int64_t groups, void* codes_cols,
                              void* scales_cols, void* codes_rows, void* scales_rows, void* stream) {
  lp_status st = check_rows(tokens, topk, cols);
  if (st != LP_OK) return st;
  const int64_t M = tokens * topk;
  // (the quantizer's own rules, as lp_r128_quant_dual has them)
  if (cols % 16 || groups < 1 || groups > 1024 || (M / 128 + groups) * (cols / 128 + 1) >= (int64_t)1 << 23) return LP_ERR_SHAPE;
  if (M * cols == 0) return LP_OK;
  const void* ptrs[] = {x, codes_cols, scales_cols, codes_rows, scales_rows};
  const void* small[] = {order, offsets};
  if ((st = check_buffers(ptrs, 5, 16)) != LP_OK || (st = check_buffers(small, 2, 4)) != LP_OK) return st;
  if (!aligned(weights, 4)) return LP_ERR_ALIGN;
  return hip_status(lp::launch_moe_gather_quant(x, tokens, topk, cols, order, weights, offsets, groups, codes_cols,
                                                scales_cols, codes_rows, scales_rows, static_cast<hipStream_t>(stream)));
}

lp_status lp_moe_combine(const void* y, int64_t tokens, int64_t topk, int64_t cols, const int32_t* rows,
                         const float* weights, void* out, void* stream) {
  lp_status st = check_rows(tokens, topk, cols);
  if (st != LP_OK) return st;
  if (tokens * cols == 0) return LP_OK;
  const void* ptrs[] = {y, out};
  const void* small[] = {rows};
  if ((st = check_buffers(ptrs, 2, 16)) != LP_OK || (st = check_buffers(small, 1, 4)) != LP_OK) return st;
  if (!aligned(weights, 4)) return LP_ERR_ALIGN;
  return hip_status(lp::launch_moe_combine(y, tokens, topk, cols, rows, weights, out, static_cast<hipStream_t>(stream)));
}

lp_status lp_moe_combine_bwd(const void* grad, const void* y, int64_t tokens, int64_t topk, int64_t cols,
                             const int32_t* rows, const float* weights, void* grad_y, float* grad_weights, void* stream) {
  lp_status st = check_rows(tokens, topk, cols);
  if (st != LP_OK) return st;
  if (tokens == 0 || (grad_y == nullptr && grad_weights == nullptr)) return LP_OK;
  if (grad_weights != nullptr) {
    if (cols > 0 && y == nullptr) return LP_ERR_NULL;
    if (!aligned(y, 16) || !aligned(grad_weights, 4)) return LP_ERR_ALIGN;
  }
  if (cols > 0 && grad == nullptr) return LP_ERR_NULL;
  if (!aligned(grad, 16) || !aligned(grad_y, 16) || !aligned(weights, 4)) return LP_ERR_ALIGN;
  const void* small[] = {rows};
  if ((st = check_buffers(small, 1, 4)) != LP_OK) return st;
  return hip_status(lp::launch_moe_combine_bwd(grad, y, tokens, topk, cols, rows, weights, grad_y, grad_weights,
                                               static_cast<hipStream_t>(stream)));
}

lp_status lp_linear_fwd_w4(const void* x, int64_t M, const lp_qtensor* w, void* y, void* stream) {
  return fwd_w4(x, M, w, nullptr, 0, y, stream);
}

lp_status lp_grouped_fwd_w4(const void* x, int64_t M, const lp_qtensor* w, const int32_t* offsets, int64_t groups,
                            void* y, void* stream) {
  if (groups < 1 || groups > 1024) return LP_ERR_SHAPE;
  return fwd_w4(x, M, w, offsets, groups, y, stream);
}

}  // extern "C"
