// grad_W = grad_out^T @ x of FP8 operands with fp32 scales per 128, dense and grouped.
#include "lp_gemm_b128_kernel.hpp"

namespace lp {
namespace gk {

hipError_t b128_dw(const Params& prm, int tile, hipStream_t s) {
  return tile == 256   ? run_b128<B256, kB128Dw>(prm, s)
         : tile == 128 ? run_b128<B128, kB128Dw>(prm, s)
                       : run_b128<B64, kB128Dw>(prm, s);
}

hipError_t b128_dw_tail(const Params& prm, hipStream_t s) { return run_b128_tail<kB128Dw>(prm, s); }

}  // namespace gk
}  // namespace lp
