// grad_X = grad_out @ W of FP8 operands with fp32 scales per 128, dense and grouped.
#include "lp_gemm_b128_kernel.hpp"

namespace lp {
namespace gk {

hipError_t b128_dx(const Params& prm, int tile, hipStream_t s) {
  return tile == 256   ? run_b128<B256, kB128Dx>(prm, s)
         : tile == 128 ? run_b128<B128, kB128Dx>(prm, s)
                       : run_b128<B64, kB128Dx>(prm, s);
}

hipError_t b128_dx_tail(const Params& prm, hipStream_t s) { return run_b128_tail<kB128Dx>(prm, s); }

}  // namespace gk
}  // namespace lp
