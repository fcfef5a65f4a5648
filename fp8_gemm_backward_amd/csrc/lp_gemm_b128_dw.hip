// grad_W = grad_out^T @ x of FP8 operands with fp32 scales per 128, dense and grouped.
#include "lp_gemm_b128_kernel.hpp"

namespace lp {
namespace gk {

hipError_t b128_dw(const Params& prm, int tile, hipStream_t s) {
  return tile == 256   ? run_b128<B256, kB128Dw>(prm, s)
         : tile == 128 ? run_b128<B128, kB128Dw>(prm, s)
                       : run_b128<B64, kB128Dw>(prm, s);
}

// The joint end of a dense product whose contraction was split: the fp32 tiles of
// the splits added in their order, eight results a thread.
__global__ __launch_bounds__(256) void b128_join_kernel(Params p, int b) {
  const int per = b * b / (8 * 256), tile = blockIdx.x / per, u = (blockIdx.x % per) * 256 + threadIdx.x;
  const int r = u / (b / 8), c = 8 * (u % (b / 8));
  const int2 pq = dense_order(p, b, tile);
  const int row = pq.x * b + r, col = pq.y * b + c;
  if (row >= p.Ptot || col >= p.Qtot) return;
  const float* src = p.ws + (size_t)tile * p.splits * b * b + r * b + c;
  f32x4 lo{}, hi{};
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, src += b * b) {
    lo += *reinterpret_cast<const f32x4*>(src);
    hi += *reinterpret_cast<const f32x4*>(src + 4);
  }
  *reinterpret_cast<u32x4*>(p.C + (int64_t)row * p.ldc + col) =
      u32x4{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
}

hipError_t b128_join(const Params& prm, int tile, hipStream_t s) {
  b128_join_kernel<<<dim3(prm.ntiles * (tile * tile / (8 * 256))), dim3(256), 0, s>>>(prm, tile);
  return hipGetLastError();
}

hipError_t b128_dw_tail(const Params& prm, hipStream_t s) { return run_b128_tail<kB128Dw>(prm, s); }

}  // namespace gk
}  // namespace lp
