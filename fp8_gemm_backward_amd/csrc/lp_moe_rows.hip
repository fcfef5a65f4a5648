// Rows of tokens to their experts and back (HBM-bound).
//
//   gather:   y[rows[t][j]] = x[t]
//   combine:  out[t] = sum_j w[t][j] y[rows[t][j]]
//   backward: grad_y[rows[t][j]] = w[t][j] grad[t],  grad_w[t][j] = grad[t] . y[rows[t][j]]
//
// All of them by token: a token's row is read (or written) once and its k rows
// written (read) from there, whichever way the indices point.
#include <type_traits>

#include "lp_device.hpp"
#include "lp_internal.hpp"
#include "lp_mxq.hpp"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 20;

struct RowArgs {
  const uint16_t* x;
  const uint16_t* y;
  uint16_t* out;
  float* grad_w;
  const int32_t* rows;
  const float* weights;
  int64_t tokens;
  int32_t k, pieces;                           // pieces of 8 columns in a row; tokens * pieces < 2^31
  uint32_t M;
  FastDiv per_row;                             // by pieces
};

// Rows (of all experts) of more than a quarter of the 256 MB cache are read and
// written past the caches: what runs between their writing and reading, an
// expert's weights at least, leaves little of them there.  32768 rows of 7168 copied
// in 91 us (5.8 TB/s; 103 by way of the caches), summed by eights in 93 (104), 16384
// rows of 4096 in 30 and 35 (39 and 40).
constexpr int64_t kCacheBytes = (int64_t)64 << 20;

__device__ __forceinline__ u32x4 load16(const uint16_t* base, int64_t row, int pieces, int c) {
  return reinterpret_cast<const u32x4*>(base)[row * pieces + c];
}
template <bool kStream>
__device__ __forceinline__ u32x4 load_row(const uint16_t* base, int64_t row, int pieces, int c) {
  const u32x4* p = reinterpret_cast<const u32x4*>(base) + row * pieces + c;
  return kStream ? __builtin_nontemporal_load(p) : *p;
}
template <bool kStream>
__device__ __forceinline__ void store_row(uint16_t* base, int64_t row, int pieces, int c, u32x4 v) {
  u32x4* p = reinterpret_cast<u32x4*>(base) + row * pieces + c;
  if constexpr (kStream) __builtin_nontemporal_store(v, p);
  else *p = v;
}

template <bool kStream>
__global__ __launch_bounds__(kThreads) void gather_kernel(RowArgs a) {
  const uint32_t units = (uint32_t)a.tokens * a.pieces;
  for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < units; u += gridDim.x * kThreads) {
    const uint32_t token = fdiv(u, a.per_row);
    const int c = (int)(u - token * a.pieces);
    const int64_t t = token;
    const u32x4 v = load16(a.x, t, a.pieces, c);
    for (int j = 0; j < a.k; ++j) {
      const uint32_t r = (uint32_t)a.rows[t * a.k + j];
      if (r < a.M) store_row<kStream>(a.out, r, a.pieces, c, v);
    }
  }
}

template <bool kWeighted, bool kStream, int kSlots>             // kSlots: rows in flight per thread
__global__ __launch_bounds__(kThreads) void combine_kernel(RowArgs a) {
  const uint32_t units = (uint32_t)a.tokens * a.pieces;
  for (uint32_t u = blockIdx.x * kThreads + threadIdx.x; u < units; u += gridDim.x * kThreads) {
    const uint32_t token = fdiv(u, a.per_row);
    const int c = (int)(u - token * a.pieces);
    const int64_t t = token;
    float s[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += kSlots) {
      u32x4 v[kSlots];
      float w[kSlots];
      uint32_t r[kSlots];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        r[i] = j0 + i < a.k ? (uint32_t)a.rows[t * a.k + j0 + i] : ~0u;
        w[i] = 1.0f;
        if (r[i] >= a.M) continue;
        v[i] = load_row<kStream>(a.y, r[i], a.pieces, c);
        if constexpr (kWeighted) w[i] = a.weights[t * a.k + j0 + i];
      }
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (r[i] >= a.M) continue;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          s[2 * d] = __builtin_fmaf(w[i], bf16_lo(v[i][d]), s[2 * d]);
          s[2 * d + 1] = __builtin_fmaf(w[i], bf16_hi(v[i][d]), s[2 * d + 1]);
        }
      }
    }
    reinterpret_cast<u32x4*>(a.out)[u] =
        u32x4{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]), pack_bf16x2(s[6], s[7])};
  }
}

// Sum over groups of kLanes lanes, in all of them.
template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int d = 1; d < kLanes; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// kOwn threads per token (of a workgroup of at least kThreads): x is the token's
// gradient.
template <bool kRows, bool kDots, bool kStream, int kSlots, int kOwn>
__global__ __launch_bounds__(kOwn < kThreads ? kThreads : kOwn) void combine_bwd_kernel(RowArgs a) {
  constexpr int kTokens = kOwn < kThreads ? kThreads / kOwn : 1, kLanes = kOwn < 64 ? kOwn : 64;
  static_assert(kOwn <= 64 || kTokens == 1);
  __shared__ float part[kOwn / kLanes][kSlots];
  const int own = threadIdx.x % kOwn, lane = own % kLanes, wave = own / kLanes;
  for (int64_t t = (int64_t)blockIdx.x * kTokens + threadIdx.x / kOwn; t < a.tokens; t += (int64_t)gridDim.x * kTokens) {
    for (int j0 = 0; j0 < a.k; j0 += kSlots) {
      uint32_t r[kSlots];
      float w[kSlots], dot[kSlots] = {};
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        r[i] = j0 + i < a.k ? (uint32_t)a.rows[t * a.k + j0 + i] : ~0u;
        w[i] = kRows && a.weights != nullptr && j0 + i < a.k ? a.weights[t * a.k + j0 + i] : 1.0f;
      }
      for (int c = own; c < a.pieces; c += kOwn) {
        const u32x4 g = load16(a.x, t, a.pieces, c);
        float f[8];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          f[2 * d] = bf16_lo(g[d]);
          f[2 * d + 1] = bf16_hi(g[d]);
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          if (r[i] >= a.M) continue;
          if constexpr (kDots) {
            const u32x4 v = load_row<kStream>(a.y, r[i], a.pieces, c);
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              dot[i] = __builtin_fmaf(f[2 * d], bf16_lo(v[d]), dot[i]);
              dot[i] = __builtin_fmaf(f[2 * d + 1], bf16_hi(v[d]), dot[i]);
            }
          }
          if constexpr (kRows)
            store_row<kStream>(a.out, r[i], a.pieces, c,
                               u32x4{pack_bf16x2(w[i] * f[0], w[i] * f[1]), pack_bf16x2(w[i] * f[2], w[i] * f[3]),
                                     pack_bf16x2(w[i] * f[4], w[i] * f[5]), pack_bf16x2(w[i] * f[6], w[i] * f[7])});
        }
      }
      if constexpr (kDots && kOwn <= 64) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          dot[i] = sum_lanes<kLanes>(dot[i]);
          if (lane == i && j0 + i < a.k) a.grad_w[t * a.k + j0 + i] = dot[i];
        }
      } else if constexpr (kDots) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          dot[i] = sum_lanes<kLanes>(dot[i]);
          if (lane == 0) part[wave][i] = dot[i];
        }
        __syncthreads();
        if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < a.k) {
          float s = 0.0f;
          for (int v = 0; v < kOwn / 64; ++v) s += part[v][threadIdx.x];
          a.grad_w[t * a.k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
      }
    }
  }
}

RowArgs args(const void* x, const void* y, void* out, float* grad_w, const int32_t* rows, const float* weights,
             int64_t tokens, int64_t topk, int64_t cols) {
  return RowArgs{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(y), static_cast<uint16_t*>(out), grad_w,
                 rows, weights, tokens, (int32_t)topk, (int32_t)(cols / 8), (uint32_t)(tokens * topk),
                 make_fastdiv((uint32_t)(cols >= 8 ? cols / 8 : 1))};
}
bool streams(const RowArgs& a) { return (int64_t)a.M * a.pieces * 16 > kCacheBytes; }
dim3 grid_of(int64_t blocks) { return dim3((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks)); }

// f with the rows in flight for k slots a token: no more than there are, at most 8
// (2048 tokens of 1040 with 4 rows backwards: 10.1 us by 4, 14.7 by 8).
template <class F>
void by_slots(int64_t k, F&& f) {
  if (k <= 2) f(std::integral_constant<int, 2>{});
  else if (k <= 4) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
}

// Threads of a token in combine_bwd (us of the dots alone by 256, 64 and 16, 8 rows a
// token unless said): short rows get 16 (2000 tokens of 128: 9.0, 5.1, 4.5; 16000 of
// 256 with 7: 48, 19, 13), longer ones of enough tokens to fill the GPU a wave (2000 of
// 1024: 12.7, 10.6, 28; of 2048 with 4: 9.0, 10.5), the rest 256, and 1024 where there
// are few (256 tokens of 7168, both results: 13.6 us, 18.6 by 256), past the caches only
// where rows are longer yet (900 of 7168, both results: 58.6 us by 1024, 47.3 by 256; 512
// of 16384 59 and 64).  Which results are asked for changes nothing: the dots have
// the same bits with the rows or without.
constexpr int64_t kFewTokens = 1024, kManyTokens = 8192;

template <bool kStream, int kOwn>
void bwd(const RowArgs& a, hipStream_t s) {
  by_slots(a.k, [&](auto slots) {
    constexpr int kSlots = decltype(slots)::value, kBlock = kOwn < kThreads ? kThreads : kOwn;
    const dim3 grid = grid_of((a.tokens * kOwn + kBlock - 1) / kBlock), block(kBlock);
    if (a.out != nullptr && a.grad_w != nullptr)
      combine_bwd_kernel<true, true, kStream, kSlots, kOwn><<<grid, block, 0, s>>>(a);
    else if (a.out != nullptr)
      combine_bwd_kernel<true, false, kStream, kSlots, kOwn><<<grid, block, 0, s>>>(a);
    else
      combine_bwd_kernel<false, true, kStream, kSlots, kOwn><<<grid, block, 0, s>>>(a);
  });
}

}  // namespace

hipError_t launch_moe_gather(const void* x, int64_t tokens, int64_t topk, int64_t cols, const int32_t* rows, void* y,
                             hipStream_t s) {
  const RowArgs a = args(x, nullptr, y, nullptr, rows, nullptr, tokens, topk, cols);
  const dim3 grid = grid_of((tokens * a.pieces + kThreads - 1) / kThreads);
  streams(a) ? gather_kernel<true><<<grid, dim3(kThreads), 0, s>>>(a) : gather_kernel<false><<<grid, dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe_combine(const void* y, int64_t tokens, int64_t topk, int64_t cols, const int32_t* rows,
                              const float* weights, void* out, hipStream_t s) {
  const RowArgs a = args(nullptr, y, out, nullptr, rows, weights, tokens, topk, cols);
  const dim3 grid = grid_of((tokens * a.pieces + kThreads - 1) / kThreads);
  const auto run = [&](auto slots) {
    constexpr int kSlots = decltype(slots)::value;
    const dim3 block(kThreads);
    if (weights != nullptr)
      streams(a) ? combine_kernel<true, true, kSlots><<<grid, block, 0, s>>>(a) : combine_kernel<true, false, kSlots><<<grid, block, 0, s>>>(a);
    else
      streams(a) ? combine_kernel<false, true, kSlots><<<grid, block, 0, s>>>(a) : combine_kernel<false, false, kSlots><<<grid, block, 0, s>>>(a);
  };
  by_slots(topk, run);
  return hipGetLastError();
}

hipError_t launch_moe_combine_bwd(const void* grad, const void* y, int64_t tokens, int64_t topk, int64_t cols,
                                  const int32_t* rows, const float* weights, void* grad_y, float* grad_w,
                                  hipStream_t s) {
  const RowArgs a = args(grad, y, grad_y, grad_w, rows, weights, tokens, topk, cols);
  const bool past = streams(a), few = tokens < kFewTokens;
  if (a.pieces <= (tokens < kManyTokens ? 16 : 32)) past ? bwd<true, 16>(a, s) : bwd<false, 16>(a, s);
  else if (!few && a.pieces <= 128) past ? bwd<true, 64>(a, s) : bwd<false, 64>(a, s);
  else if (few && a.pieces > (past ? 1024 : kThreads)) past ? bwd<true, 1024>(a, s) : bwd<false, 1024>(a, s);
  else past ? bwd<true, kThreads>(a, s) : bwd<false, kThreads>(a, s);
  return hipGetLastError();
}

}  // namespace lp
