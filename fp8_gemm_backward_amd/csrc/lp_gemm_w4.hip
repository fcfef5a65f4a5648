// Forward y = x @ W^T of few bf16 rows by a weight in 4 bits (MXFP4, NVFP4),
// dense and grouped.
//
// The weight is read once and everything else is small, so the call is a
// stream over W.  A wave owns 16 columns of y (16 rows of W), up to 16 kRT rows
// of x and every kWK-th 256-deep block of the contraction.  Lane l of
// v_mfma_f32_16x16x32_bf16 holds eight contraction elements of row l % 16; any
// order of the contraction will do as long as x has the same, so a lane takes
// 32 consecutive elements (16 bytes of codes, one MXFP4 scale or two NVFP4
// scales) straight from global memory and decodes eight of them per MFMA, in
// registers, as lp_dequant does.  The sums of the kWK waves that share 16
// columns are added in wave order at the end, so the result does not depend on
// timing.
#include "lp_gemm_kernel.hpp"

namespace lp {
namespace gk {
namespace {

constexpr int kWaves = 8;
constexpr int kBlock = 256;                     // contraction elements of a block: 128 bytes of codes a row

template <int F, int kRT>
struct Block {
  Raw<F, -1> w[2];
  u32x4 x[kRT][2][4];
};

struct W4Args {
  Params p;
  int32_t row_tiles;                            // row tiles of the grid
};

template <int F, int kWK, int kRT>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2))) void w4_kernel(W4Args a) {
  constexpr int kRows = 16 * kRT, kDepth = kRT > 1 ? 1 : 2, WN = kWaves / kWK;
  using Blk = Block<F, kRT>;
  const Params& p = a.p;
  __shared__ union {
    int32_t ends[kMaxGroups];
    f32x4 sum[kWK == 1 ? 1 : kWaves][kRT][64];
  } sh;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave % kWK, wn = wave / kWK;
  // Workgroups are dealt to the 8 XCDs in turn: the row tiles of one column
  // tile share an XCD, whose L2 then serves the weight's second reads.
  const int xcd = blockIdx.x % 8, j = blockIdx.x / 8;
  const int rt = j % a.row_tiles, n0 = (((j / a.row_tiles) * 8 + xcd) * WN + wn) * 16;
  int g = 0, p0 = rt * kRows, pend = p.Ptot;
  if (p.offsets != nullptr) {
    for (int i = tid; i < p.groups; i += 64 * kWaves) sh.ends[i] = p.offsets[i];
    __syncthreads();
    const GroupHit hit = find_row_tile<kRows>(sh.ends, p.groups, p.Ptot, rt, [](int) { return true; });
    if (!hit.found) return;
    g = __builtin_amdgcn_readfirstlane(hit.g);
    p0 = __builtin_amdgcn_readfirstlane(hit.start + (rt - hit.seen) * kRows);
    pend = __builtin_amdgcn_readfirstlane(hit.end);
  }
  if (p0 >= pend) return;

  const int K = p.Ktot, nb = n0 < p.Qtot ? (K + kBlock - 1) / kBlock : 0;   // no block for columns past the end
  const int r = lane & 15, h = lane >> 4;
  const Rsrc wr = make_rsrc(p.Q.codes + (int64_t)g * p.Q.code_batch + (int64_t)n0 * p.Q.code_ld, (int64_t)16 * p.Q.code_ld);
  const Rsrc sr = make_rsrc(p.Q.scales + (int64_t)g * p.Q.scale_batch + (int64_t)n0 * p.Q.scale_ld, (int64_t)16 * p.Q.scale_ld);
  const Rsrc xr = make_rsrc(p.P.codes + (int64_t)p0 * p.P.code_ld, (int64_t)(pend - p0) * p.P.code_ld);
  float ts = 0.0f;
  if constexpr (F == NVFP4) ts = *p.Q.tensor_scale;

  // Block kb of the contraction; blocks and columns past the end read as zero.
  auto load = [&](Blk& b, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k0 = kb * kBlock + 128 * e + 32 * h;             // K % 32 == 0: a lane's elements are all in or all out
      const bool in = kb < nb && k0 < K;
      b.w[e].c = bload16(wr, in ? r * p.Q.code_ld + k0 / 2 : kOOB);
      if constexpr (F == NVFP4)
        b.w[e].s = __builtin_amdgcn_raw_buffer_load_b16(sr, in ? r * p.Q.scale_ld + k0 / 16 : kOOB, 0, 0);
      else
        b.w[e].s = __builtin_amdgcn_raw_buffer_load_b8(sr, in ? r * p.Q.scale_ld + k0 / 32 : kOOB, 0, 0);
#pragma unroll
      for (int t = 0; t < kRT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) b.x[t][e][q] = bload16(xr, in ? (r + 16 * t) * p.P.code_ld + 2 * k0 + 16 * q : kOOB);
    }
  };

  f32x4 acc[kRT] = {};
  auto multiply = [&](const Blk& b) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      static_for<4>([&](auto piece) __attribute__((always_inline)) {
        constexpr int J = decltype(piece)::value;
        float sc;
        u32x4 w;
        w[0] = decode_quarter<F, -1, J, 0>(b.w[e], ts, sc);
        w[1] = decode_quarter<F, -1, J, 1>(b.w[e], ts, sc);
        w[2] = decode_quarter<F, -1, J, 2>(b.w[e], ts, sc);
        w[3] = decode_quarter<F, -1, J, 3>(b.w[e], ts, sc);
#pragma unroll
        for (int t = 0; t < kRT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, b.x[t][e][J]),
                                                           acc[t], 0, 0, 0);
      });
  };

  Blk ring[kDepth];
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(ring[i], wk + i * kWK);
  for (int kb = wk; kb < nb; kb += kDepth * kWK) {
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (kb + i * kWK < nb) multiply(ring[i]);
      load(ring[i], kb + (kDepth + i) * kWK);
    }
  }

  if constexpr (kWK > 1) {
    __syncthreads();                                             // group ends read
#pragma unroll
    for (int t = 0; t < kRT; ++t) sh.sum[wave][t][lane] = acc[t];
    __syncthreads();
    if (wk != 0) return;
#pragma unroll
    for (int w = 1; w < kWK; ++w) {
#pragma unroll
      for (int t = 0; t < kRT; ++t) {
        const f32x4 o = sh.sum[wave + w][t][lane];
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[t][d] += o[d];
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kRT; ++t)
    if (p0 + r + 16 * t < pend && n0 < p.Qtot)
      *reinterpret_cast<u32x2*>(p.C + (int64_t)(p0 + r + 16 * t) * p.ldc + n0 + 4 * h) =
          u32x2{pack_bf16x2(acc[t][0], acc[t][1]), pack_bf16x2(acc[t][2], acc[t][3])};
}

int64_t row_tiles(const Params& p, int rows) {
  return p.offsets ? p.Ptot / rows + p.groups : (p.Ptot + rows - 1) / rows;
}

template <int F, int kWK, int kRT>
hipError_t launch(W4Args a, hipStream_t s) {
  const int64_t rt = row_tiles(a.p, 16 * kRT), cols = 16 * kWaves / kWK;
  a.row_tiles = (int32_t)rt;
  const int64_t nt = ((a.p.Qtot + cols - 1) / cols + 7) / 8 * 8;
  w4_kernel<F, kWK, kRT><<<dim3((uint32_t)(rt * nt)), dim3(64 * kWaves), 0, s>>>(a);
  return hipGetLastError();
}

template <int F>
hipError_t launch_split(const W4Args& a, hipStream_t s) {
  const int64_t waves = row_tiles(a.p, 16) * ((a.p.Qtot + 15) / 16);
  if (a.p.offsets != nullptr)
    return waves >= 4096 ? launch<F, 1, 1>(a, s) : waves >= 1024 ? launch<F, 4, 1>(a, s) : launch<F, 8, 1>(a, s);
  return waves <= kCUs       ? launch<F, 8, 1>(a, s)
         : waves <= 2 * kCUs ? launch<F, 4, 1>(a, s)
         : waves <= 4 * kCUs ? launch<F, 2, 1>(a, s)
                             : launch<F, 1, 1>(a, s);
}

}  // namespace

// (A launch has fewer than 2^32 threads.)
bool w4_fits(const Params& p) {
  if (p.offsets != nullptr)
    return p.Ptot <= 8 * (int64_t)p.groups && row_tiles(p, 16) * (p.Qtot / 16 + 1) < (int64_t)1 << 25;
  return p.Ptot <= 64;
}

hipError_t w4_fwd(const Params& prm, int fmt_w, hipStream_t s) {
  const W4Args a{prm, 0};
  return fmt_w == LP_MXFP4 ? launch_split<MXFP4>(a, s) : launch_split<NVFP4>(a, s);
}

}  // namespace gk
}  // namespace lp
