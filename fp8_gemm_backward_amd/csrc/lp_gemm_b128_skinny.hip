// Forward y = x @ W^T of few rows: FP8 operands with fp32 scales per 128,
// dense and grouped (single tokens, small decoding batches, a few rows per
// expert).
//
// The weight is read once and everything else is small, so the call is a
// stream over W.  A wave owns 16 columns of y (16 rows of W), up to 16 kRT rows
// of x and every kWK-th 128-deep block of the contraction, which it takes
// straight from global memory into the operand registers of
// v_mfma_f32_16x16x128_f8f6f4 (no LDS: nothing is shared), kDepth blocks in
// flight.  Each block's product is multiplied by its two scales and added in
// fp32; the sums of the kWK waves that share 16 columns are added in wave
// order at the end, so the result does not depend on timing.
//
// Bound by HBM where the weight is large (96 tokens over 64 experts of 2048 x
// 7168: 95 us, 4.8 TB/s of weights), by latency otherwise: 8 x 4096 x 4096
// 7.7 us with the weight in HBM, of which 3.4 are its bytes, about two the launch
// and the rest the first loads' way there and back and the joint sums.
//
// kFuse (at most kFuseRows rows, dense): x comes as bf16 and every workgroup
// quantizes it into LDS by the rule of lp_r128.hpp (a few KiB, read from L2)
// while its first weight loads are in flight, which saves the quantizer's
// launch.
#include "lp_gemm_b128_kernel.hpp"
#include "lp_r128.hpp"

namespace lp {
namespace gk {
namespace {

constexpr int kWaves = 8;
constexpr int kFuseLds = 64 * 1024;             // codes of a fused x

struct SkinnyArgs {
  Params p;
  const uint16_t* x;                            // bf16 x (kFuse)
  int32_t row_tiles;                            // row tiles of the grid
};

template <int kRT>
struct Block {                                  // one contraction block's operands
  u32x4 w[2], x[kRT][2];
  float sw, sx[kRT];
};

__device__ __forceinline__ float bload_f32(Rsrc r, int32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}

template <int kWK, bool kFuse, int kRT>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(kRT > 1 ? 2 : 4))) void b128_skinny(SkinnyArgs a) {
  constexpr int kRows = 16 * kRT, kDepth = 4;
  using Blk = Block<kRT>;
  const Params& p = a.p;
  constexpr int WN = kWaves / kWK;
  __shared__ union {
    int32_t ends[kMaxGroups];
    f32x4 sum[kWK == 1 ? 1 : kWaves][kRT][64];
  } sh;
  extern __shared__ __attribute__((aligned(16))) uint8_t xq[];   // kFuse: scales [blocks][kFuseRows], codes [rows][K]
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

  const int K = p.Ktot, nb = n0 < p.Qtot ? (K + kRun - 1) / kRun : 0;   // no block for columns past the end
  const int r = lane & 15, h = lane >> 4;
  const Rsrc wr = make_rsrc(p.Q.codes + (int64_t)g * p.Q.code_batch + (int64_t)n0 * K, (int64_t)16 * K);
  const Rsrc xr = make_rsrc(p.P.codes + (int64_t)p0 * K, (int64_t)(pend - p0) * K);
  const Rsrc swr = make_rsrc(p.Q.scales + (int64_t)g * p.Q.scale_batch + (int64_t)(n0 / kRun) * p.Q.scale_ld, p.Q.scale_ld);
  const uint8_t* const sxp = p.P.scales + (int64_t)p0 * 4;
  float* const xs = reinterpret_cast<float*>(xq);
  const int nbk = (K + kRun - 1) / kRun;

  // Block kb of the contraction; blocks and columns past the end read as zero.
  auto load = [&](Blk& b, int kb) {
    const int k0 = kb * kRun + 16 * h;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool in = kb < nb && k0 + 64 * e < K;
      b.w[e] = bload16(wr, in ? r * K + k0 + 64 * e : kOOB);
      if constexpr (!kFuse) {
#pragma unroll
        for (int t = 0; t < kRT; ++t) b.x[t][e] = bload16(xr, in ? (r + 16 * t) * K + k0 + 64 * e : kOOB);
      }
    }
    b.sw = bload_f32(swr, kb < nb ? 4 * kb : kOOB);
    if constexpr (!kFuse) {
      const Rsrc sxr = make_rsrc(sxp + (int64_t)kb * p.P.scale_ld, kb < nb ? (int64_t)(pend - p0) * 4 : 0);
#pragma unroll
      for (int t = 0; t < kRT; ++t) b.sx[t] = bload_f32(sxr, (r + 16 * t) * 4);
    }
  };

  f32x4 acc[kRT] = {};
  auto multiply = [&](Blk& b, int kb) {
    if constexpr (kFuse) {
      const int row = r < pend - p0 ? r : 0;                     // rows past the end: not stored
      const uint8_t* src = xq + 4 * kFuseRows * nbk + row * nbk * kRun + kb * kRun + 16 * h;
#pragma unroll
      for (int e = 0; e < 2; ++e) b.x[0][e] = *reinterpret_cast<const u32x4*>(src + 64 * e);
      b.sx[0] = xs[kb * kFuseRows + row];
    }
#pragma unroll
    for (int t = 0; t < kRT; ++t) {
      i32x8b w, x;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        w[d] = (int)b.w[d / 4][d % 4];
        x[d] = (int)b.x[t][d / 4][d % 4];
      }
      const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{}, 0, 0, 0, 0, 0, 0);
      const float s = b.sx[t] * b.sw;
#pragma unroll
      for (int d = 0; d < 4; ++d) acc[t][d] = __builtin_fmaf(part[d], s, acc[t][d]);
    }
  };

  Blk ring[kDepth];
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(ring[i], wk + i * kWK);
  if constexpr (kFuse) {
    // Sixteen lanes quantize a run, as the quantizer does.
    const int rows = pend - p0, runs = rows * nbk;
    for (int u = tid / 16; u < runs; u += 4 * kWaves) {
      const int row = u / nbk, kb = u - row * nbk, k = kb * kRun + 8 * (tid & 15);
      const u32x4 v = k < K ? *reinterpret_cast<const u32x4*>(a.x + (int64_t)(p0 + row) * K + k) : u32x4{0u, 0u, 0u, 0u};
      const RunScale q = run_scale(row16_max(amax8(v)));
      u32x2 c = run_codes8(v, q);
      if (k >= K) c = u32x2{0u, 0u};
      *reinterpret_cast<u32x2*>(xq + 4 * kFuseRows * nbk + row * nbk * kRun + k) = c;
      if ((tid & 15) == 0) xs[kb * kFuseRows + row] = q.s;
    }
    __syncthreads();
  }
  for (int kb = wk; kb < nb; kb += kDepth * kWK) {
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (kb + i * kWK < nb) multiply(ring[i], kb + i * kWK);
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

template <int kWK, bool kFuse, int kRT>
hipError_t launch(SkinnyArgs a, size_t lds, hipStream_t s) {
  const int64_t rt = row_tiles(a.p, 16 * kRT), cols = 16 * kWaves / kWK;
  a.row_tiles = (int32_t)rt;
  const int64_t nt = ((a.p.Qtot + cols - 1) / cols + 7) / 8 * 8;
  b128_skinny<kWK, kFuse, kRT><<<dim3((uint32_t)(rt * nt)), dim3(64 * kWaves), lds, s>>>(a);
  return hipGetLastError();
}
// Waves over the columns, kWK to each: dense, as many as make one workgroup per
// CU (1 x 16384 x 1024 7.6 us with 2, 9.8 with 4; 8 x 8192 x 2048 7.6 with 4, 9.9 with
// 8; 8 x 4096 x 2048 6.4 with 8, 7.0 with 4).  Grouped, whose row tiles the host only
// bounds, 4 or 8 until the waves are many (16 rows in 8 groups, 2048 x 4096: 18.9
// us with 4, 26.5 with 1).
template <bool kFuse, int kRT>
hipError_t launch_split(const SkinnyArgs& a, size_t lds, hipStream_t s) {
  const int64_t waves = row_tiles(a.p, 16 * kRT) * ((a.p.Qtot + 15) / 16);
  if (a.p.offsets != nullptr)
    return waves >= 4096   ? launch<1, kFuse, kRT>(a, lds, s)
           : waves >= 1024 ? launch<4, kFuse, kRT>(a, lds, s)
                           : launch<8, kFuse, kRT>(a, lds, s);
  return waves <= kCUs       ? launch<8, kFuse, kRT>(a, lds, s)
         : waves <= 2 * kCUs ? launch<4, kFuse, kRT>(a, lds, s)
         : waves <= 4 * kCUs ? launch<2, kFuse, kRT>(a, lds, s)
                             : launch<1, kFuse, kRT>(a, lds, s);
}

}  // namespace

hipError_t b128_fwd_fused(const Params& prm, const void* x, hipStream_t s) {
  const size_t nb = ((size_t)prm.Ktot + kRun - 1) / kRun;
  const size_t lds = nb * (4 * kFuseRows + (size_t)prm.Ptot * kRun);
  return launch_split<true, 1>(SkinnyArgs{prm, static_cast<const uint16_t*>(x), 0}, lds, s);
}

// Whether 32 rows a wave rather than 16: where 16 would make more waves than
// there are CUs.
static bool wide_rows(const Params& p) {
  return p.offsets == nullptr && p.Ptot > 16 && row_tiles(p, 16) * ((p.Qtot + 15) / 16) > kCUs;
}

// Up to 16 rows, 8 in a group's mean, or 64 rows of few columns, always at
// most one wave a column tile and CU: the tiles of 64 x 64 would leave most CUs
// idle, and each of theirs has the whole contraction to go through.  (Weights
// from HBM: 32 x 4096 x 4096 10.7 us by 32 rows a wave, 11.5 by 16, 14.4 on tiles; 64 x
// 2048 x 7168 15.3, 17.2, 22.3; 32 x 2048 x 7168 15.5, 10.9, 22.0; more waves: 32 x 8192 x
// 2048 10.4, 11.4, 9.6.  64 experts of 2048 x 7168: 512 tokens 196 to 235 us against 249 to
// 259 on 128 x 128 tiles, 1024 tokens 330 against 262.)
bool b128_skinny_fits(const Params& p) {
  if (p.offsets != nullptr)                                      // (a launch has fewer than 2^32 threads)
    return p.Ptot <= 8 * (int64_t)p.groups && row_tiles(p, 16) * (p.Qtot / 16 + 1) < (int64_t)1 << 25;
  return p.Ptot <= 16 || (p.Ptot <= 64 && row_tiles(p, 32) * ((p.Qtot + 15) / 16) <= kCUs);
}

hipError_t b128_fwd_skinny(const Params& prm, hipStream_t s) {
  const SkinnyArgs a{prm, nullptr, 0};
  return wide_rows(prm) ? launch<8, false, 2>(a, 0, s) : launch_split<false, 1>(a, 0, s);
}

}  // namespace gk

bool fwd_dyn_fuses(int64_t M, int64_t K, bool grouped) {
  return !grouped && M <= gk::kFuseRows && M * ((K + gk::kRun - 1) / gk::kRun) * gk::kRun <= gk::kFuseLds;
}

}  // namespace lp
