// Products of E4M3 operands with fp32 scales per 128 contraction elements,
// on gfx950's FP8 MFMA.
//
// An activation or gradient has one scale per run of 128 along the
// contraction (LP_FP8_R128), a weight one per 128 x 128 block (LP_FP8_B128).
// Within one 128-deep block b of the contraction every scale is constant
// along the contraction, so it leaves the inner sum:
//
//   fwd: y[m][n]  = sum_b sx[b][m] * sw[n/128][b] * sum_{k in b} cx[m][k] cw[n][k]
//   dX:  dx[m][k] = sum_b sg[b][m] * sw[b][k/128] * sum_{n in b} cg[m][n] cw[n][k]
//   dW:  dw[n][k] = sum_b sg[b][n] * sx[b][k]     * sum_{m in b} cg[m][n] cx[m][k]
//
// The inner sum is one v_mfma_f32_16x16x128_f8f6f4 into a fresh fp32
// accumulator (E4M3 products are exact in fp32); the outer sum is an fp32
// multiply-add per result.  The scales are general fp32 numbers, which the
// block-scaled MFMA (powers of two) cannot apply.
//
// Cost per 16 x 16 x 128: 32 MFMA cycles and 4 multiply-adds (16 cycles of
// the vector ALU, which runs beside the matrix core); grad_W, whose scales
// vary along both sides of the tile, needs 4 more multiplies.  The running
// sums must be ordinary vector registers (vector instructions cannot use
// accumulation registers), which sets the tile shape: 256 x 256 outputs by
// eight waves of 128 x 64 (128 registers of sums, two waves per SIMD), or,
// for few tiles, 128 x 128 by four waves of 64 x 64.
//
// A 128-deep stage of both operands and its scales goes from global memory
// straight into LDS, two stages deep; one barrier per stage.  LDS layouts:
// * contraction contiguous in memory (x and W in fwd, the gradient in dX):
//   [row][128 B], 16-byte chunk c of row r at c ^ ((r >> 1) & 7);
// * contraction along the rows (W in dX, both operands in dW): [k][columns],
//   read with the transposing ds_read_b64_tr_b8, whose 32 lanes read rows
//   n0 .. n0+7 and n0+16 .. n0+23 of one chunk; chunk c of row n is at
//   c ^ swz_cols(n), which puts them in distinct 16-byte slots of 256 bytes.
// Lane l of the MFMA holds row (column) l % 16 of its operand and, h = l / 16,
// the contraction bytes 16 h .. + 15 and 64 + 16 h .. + 15.  Any order inside
// the instruction gives the same sum as long as both operands use it; this one
// reads neighbouring 16-byte chunks in neighbouring lane rows, because the
// 16 lanes that a 16-byte LDS read serves together are 0-3, 12-15, 20-27 (and
// so on): with chunks 2 h and 2 h + 1 instead, 45% of the LDS cycles of the
// forward were bank conflicts.  The result is D[q][p]: lane l holds column
// p = l % 16 and rows q = 4 (l / 16) .. + 3.
#pragma once

#include "lp_gemm_kernel.hpp"

namespace lp {
namespace gk {

typedef int i32x8b __attribute__((ext_vector_type(8)));
typedef int i32x2b __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2b lds_i32x2b;

enum : int { kB128Fwd = 0, kB128Dx = 1, kB128Dw = 2 };

constexpr int kRun = 128;                       // contraction elements per scale

template <int kBP, int kBQ, int kWP, int kWQ>
struct BCfg {
  static constexpr int BP = kBP, BQ = kBQ, WP = kWP, WQ = kWQ;
  static constexpr int NWQ = BQ / WQ, NW = (BP / WP) * NWQ;
  static constexpr int FP = WP / 16, FQ = WQ / 16;
  static constexpr int PB = BP * kRun / 1024 / NW, QB = BQ * kRun / 1024 / NW;   // 1 KiB loads per wave and stage
  static constexpr int kP = 0, kQ = BP * kRun, kPS = kQ + BQ * kRun, kQS = kPS + BP * 4;
  static constexpr int STAGE = kQS + BQ * 4;
  static_assert(NW == BP / 64 + BQ / 64, "one scale load per wave");
  static_assert(PB == 4 && QB == 4, "load offsets are written for four blocks per wave and operand");
};
using B256 = BCfg<256, 256, 128, 64>;
using B128 = BCfg<128, 128, 64, 64>;

// Chunk swizzle of a [k][kCols bytes] tile (see above).
template <int kCols>
__device__ __forceinline__ int swz_cols(int n) {
  return (kCols == 256 ? 2 * (n & 7) : 2 * ((n >> 1) & 3)) ^ ((n >> 4) & 1);
}

// Direct loads of one operand.  kKMajor: kMN rows of 128 bytes; otherwise
// 128 rows of kMN bytes.
template <bool kKMajor, int kMN>
struct B128Loader {
  const uint8_t* base;      // first byte of the tile's rows (k-major) or of the tensor's group
  int64_t bytes;            // k-major: bytes from base to the end of the tile's rows
  int32_t ld;
  int32_t off[2];           // lane offset of blocks of either parity (128 columns: of blocks 0, 1 and 2, 3)
  int32_t kcol[2];          // k-major: the lane's first column in the stage
  static constexpr int kStep = !kKMajor && kMN == 128 ? 2 : 1;   // blocks between the two offsets
  int32_t lds;

  __device__ __forceinline__ void init(const Op& op, int g, int mn0, int mnend, int wave, int lane) {
    ld = op.code_ld;
    lds = 4096 * wave;
    if constexpr (kKMajor) {
      base = op.codes + (int64_t)g * op.code_batch + (int64_t)mn0 * ld;
      bytes = (int64_t)(mnend - mn0) * ld;
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int row = 8 * (4 * wave + o) + lane / 8;
        kcol[o] = 16 * ((lane & 7) ^ ((row >> 1) & 7));
        off[o] = row * ld + kcol[o] - 8 * o * ld;                 // + 8 u ld
      }
    } else {
      base = op.codes + (int64_t)g * op.code_batch;
      bytes = 0;
      constexpr int LPR = kMN / 16, RPB = 64 / LPR;               // lanes per row, rows per block
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int n = RPB * (4 * wave + kStep * o) + lane / LPR;
        kcol[o] = 0;
        off[o] = (n - RPB * kStep * o) * ld + mn0 + 16 * ((lane % LPR) ^ swz_cols<kMN>(n));
      }
    }
  }
  // Block u of the stage [k0, k0 + 128); what lies at or past kend reads as zero.
  template <int u>
  __device__ __forceinline__ void load(uint8_t* dst, int k0, int kend) const {
    if constexpr (kKMajor) {
      const Rsrc r = make_rsrc(base + k0, bytes - k0);
      dma<16>(r, (lds_void*)(dst + lds + 1024 * u), k0 + kcol[u & 1] >= kend ? kOOB : off[u & 1], 8 * u * ld);
    } else {
      const Rsrc r = make_rsrc(base + (int64_t)k0 * ld, (int64_t)(kend - k0) * ld);
      dma<16>(r, (lds_void*)(dst + lds + 1024 * u), off[u / kStep & 1], (1024 / kMN) * u * ld);
    }
  }
};

// Fragment reads of one operand: 16 rows (columns) x 128.
template <bool kKMajor, int kMN>
struct B128Frag {
  int32_t a;
  __device__ __forceinline__ void init(int mn, int lane) {       // mn: the wave's first row (column), a multiple of 64
    const int r = lane & 15, h = lane >> 4;
    if constexpr (kKMajor) {
      a = (mn + r) * kRun + 16 * (h ^ ((r >> 1) & 7));
    } else {
      const int n = 16 * h + r / 2;
      a = n * kMN + 16 * ((mn / 16) ^ swz_cols<kMN>(n)) + 8 * (r & 1);
    }
  }
  template <int f>
  __device__ __forceinline__ i32x8b read(const uint8_t* tile) const {
    i32x8b v;
    if constexpr (kKMajor) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(tile + (a ^ (64 * e)) + f * 16 * kRun);
#pragma unroll
        for (int d = 0; d < 4; ++d) v[4 * e + d] = (int)x[d];
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const i32x2b x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2b*)(tile + (a ^ (16 * f)) + (64 * (t / 2) + 8 * (t % 2)) * kMN));
        v[2 * t] = x[0];
        v[2 * t + 1] = x[1];
      }
    }
    return v;
  }
};

template <class C, int kOp>
__global__ __launch_bounds__(64 * C::NW) __attribute__((amdgpu_waves_per_eu(2, 2))) void b128_kernel(Params p) {
  constexpr bool kDW = kOp == kB128Dw;
  constexpr bool kPK = !kDW, kQK = kOp == kB128Fwd;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * C::STAGE];
  static_assert(kMaxGroups * 4 <= C::STAGE, "group ends alias stage 0");
  static_assert(C::BP * C::BQ * 2 <= 2 * C::STAGE, "the epilogue staging fits the stages");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wp = wave / C::NWQ, wq = wave % C::NWQ;
  Tile t = select_tile<C, kDW>(p, reinterpret_cast<int32_t*>(smem));
  if (!t.valid) return;
  // The same in every lane, which the compiler cannot see through the LDS
  // reads behind it: in scalar registers from here on.
  for (int* v : {&t.g, &t.p0, &t.pend, &t.q0, &t.kbeg, &t.kend}) *v = __builtin_amdgcn_readfirstlane(*v);
  __syncthreads();                                               // group ends read; stage 0 reusable

  const int kbeg = t.kbeg, kend = t.kend;
  B128Loader<kPK, C::BP> lp;
  B128Loader<kQK, C::BQ> lq;
  lp.init(p.P, 0, t.p0, t.pend, wave, lane);
  lq.init(p.Q, kDW ? 0 : t.g, t.q0, p.Qtot, wave, lane);

  // Scales of the stage, one fp32 per row of the P tile then one per column
  // of the Q tile, 64 a wave.
  const bool sp_wave = wave < C::BP / 64;
  const int64_t run0 = kDW ? (kbeg / kRun + t.g) : 0;            // first scale row of the contraction
  const int sv = sp_wave ? wave : wave - C::BP / 64;
  const uint8_t* sbase;
  int64_t sstep;                                                 // bytes per stage
  int32_t soff;
  int64_t slen;
  if (sp_wave || kDW) {
    const Op& o = sp_wave ? p.P : p.Q;
    const int first = (sp_wave ? t.p0 : t.q0) + 64 * sv;
    sbase = o.scales + run0 * o.scale_ld;
    sstep = o.scale_ld;
    soff = (first + lane) * 4;
    slen = o.scale_ld;
  } else {
    const int qb = (t.q0 + 64 * sv) / kRun;                      // the 128-column block of these 64 columns
    sbase = p.Q.scales + (int64_t)t.g * p.Q.scale_batch + (kQK ? (int64_t)qb * p.Q.scale_ld : 0);
    sstep = kQK ? 4 : p.Q.scale_ld;
    soff = kQK ? 0 : qb * 4;
    slen = kQK ? (qb * kRun < p.Qtot ? 4 : 0) : p.Q.scale_ld;
  }

  const int nk = (kend - kbeg + kRun - 1) / kRun;
  // Load u of stage kb: blocks of P, blocks of Q, scales.  Stages at or past
  // the end of the contraction read nothing (zeros).
  constexpr int kLoads = C::PB + C::QB + 1;
  auto issue = [&](auto ui, uint8_t* sb, int kb) {
    constexpr int u = decltype(ui)::value;
    const int k0 = kbeg + kb * kRun;
    if constexpr (u < C::PB) lp.template load<u>(sb + C::kP, k0, kend);
    else if constexpr (u < C::PB + C::QB) lq.template load<u - C::PB>(sb + C::kQ, k0, kend);
    else dma<4>(make_rsrc(sbase + kb * sstep, kb < nk ? slen : 0), (lds_void*)(sb + C::kPS + 256 * wave), soff, 0);
  };

  B128Frag<kPK, C::BP> fp;
  B128Frag<kQK, C::BQ> fq;
  fp.init(wp * C::WP, lane);
  fq.init(wq * C::WQ, lane);
  const int psa = C::kPS + (wp * C::WP + (lane & 15)) * 4;
  const int qsa = C::kQS + (wq * C::WQ + (kDW ? 4 * (lane >> 4) : 0)) * 4;

  f32x4 acc[C::FP][C::FQ];
#pragma unroll
  for (int i = 0; i < C::FP; ++i)
#pragma unroll
    for (int j = 0; j < C::FQ; ++j) acc[i][j] = f32x4{};

  // One stage: FP x FQ MFMAs (rows of FQ), the products of MFMA m added to
  // the sums after MFMA m + kLag has been issued.  P fragments are read kAhead
  // rows early; once the stage's last one is in registers, in row kSync, one
  // barrier says both that every wave is done with this buffer and that the
  // next stage has landed.  The rows that remain cover the next stage's first
  // reads: P's first fragments and each Q fragment after its last MFMA.  The
  // loads of the stage after that go into this buffer, one per MFMA from the
  // barrier on: a wave that issues them in one go waits for the memory
  // pipeline to take them, with its MFMAs behind them.
  constexpr int kLag = 2, kRing = kLag + 1, NM = C::FP * C::FQ;
  constexpr int kAhead = 1, kSlots = 2 * kAhead, kSync = C::FP - kAhead;
  constexpr int kEarly = NM - kSync * C::FQ < kLoads ? NM - kSync * C::FQ : kLoads;   // loads before the stage's end
  static_assert(C::FP % kSlots == 0, "a row's slot is the same in every stage");
  i32x8b q[C::FQ], pf[kSlots];
  if (nk > 0) {
    static_for<kLoads>([&](auto u) { issue(u, smem, 0); });
    static_for<kEarly>([&](auto u) { issue(u, smem + C::STAGE, 1); });
    barrier_vm<kEarly>();
    static_for<kAhead>([&](auto i) { pf[decltype(i)::value] = fp.template read<decltype(i)::value>(smem + C::kP); });
    static_for<C::FQ>([&](auto j) { q[decltype(j)::value] = fq.template read<decltype(j)::value>(smem + C::kQ); });
  }
  int cur = 0;
  for (int kb = 0; kb < nk; ++kb) {
    uint8_t* const sb = smem + cur;
    uint8_t* const nx = smem + (C::STAGE - cur);
    float sp[C::FP], w;
    f32x4 sq[kDW ? C::FQ : 1];
#pragma unroll
    for (int i = 0; i < C::FP; ++i) sp[i] = *reinterpret_cast<const float*>(sb + psa + 64 * i);
    if constexpr (kDW) {
#pragma unroll
      for (int j = 0; j < C::FQ; ++j) sq[j] = *reinterpret_cast<const f32x4*>(sb + qsa + 64 * j);
    } else {
      w = *reinterpret_cast<const float*>(sb + qsa);
    }
    f32x4 part[kRing];
    static_for<NM + kLag>([&](auto mi) {
      constexpr int m = decltype(mi)::value;
      constexpr int i = m / C::FQ, j = m % C::FQ;
      if constexpr (m == kSync * C::FQ) barrier_vm<0>();
      if constexpr (m < NM) {
        if constexpr (j == 0) {
          constexpr int n = i + kAhead;
          if constexpr (n < C::FP) pf[n % kSlots] = fp.template read<n>(sb + C::kP);
          else pf[n % kSlots] = fp.template read<n - C::FP>(nx + C::kP);
        }
        part[m % kRing] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[j], pf[i % kSlots], f32x4{}, 0, 0, 0, 0, 0, 0);
        if constexpr (i == C::FP - 1) q[j] = fq.template read<j>(nx + C::kQ);
        if constexpr (m >= kSync * C::FQ && m - kSync * C::FQ < kEarly) {
          issue(IC<m - kSync * C::FQ>{}, sb, kb + 2);
        }
        if constexpr (m < kLoads - kEarly) {
          issue(IC<m + kEarly>{}, nx, kb + 1);
        }
      }
      if constexpr (m >= kLag) {
        constexpr int d = m - kLag, di = d / C::FQ, dj = d % C::FQ;
        if constexpr (!kDW && dj == 0) sp[di] *= w;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float f = kDW ? sp[di] * sq[kDW ? dj : 0][r] : sp[di];
          acc[di][dj][r] = __builtin_fmaf(part[d % kRing][r], f, acc[di][dj][r]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    cur = C::STAGE - cur;
  }
  barrier_vm<0>();                                               // the last loads (zeros) have landed

  // bf16 results through LDS, so that each row of the wave tile is stored as
  // one 128-byte line: 8-byte slot s of row r at s ^ (r & 15).
  constexpr int ROWB = C::WQ * 2;
  static_assert(ROWB == 128, "one line per row");
  uint8_t* const stg = smem + wave * (C::WP * ROWB);
#pragma unroll
  for (int i = 0; i < C::FP; ++i) {
    const int r = lane & 15;
#pragma unroll
    for (int j = 0; j < C::FQ; ++j) {
      const int slot = 4 * j + (lane >> 4);
      *reinterpret_cast<u32x2*>(stg + (16 * i + r) * ROWB + 8 * (slot ^ r)) =
          u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
    }
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);                            // lgkmcnt(0): own staging writes done
  uint16_t* const out = p.C + (kDW ? (int64_t)t.g * p.c_batch : 0);
  const int c16 = lane & 7, col = t.q0 + wq * C::WQ + 8 * c16;
#pragma unroll 4
  for (int it = 0; it < C::WP / 8; ++it) {
    const int r = 8 * it + lane / 8;
    const u32x2 lo = *reinterpret_cast<const u32x2*>(stg + r * ROWB + 8 * ((2 * c16) ^ (r & 15)));
    const u32x2 hi = *reinterpret_cast<const u32x2*>(stg + r * ROWB + 8 * ((2 * c16 + 1) ^ (r & 15)));
    const int row = t.p0 + wp * C::WP + r;
    if (row < t.pend && col < p.Qtot)
      *reinterpret_cast<u32x4*>(out + (int64_t)row * p.ldc + col) = u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
}

template <class C, int kOp>
inline hipError_t run_b128(const Params& prm, hipStream_t s) {
  if (prm.ntiles <= 0) return hipSuccess;
  b128_kernel<C, kOp><<<dim3(prm.ntiles), dim3(64 * C::NW), 0, s>>>(prm);
  return hipGetLastError();
}

}  // namespace gk
}  // namespace lp
