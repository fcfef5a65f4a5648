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
// accumulator (E4M3 products are exact in fp32; inside the instruction the
// core aligns them and drops low bits, at most 2^-12.6 of their magnitudes' sum
// on random codes, 2^-11.8 where one product of 448 x 448 meets small ones); the outer sum is an fp32 multiply-add per result, rounded
// once, to bf16, when the contraction is done.  The scales are general fp32 numbers, which the
// block-scaled MFMA (powers of two) cannot apply.
//
// Cost per 16 x 16 x 128: 32 MFMA cycles and 4 multiply-adds (16 cycles of
// the vector ALU, which runs beside the matrix core); grad_W, whose scales
// vary along both sides of the tile, needs 4 more multiplies.  The running
// sums must be ordinary vector registers (vector instructions cannot use
// accumulation registers), which sets the tile shape: 256 x 256 outputs by
// eight waves of 128 x 64 (128 registers of sums, two waves per SIMD), or,
// for few tiles, 128 x 128 by two groups of four waves of 64 x 64, or 64 x 64 by
// four groups of two waves of 32 x 64; the groups of waves share the
// contraction.
//
// 8192 x 4096 outputs: 1.59 us (forward, grad_X) and 1.86 us (grad_W) per 128 deep
// stage and round of 256 tiles, 2.69 and 2.31 PFLOP/s asymptotically; with a contraction of 4096
// 117, 116 and 135 us (2.35, 2.37, 2.04 PFLOP/s).  A plain FP8 product of the vendor's
// library without block scales reaches 2.83 PFLOP/s at 8192^3.  Bound by the
// stages' loads, instruction issue and power: without the loads 3.6 PFLOP/s, about half
// of the difference by the clock (2.2 GHz, 1.9 with them), half by waiting.  The matrix
// cores are busy 46 to 55% of the time, LDS 27%, and the waves wait for a quarter of
// it.  Leaving out grad_W's 128 multiplies per wave and stage takes 272 us to 228 over
// a contraction of 8192.
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

template <int kBP, int kBQ, int kWP, int kWQ, int kStages, int kSplit = 1>
struct BCfg {
  static constexpr int NS = kStages;                             // LDS stages
  static constexpr int KW = kSplit;                              // groups of waves that share the contraction
  static constexpr int BP = kBP, BQ = kBQ, WP = kWP, WQ = kWQ;
  static constexpr int NWQ = BQ / WQ, NW = (BP / WP) * NWQ;
  static constexpr int FP = WP / 16, FQ = WQ / 16;
  static constexpr int PB = BP * kRun / 1024 / NW, QB = BQ * kRun / 1024 / NW;   // 1 KiB loads per wave and stage
  static constexpr int kP = 0, kQ = BP * kRun, kPS = kQ + BQ * kRun, kQS = kPS + BP * 4;
  static constexpr int STAGE = kQS + BQ * 4;
  static_assert(NW >= BP / 64 + BQ / 64, "one scale load per wave");
};
using B256 = BCfg<256, 256, 128, 64, 2>;
using B256N = BCfg<256, 128, 64, 64, 3>;
using B128 = BCfg<128, 128, 64, 64, 2, 2>;
using B64 = BCfg<64, 64, 32, 64, 2, 4>;

// Chunk swizzle of a [k][kCols bytes] tile (see above).
template <int kCols>
__device__ __forceinline__ int swz_cols(int n) {
  const int g = (n >> 4) & 1;
  return kCols == 256 ? 2 * (n & 7) ^ g : kCols == 128 ? 2 * ((n >> 1) & 3) ^ g : ((n >> 2) & 1) ^ (2 * g);
}

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>(((uint64_t)(uint32_t)scalar((int)(v >> 32)) << 32) | (uint32_t)scalar((int)v));
}

// The buffer resource of a window.  Its words must reach the loads' inline
// assembly from scalar arithmetic: a scalar register written by a vector
// instruction may be read by a memory instruction only five instructions
// later, which nothing checks inside inline assembly.  So a tile's addresses
// go through scalar() once, five instructions ahead of every load
// (scalars_settle), and move on by 32-bit steps.
__device__ __forceinline__ void scalars_settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 4");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ Rsrc window(const uint8_t* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, bytes > 0 ? bytes : 0, 0x00020000);
}

// Direct loads of one operand, stage by stage.  kKMajor: kMN rows of 128
// bytes; otherwise 128 rows of kMN bytes.  The buffer range of a stage is kept
// in 32-bit scalars that move on by one stage (a tile's rows span fewer than
// 2^31 bytes): computed anew with 64-bit clamps for every stage, it cost some
// 350 cycles a stage.
// kBlk: 1 KiB blocks per wave (2 or 4).
template <bool kKMajor, int kMN, int kBlk>
struct B128Loader {
  static_assert(kBlk == 2 || kBlk == 4, "the lane offsets below are written for these");
  const uint8_t* base;      // first byte of the stage's window
  int32_t bytes;            // k-major: bytes from base to the end of the tile's rows
  int32_t left;             // contraction elements from the stage's start to the end
  int32_t ld;
  int32_t mn;               // otherwise: the tile's first column
  int32_t off[2];           // lane offset of blocks of either parity (128 columns: of blocks 0, 1 and 2, 3)
  int32_t kcol;             // k-major: the lane's first column in the stage, even blocks (odd ones: ^ 64)
  int32_t lds;
  static constexpr int kStep = !kKMajor && kMN == 128 ? 2 : 1;   // blocks between the two offsets

  __device__ __forceinline__ void init(const Op& op, int wave, int lane) {
    ld = op.code_ld;
    lds = 1024 * kBlk * wave;
    kcol = 0;
    if constexpr (kKMajor) {
      const int row = 8 * kBlk * wave + lane / 8;
      kcol = 16 * ((lane & 7) ^ ((row >> 1) & 7));
      off[0] = row * ld + kcol;                                  // + 8 u ld
      off[1] = row * ld + (kcol ^ 64);
    } else {
      constexpr int LPR = kMN / 16, RPB = 64 / LPR;               // lanes per row, rows per block
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int n = RPB * (kBlk * wave + kStep * o) + lane / LPR;
        off[o] = (n - RPB * kStep * o) * ld + 16 * ((lane % LPR) ^ swz_cols<kMN>(n));
      }
    }
  }
  // To the first stage of a tile: rows (columns) mn0 .. of group g, contraction [kbeg, kend).
  __device__ __forceinline__ void start(const Op& op, int g, int mn0, int mnend, int kbeg, int kend) {
    asm volatile("" : "+s"(ld), "+s"(lds));                      // (keeps what follows from them out of the tile loop's registers)
    left = kend - kbeg;
    mn = mn0;
    base = scalar(op.codes + (int64_t)g * op.code_batch + (kKMajor ? (int64_t)mn0 * ld + kbeg : (int64_t)kbeg * ld + mn0));
    bytes = kKMajor ? scalar((mnend - mn0 < kMN ? mnend - mn0 : kMN) * ld - kbeg) : 0;
  }
  // Block u of the stage; what lies past the end of the contraction reads as zero.
  template <int u>
  __device__ __forceinline__ void load(uint8_t* dst) const {
    if constexpr (kKMajor) {
      const Rsrc r = window(base, bytes);
      dma<16>(r, (lds_void*)(dst + lds + 1024 * u), (kcol ^ (64 * (u & 1))) >= left ? kOOB : off[u & 1], 8 * u * ld);
    } else {
      // The rows that exist, 0 .. 128.  (Written as one expression, the clamp
      // to both ends becomes a vector instruction.)
      int rows;
      asm("s_min_i32 %0, %1, %2" : "=s"(rows) : "s"(left), "s"(kRun) : "scc");
      const Rsrc r = window(base, (rows > 0 ? rows : 0) * ld - mn);
      dma<16>(r, (lds_void*)(dst + lds + 1024 * u), off[u / kStep & 1], (1024 / kMN) * u * ld);
    }
  }
  // On by n stages.
  __device__ __forceinline__ void advance(int n) {
    left -= n * kRun;
    base += kKMajor ? (uint32_t)(n * kRun) : (uint32_t)(n * kRun * ld);
    bytes -= n * kRun;
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
      // (tile is a multiple of 256: one sum for all f, where a ^ 16 f would keep a register each)
      const uint32_t at = ((uint32_t)(uintptr_t)(lds_i32x2b*)tile + (uint32_t)a) ^ (16 * f);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const i32x2b x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2b*)(uintptr_t)(at + (64 * (t / 2) + 8 * (t % 2)) * kMN));
        v[2 * t] = x[0];
        v[2 * t + 1] = x[1];
      }
    }
    return v;
  }
};

// Params::tail (the host's choice to split by round): the whole rounds of kCUs
// tiles when the last, partial one has at most kCUs / 2, every tile otherwise;
// what that leaves is taken by a second launch in kParts parts of each
// 256 x 256 tile: 256 x 128, 128 x 128 or 64 x 64.
struct Rounds {
  int full, rest;
  bool split;
};
__device__ __forceinline__ Rounds rounds_of(const Params& p, int all) {
  const int full = all / kCUs * kCUs, rest = all - full;
  return Rounds{full, rest, p.tail != 0 && full > 0 && rest > 0 && 2 * rest <= kCUs};
}
// Workgroup hw's whole tile (-1: none) and part of it.
template <int kParts>
__device__ __forceinline__ int2 tile_of(const Params& p, int all, int hw) {
  const Rounds r = rounds_of(p, all);
  const int nt = kParts > 1 ? (r.split ? kParts * r.rest : 0) : r.split ? r.full : all;
  if (hw >= nt) return make_int2(-1, 0);
  const int i = xcd_remap(hw, nt);
  return kParts > 1 ? make_int2(r.full + i / kParts, i % kParts) : make_int2(i, 0);
}
template <class C, int kParts>
inline constexpr int kWholeRows = kParts > 1 ? 256 : C::BP;      // of a whole tile
template <class C, int kParts>
inline constexpr int kPartCols = kParts > 1 ? 256 / C::BQ : 1;   // parts side by side

// Row and column of tile i of a dense product.
__device__ __forceinline__ int2 dense_order(const Params& p, int rows, int i) {
  return p.gm > 1 ? grouped_order(i, (p.Ptot + rows - 1) / rows, p.nq, p.gm) : make_int2(i / p.nq, i % p.nq);
}

// Tiles of a dense product: a contiguous range for each XCD, in blocks that
// share operand rows and columns.  Params::splits workgroups share a tile's
// contraction, split_len elements each, and leave fp32 tiles (b128_join).
template <class C, int kParts>
__device__ __forceinline__ Tile dense_tile(const Params& p, int hw) {
  constexpr int kRows = kWholeRows<C, kParts>, kCols = kPartCols<C, kParts>;
  int split = 0;
  int2 w;
  if (kParts == 1 && C::KW > 1 && p.splits > 1) {                // the splits of a tile are neighbours
    const int i = xcd_remap(hw, p.ntiles * p.splits);
    w = make_int2(i / p.splits, 0);
    split = i - w.x * p.splits;
  } else {
    w = tile_of<kParts>(p, p.ntiles, hw);
    if (w.x < 0) return Tile{0, 0, 0, 0, 0, 0, 0, 0, false};
  }
  const int2 pq = dense_order(p, kRows, w.x);
  Tile t{0, pq.x * kRows + w.y / kCols * C::BP, p.Ptot, (pq.y * kCols + w.y % kCols) * C::BQ, 0, p.Ktot, w.x, split, false};
  t.valid = t.p0 < p.Ptot && t.q0 < p.Qtot;
  if (kParts == 1 && C::KW > 1 && p.splits > 1) {
    t.kbeg = split * p.split_len;
    t.kend = p.Ktot - t.kbeg < p.split_len ? p.Ktot : t.kbeg + p.split_len;
  }
  return t;
}

// Tiles of a grouped forward or grad_X.  Row tiles of 256 rows or less never
// straddle a group; the workgroups deal the tiles that exist (their number is
// known on the device only) to the eight XCDs in contiguous ranges, in each
// group's blocked order (grouped_order).  Dealing the host's upper bound
// instead leaves the last XCD idle: 16384 rows in 8 equal groups, 512 tiles
// bounded by 576, took 163 us for 124.
//
// Every wave scans 64 groups at a time, one a lane: the clamped ends are a
// running maximum, the row tiles before each group a running sum (wave_scan).
struct GroupScan {
  int start, end, seen;      // of this lane's group: first row, end row, row tiles before it
  int last_end, last_seen;   // after the 64 groups
};
template <int BP>
__device__ __forceinline__ GroupScan scan_groups(const Params& p, int M, int base, int end0, int seen0) {
  const int lane = threadIdx.x & 63;
  int e = base + lane < p.groups ? p.offsets[base + lane] : 0;
  e = e > M ? M : e;
  e = e < end0 ? end0 : e;
  e = wave_scan(e, [](int a, int b) { return a > b ? a : b; });
  int s = __shfl_up(e, 1);
  s = lane == 0 ? end0 : s;
  const int n = (e - s + BP - 1) / BP;
  const int sum = wave_scan(n, [](int a, int b) { return a + b; });
  return GroupScan{s, e, seen0 + sum - n, __builtin_amdgcn_readlane(e, 63), seen0 + __builtin_amdgcn_readlane(sum, 63)};
}

// sc0: the scan of at most 64 groups, unless there are more.
template <class C, int kParts>
__device__ __forceinline__ Tile grouped_tile(const Params& p, const GroupScan& sc0, int hw) {
  constexpr int kRows = kWholeRows<C, kParts>, kCols = kPartCols<C, kParts>;
  Tile t{0, 0, 0, 0, 0, p.Ktot, 0, 0, false};
  GroupScan sc = sc0;
  int end0 = 0, rows = sc0.last_seen;
  if (p.groups > 64) {
    rows = 0;
    for (int base = 0; base < p.groups; base += 64) {
      sc = scan_groups<kRows>(p, p.Ptot, base, end0, rows);
      end0 = sc.last_end;
      rows = sc.last_seen;
    }
  }
  const int nq = kParts > 1 ? (p.Qtot + 255) / 256 : p.nq;
  const int2 whole = tile_of<kParts>(p, rows * nq, hw);
  if (whole.x < 0) return t;
  const int tile = whole.x, part = whole.y;
  const int pidx = tile / nq;
  if (p.groups > 64) {
    end0 = rows = 0;
    for (int base = 0; base < p.groups; base += 64) {
      sc = scan_groups<kRows>(p, p.Ptot, base, end0, rows);
      if (pidx < sc.last_seen) {
        t.g = base;
        break;
      }
      end0 = sc.last_end;
      rows = sc.last_seen;
    }
  }
  // The last group with at most pidx row tiles before it: the later ones of
  // those are never empty.
  const int l = 63 - __builtin_clzll(__builtin_amdgcn_ballot_w64(sc.seen <= pidx && sc.end > sc.start));
  t.g += l;
  const int start = __builtin_amdgcn_readlane(sc.start, l), seen = __builtin_amdgcn_readlane(sc.seen, l);
  t.pend = __builtin_amdgcn_readlane(sc.end, l);
  int2 pq = make_int2(pidx - seen, tile - pidx * nq);
  if (p.gm > 1) pq = grouped_order(tile - seen * nq, (t.pend - start + kRows - 1) / kRows, nq, p.gm);
  t.p0 = start + pq.x * kRows + part / kCols * C::BP;
  t.q0 = (pq.y * kCols + part % kCols) * C::BQ;
  t.valid = t.q0 < p.Qtot && t.p0 < t.pend;
  return t;
}

// Tiles of a grouped grad_W over at most 64 groups, every group having the
// same number: longest contraction first (ties by group index), which keeps
// the last round short.  Inside a group each XCD takes one contiguous range of
// the tiles, row tiles fastest, so that it reads few of the group's gradient
// and input columns more than once.  rank: the lane's group's place.
__device__ __forceinline__ int size_rank(const GroupScan& sc, int groups) {
  const int lane = threadIdx.x & 63, size = sc.end - sc.start;
  int rank = 0;
  for (int j = 0; j < groups; ++j) rank += __builtin_amdgcn_readlane(size, j) >= size + (lane <= j);
  return rank;
}
template <class C>
__device__ __forceinline__ Tile grouped_dw_tile(const Params& p, const GroupScan& sc, int rank, int hw) {
  const int lane = threadIdx.x & 63;
  const int per = p.ntiles / p.groups, want = hw / per;
  const int g = __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < p.groups && rank == want));
  const int tile = xcd_remap(hw - want * per, per), np = per / p.nq;
  return Tile{g, (tile % np) * C::BP, p.Ptot, (tile / np) * C::BQ, __builtin_amdgcn_readlane(sc.start, g),
              __builtin_amdgcn_readlane(sc.end, g), 0, 0, true};
}

// Whether a launch's workgroups take one tile after another, 256 of them side
// by side: on 256 x 256 tiles, and where the tiles can be told from registers
// (no more than 64 groups).  The next tile's loads then start before a tile's
// results are stored, and groups are scanned once: grad_W of 64 experts of
// 2048 x 7168, 1024 rows 387 -> 335 us, 32768 rows 850 -> 779; their grad_X of
// 32768 rows 606 -> 585; dense 8192 x 4096 x 4096 forward 121.8 -> 117.4,
// grad_X 120.2 -> 115.9, grad_W 139.9 -> 134.9.
// A grouped grad_W's tiles differ in length, and dealt ahead (every other round in
// reverse) they end less evenly than dispatched one by one: from eight rounds
// on, or four when no group can have more than 32 stages.  (4096 rows, 5.5 rounds:
// 16 even groups of 2048 x 2816 72.6 us dispatched, 58.7 in turns, 32 skewed ones of 1024 x
// 2816 52.3, 48.2; but with 16384 rows 83.4, 100.2.  In reverse: 32 skewed groups of
// 2048 x 4096, 16384 rows, 226 -> 216.)
template <class C, int kOp>
__host__ __device__ __forceinline__ bool takes_turns(const Params& p) {
  if (C::KW > 1 || C::NS > 2 || (p.offsets != nullptr && p.groups > 64)) return false;
  const bool uneven = kOp == kB128Dw && p.offsets != nullptr;
  return p.ntiles > (!uneven ? 1 : p.Ktot <= 32 * kRun ? 4 : 8) * kCUs;
}

// LDS of this wave written and read, and every wave here (loads into the stages
// go on).
__device__ __forceinline__ void barrier_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <class C>
inline constexpr bool kOwnRowsOf = C::KW == 1 && C::NS == 2;     // results pass through LDS of their own, 2 KiB a wave
template <class C>
inline constexpr int kLdsOf = C::KW * C::NS * C::STAGE + (kOwnRowsOf<C> ? C::NW * 2048 : 0);

template <class C, int kOp, int kParts>
__device__ __forceinline__ void b128_tiles_of(const Params& p, uint8_t* all_smem) {
  constexpr bool kDW = kOp == kB128Dw;
  constexpr bool kPK = !kDW, kQK = kOp == kB128Fwd;
  constexpr bool kOwnRows = kOwnRowsOf<C>;
  static_assert(kMaxGroups * 4 <= C::STAGE, "group ends alias stage 0");
  static_assert(kOwnRows || C::BP * C::BQ * (C::KW > 1 ? 4 : 2) <= C::NS * C::STAGE, "the epilogue staging fits the stages");

  const int tid = threadIdx.x, lane = tid & 63;
  const int gwave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = gwave / C::NW, wave = gwave % C::NW;            // group, and wave in the group
  const int wp = wave / C::NWQ, wq = wave % C::NWQ;
  uint8_t* const smem = all_smem + kw * (C::NS * C::STAGE);      // the group's stages
  int32_t* const ends = reinterpret_cast<int32_t*>(all_smem);
  const bool turns = takes_turns<C, kOp>(p);
  GroupScan sc{};
  int rank = 0;
  if (p.offsets != nullptr && p.groups <= 64) {
    sc = scan_groups<kParts == 1 ? C::BP : 256>(p, kDW ? p.Ktot : p.Ptot, 0, 0, 0);
    if (kDW) rank = size_rank(sc, p.groups);
  }
  auto pick = [&](int hw) {                                      // of a dense product or at most 64 groups
    if (p.offsets == nullptr) return dense_tile<C, kParts>(p, hw);
    return kDW ? grouped_dw_tile<C>(p, sc, rank, hw) : grouped_tile<C, kParts>(p, sc, hw);
  };
  int hw = blockIdx.x, round = 0;
  Tile t;
  if (kDW && p.offsets != nullptr && p.groups > 64) {
    t = select_tile<C, kDW>(p, ends);
    __syncthreads();                                             // group ends read; stage 0 reusable
  } else {
    t = pick(hw);
  }
  if (!t.valid) return;

  B128Loader<kPK, C::BP, C::PB> lp;
  B128Loader<kQK, C::BQ, C::QB> lq;
  lp.init(p.P, wave, lane);
  lq.init(p.Q, wave, lane);

  // Scales of the stage, one fp32 per row of the P tile then one per column
  // of the Q tile, 64 a wave.
  const bool sp_wave = wave < C::BP / 64;
  const int sv = sp_wave ? wave : (wave - C::BP / 64) % (C::BQ / 64);   // (spare waves load a Q part once more)
  const uint8_t* sbase;                                          // of the stage
  uint32_t sstep;                                                // bytes per stage
  const int32_t soff = sp_wave || kDW ? lane * 4 : 0;            // lane offset
  int32_t slen;                                                  // bytes that exist
  auto begin = [&] {                                             // to tile t
    // The same in every lane, which the compiler cannot see: in scalar registers
    // from here on.
    for (int* v : {&t.g, &t.p0, &t.pend, &t.q0, &t.kbeg, &t.kend}) *v = scalar(*v);
    lp.start(p.P, 0, t.p0, t.pend, t.kbeg, t.kend);
    lq.start(p.Q, kDW ? 0 : t.g, t.q0, p.Qtot, t.kbeg, t.kend);
    lp.advance(kw);
    lq.advance(kw);
    const int64_t run0 = t.kbeg / kRun + (kDW ? t.g : 0);        // first scale row of the contraction
    if (sp_wave || kDW) {
      const int first = (sp_wave ? t.p0 : t.q0) + 64 * sv, cols = (sp_wave ? p.Ptot : p.Qtot) - first;
      sstep = sp_wave ? p.P.scale_ld : p.Q.scale_ld;
      sbase = (sp_wave ? p.P.scales : p.Q.scales) + run0 * sstep + (int64_t)first * 4;
      slen = (cols < 0 ? 0 : cols < 64 ? cols : 64) * 4;
    } else {
      const int qb = (t.q0 + 64 * sv) / kRun;                    // the 128-column block of these 64 columns
      sbase = p.Q.scales + (int64_t)t.g * p.Q.scale_batch + (kQK ? (int64_t)qb * p.Q.scale_ld : qb * 4);
      sstep = kQK ? 4 : p.Q.scale_ld;
      sbase += run0 * sstep;
      slen = qb * kRun < p.Qtot ? 4 : 0;
    }
    sbase += (uint64_t)kw * sstep;
    sbase = scalar(sbase);
    sstep = scalar((int)sstep) * C::KW;
    slen = scalar(slen);
    scalars_settle();
  };

  // Load u of the next stage to be loaded: blocks of P, blocks of Q, scales
  // (the last one moves on to the stage after).  Stages past the end of the
  // contraction read nothing (zeros).
  constexpr int kLoads = C::PB + C::QB + 1;
  auto issue = [&](auto ui, uint8_t* sb) {
    constexpr int u = decltype(ui)::value;
    if constexpr (u < C::PB) {
      lp.template load<u>(sb + C::kP);
    } else if constexpr (u < C::PB + C::QB) {
      lq.template load<u - C::PB>(sb + C::kQ);
    } else {
      const Rsrc r = window(sbase, lp.left > 0 ? slen : 0);
      dma<4>(r, (lds_void*)(sb + (sp_wave ? C::kPS : C::kQS) + 256 * sv), soff, 0);
      sbase += sstep;
      lp.advance(C::KW);
      lq.advance(C::KW);
    }
  };

  B128Frag<kPK, C::BP> fp;
  B128Frag<kQK, C::BQ> fq;
  fp.init(wp * C::WP, lane);
  fq.init(wq * C::WQ, lane);
  const int psa = C::kPS + (wp * C::WP + (lane & 15)) * 4;
  const int qsa = C::kQS + (wq * C::WQ + (kDW ? 4 * (lane >> 4) : 0)) * 4;

  // One stage: FP x FQ MFMAs (rows of FQ), the products of MFMA m added to
  // the sums after MFMA m + kLag has been issued.  P fragments are read kAhead
  // rows early; once the stage's last one is in registers, in row kSync, one
  // barrier says both that every wave is done with this buffer and that the
  // next stage has landed.  The rows that remain cover the next stage's first
  // reads: P's first fragments and each Q fragment after its last MFMA.  The
  // loads of stage kb + NS go into this buffer, one per MFMA from the barrier
  // on: a wave that issues them in one go waits for the memory
  // pipeline to take them, with its MFMAs behind them.
  constexpr int kLag = 2, kRing = kLag + 1, NM = C::FP * C::FQ;
  constexpr int kAhead = 1, kSlots = 2 * kAhead, kSync = C::FP - kAhead;
  constexpr int kEarly = NM - kSync * C::FQ < kLoads ? NM - kSync * C::FQ : kLoads;   // loads before the stage's end
  static_assert(C::FP % kSlots == 0, "a row's slot is the same in every stage");
  f32x4 acc[C::FP][C::FQ];
  int nk;                                                        // stages of a group of waves
  auto first_loads = [&] {
    nk = (t.kend - t.kbeg + C::KW * kRun - 1) / (C::KW * kRun);
    if (nk <= 0) return;
    static_for<C::NS - 1>([&](auto si) {
      constexpr int st = decltype(si)::value;
      static_for<kLoads>([&](auto u) { issue(u, smem + st * C::STAGE); });
    });
    static_for<kEarly>([&](auto u) { issue(u, smem + (C::NS - 1) * C::STAGE); });
  };
  begin();
  first_loads();
  bool stores_behind = false;                                    // the last tile's, 2 FP a wave, issued after the first loads
  for (;;) {
    int cur = 0;
    asm volatile("" : "+s"(cur));                                // (its multiples stay out of the registers of the tile loop)
    i32x8b q[C::FQ], pf[kSlots];
#pragma unroll
    for (int i = 0; i < C::FP; ++i)
#pragma unroll
      for (int j = 0; j < C::FQ; ++j) acc[i][j] = f32x4{};
    if (nk > 0) {
      constexpr int kWait = (C::NS - 2) * kLoads + kEarly;
      if (kOwnRows && stores_behind) barrier_vm<kWait + 2 * C::FP>();
      else barrier_vm<kWait>();
      static_for<kAhead>([&](auto i) { pf[decltype(i)::value] = fp.template read<decltype(i)::value>(smem + cur + C::kP); });
      static_for<C::FQ>([&](auto j) { q[decltype(j)::value] = fq.template read<decltype(j)::value>(smem + cur + C::kQ); });
    }
    for (int kb = 0; kb < nk; ++kb) {
      uint8_t* const sb = smem + cur;
      const int next = cur + C::STAGE < C::NS * C::STAGE ? cur + C::STAGE : 0;
      uint8_t* const nx = smem + next;
      uint8_t* const pv = smem + (cur > 0 ? cur - C::STAGE : (C::NS - 1) * C::STAGE);   // the stage before
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
      f32x4 part[kRing], fac{};
      static_for<NM + kLag>([&](auto mi) {
        constexpr int m = decltype(mi)::value;
        constexpr int i = m / C::FQ, j = m % C::FQ;
        if constexpr (m == kSync * C::FQ) barrier_vm<(C::NS - 2) * kLoads>();
        if constexpr (m < NM) {
          if constexpr (j == 0) {
            constexpr int n = i + kAhead;
            if constexpr (n < C::FP) pf[n % kSlots] = fp.template read<n>(sb + C::kP);
            else pf[n % kSlots] = fp.template read<n - C::FP>(nx + C::kP);
          }
          part[m % kRing] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q[j], pf[i % kSlots], f32x4{}, 0, 0, 0, 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (i == C::FP - 1) q[j] = fq.template read<j>(nx + C::kQ);
          if constexpr (m >= kSync * C::FQ && m - kSync * C::FQ < kEarly) {
            issue(IC<m - kSync * C::FQ>{}, sb);
          }
          // The rest of the stage begun in the row before, all ahead of the barrier,
          // which counts whole stages.
          if constexpr (m < kSync * C::FQ) {
            static_for<kLoads - kEarly>([&](auto li) {
              constexpr int l = decltype(li)::value;
              if constexpr ((l < kSync * C::FQ ? l : kSync * C::FQ - 1) == m) issue(IC<l + kEarly>{}, pv);
            });
          }
        }
        if constexpr (m >= kLag) {
          constexpr int d = m - kLag, di = d / C::FQ, dj = d % C::FQ;
          if constexpr (!kDW && dj == 0) sp[di] *= w;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float f = kDW ? fac[r] : sp[di];
            acc[di][dj][r] = __builtin_fmaf(part[d % kRing][r], f, acc[di][dj][r]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        // The next product's factors, one step ahead of their use (right before it:
        // 8192 x 4096 x 8192 272 us, 267).
        if constexpr (kDW && m + 1 >= kLag && m + 1 - kLag < NM) {
          constexpr int d = m + 1 - kLag;
#pragma unroll
          for (int r = 0; r < 4; ++r) fac[r] = sp[d / C::FQ] * sq[kDW ? d % C::FQ : 0][r];
          __builtin_amdgcn_sched_barrier(0);
        }
      });
      cur = next;
    }
    barrier_vm<0>();                                             // the last loads (zeros) have landed

    uint16_t* const out = p.C + (kDW ? (int64_t)t.g * p.c_batch : 0);
    if constexpr (C::KW > 1) {
      // The groups' sums through LDS, added in group order: 16-byte piece c of
      // row r of a group's tile at c ^ (r & 15).
      float* const mine = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int i = 0; i < C::FP; ++i)
#pragma unroll
        for (int j = 0; j < C::FQ; ++j) {
          const int r = wp * C::WP + 16 * i + (lane & 15), c = (wq * C::WQ) / 4 + 4 * j + (lane >> 4);
          *reinterpret_cast<f32x4*>(mine + r * C::BQ + 4 * (c ^ (r & 15))) = acc[i][j];
        }
      __syncthreads();
      for (int u = tid; u < C::BP * C::BQ / 8; u += 64 * C::NW * C::KW) {
        const int r = u / (C::BQ / 8), c = 2 * (u % (C::BQ / 8));
        float e[8];
#pragma unroll
        for (int g = 0; g < C::KW; ++g) {
          const float* src = reinterpret_cast<const float*>(all_smem + g * (C::NS * C::STAGE)) + r * C::BQ;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(src + 4 * ((c + h) ^ (r & 15)));
#pragma unroll
            for (int d = 0; d < 4; ++d) e[4 * h + d] = g == 0 ? v[d] : e[4 * h + d] + v[d];
          }
        }
        if (p.splits > 1) {
          f32x4* const part = reinterpret_cast<f32x4*>(p.ws + ((size_t)t.tile * p.splits + t.split) * (C::BP * C::BQ) + r * C::BQ + 4 * c);
          part[0] = f32x4{e[0], e[1], e[2], e[3]};
          part[1] = f32x4{e[4], e[5], e[6], e[7]};
          continue;
        }
        const int row = t.p0 + r, col = t.q0 + 4 * c;
        if (row < t.pend && col < p.Qtot)
          *reinterpret_cast<u32x4*>(out + (int64_t)row * p.ldc + col) =
              u32x4{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7])};
      }
      return;
    }

    if constexpr (kOwnRows) {
      // The next tile's first loads go ahead of this one's stores.
      const Tile done = t;
      bool more = false;
      if (turns) {
        const int x = blockIdx.x & 7, j = blockIdx.x >> 3, last = (int)(gridDim.x >> 3) - 1;   // XCD, place in it
        ++round;
        hw = round * (int)gridDim.x + 8 * (kDW && p.offsets != nullptr && (round & 1) ? last - j : j) + x;
        more = hw < p.ntiles;
        if (more) {
          t = pick(hw);
          more = t.valid;
        }
        if (more) {
          begin();
          first_loads();
        }
      }
      // bf16 results, 16 rows at a time, through the wave's own 2 KiB of LDS, so
      // that a store of eight lanes writes a row's 128 bytes: 8-byte slot s of row
      // r at s ^ 2 (r & 7).  No barrier, and the stages stay free for the loads.
      // (The whole tile through the stages, rows of 512 bytes: grad_W of 8192 x 4096
      // x 128 24.5 us, 20.1 this way.)
      uint8_t* const mine = all_smem + C::NS * C::STAGE + wave * 2048;
      int el = lane;
      asm volatile("" : "+v"(el));                               // (keeps the addresses below out of the main loop's registers)
      const int c8 = el & 7, r8 = el >> 3, r16 = el & 15;
      const int col = done.q0 + wq * C::WQ + 8 * c8, row = done.p0 + wp * C::WP + r8;
      const bool whole = done.p0 + C::BP <= done.pend && done.q0 + C::BQ <= p.Qtot;
      uint8_t* to = reinterpret_cast<uint8_t*>(out + (int64_t)(done.p0 + wp * C::WP) * p.ldc + done.q0 + wq * C::WQ);
      const uint32_t lane_to = 2u * ((uint32_t)r8 * p.ldc + 8 * c8);
      auto store = [&](auto all) {
#pragma unroll
        for (int i = 0; i < C::FP; ++i) {
#pragma unroll
          for (int j = 0; j < C::FQ; ++j)
            *reinterpret_cast<u32x2*>(mine + r16 * 128 + 8 * ((4 * j + (el >> 4)) ^ (2 * (r16 & 7)))) =
                u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(mine + (8 * h + r8) * 128 + 16 * (c8 ^ r8));
            if (decltype(all)::value || (row + 16 * i + 8 * h < done.pend && col < p.Qtot)) {
              u32x4* const dst = reinterpret_cast<u32x4*>(to + lane_to);
              // grad_W is often larger than the caches: streamed (64 experts of 2048 x
              // 7168, 32768 rows: 1008 us without, 911 us, both by whole rows).
              if constexpr (kDW) __builtin_nontemporal_store(v, dst);
              else *dst = v;
            }
            to += (int64_t)16 * p.ldc;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      // Rows that begin inside a 128-byte line: the waves that share 16 rows put
      // them together, so that a row's 512 bytes have two broken lines and not eight.
      // Memory takes a broken line of streamed stores several times over (57 experts
      // of 3760 x 1040, 8000 rows 187 us, 156 this way; 3840 x 1024 111).  Stores that are not
      // streamed meet in L2, which loses more where there is work beside (243 us for
      // 207, 190 this way, 32 experts of 2064 x 4112).
      const bool broken = kDW && ((p.ldc & 63) != 0 || (reinterpret_cast<uintptr_t>(p.C) & 127) != 0);
      auto store_joint = [&] {
        uint8_t* const joint = all_smem + C::NS * C::STAGE + wp * (C::NWQ * 2048);
        const int c32 = el & 31, r0 = 4 * wq + (el >> 5), jcol = done.q0 + 8 * c32;
#pragma unroll
        for (int i = 0; i < C::FP; ++i) {
#pragma unroll
          for (int j = 0; j < C::FQ; ++j)
            *reinterpret_cast<u32x2*>(joint + r16 * (2 * C::BQ) + 8 * ((wq * (C::WQ / 4) + 4 * j + (el >> 4)) ^ (2 * r16))) =
                u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
          barrier_lds();
          u32x4 v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[h] = *reinterpret_cast<const u32x4*>(joint + (r0 + 2 * h) * (2 * C::BQ) + 16 * (c32 ^ (r0 + 2 * h)));
          barrier_lds();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = done.p0 + wp * C::WP + 16 * i + r0 + 2 * h;
            if (at < done.pend && jcol < p.Qtot)
              __builtin_nontemporal_store(v[h], reinterpret_cast<u32x4*>(out + (int64_t)at * p.ldc + jcol));
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if (broken) store_joint();
      else if (whole) store(IC<1>{});
      else store(IC<0>{});
      if (!more) return;
      stores_behind = whole;
      continue;
    }

    // bf16 results through LDS, so that a store writes whole rows of the tile:
    // 8-byte slot s of row r at s ^ 2 (r & 15).
    constexpr int ROWB = C::BQ * 2, LPR = ROWB / 16, RPI = 64 / LPR;   // lanes per row, rows per store
    const int c16 = lane % LPR, col = t.q0 + 8 * c16;
#pragma unroll
    for (int i = 0; i < C::FP; ++i) {
      const int r = wp * C::WP + 16 * i + (lane & 15);
#pragma unroll
      for (int j = 0; j < C::FQ; ++j) {
        const int slot = wq * (C::WQ / 4) + 4 * j + (lane >> 4);
        *reinterpret_cast<u32x2*>(smem + r * ROWB + 8 * (slot ^ (2 * (r & 15)))) =
            u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
      }
    }
    __syncthreads();
#pragma unroll 4
    for (int it = 0; it < C::BP / (RPI * C::NW); ++it) {
      const int r = (it * C::NW + wave) * RPI + lane / LPR, row = t.p0 + r;
      const u32x4 v = *reinterpret_cast<const u32x4*>(smem + r * ROWB + 16 * (c16 ^ (r & 15)));
      if (row < t.pend && col < p.Qtot) *reinterpret_cast<u32x4*>(out + (int64_t)row * p.ldc + col) = v;
    }
    return;
  }
}

template <class C, int kOp>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void b128_kernel(Params p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLdsOf<C>];
  b128_tiles_of<C, kOp, 1>(p, smem);
}

// The last, partial round, in the smallest parts that fit one round: 64 x 64
// (the contraction over four groups of waves), then 128 x 128 if it has 32
// stages, else halves.  (4100 x 4096 x 2048, 16 tiles left, 53.7 us whole, 48.7 in
// halves, 41.2 in sixteenths; 6000 x 2800 x 2832, 8 left, 82.7, 72.9, 59.3.  Forward of
// 2048 x 4096 in 8 groups, 48 left, 150 us in halves, 145 in quarters; 56 stages, 64
// left, 493 -> 485; but 16 stages, 64 left, 155 -> 158.)
template <int kOp>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void b128_tail_kernel(Params p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLdsOf<B256N>];
  static_assert(kLdsOf<B128> <= kLdsOf<B256N> && kLdsOf<B64> <= kLdsOf<B256N>);
  int all = p.ntiles;
  if (kOp != kB128Dw && p.offsets != nullptr) {
    GroupScan sc{};
    for (int base = 0; base < p.groups; base += 64) sc = scan_groups<256>(p, p.Ptot, base, sc.last_end, sc.last_seen);
    all = sc.last_seen * ((p.Qtot + 255) / 256);
  }
  const Rounds r = rounds_of(p, all);
  if (!r.split) return;
  if (16 * r.rest <= kCUs) b128_tiles_of<B64, kOp, 16>(p, smem);
  else if (4 * r.rest <= kCUs && p.Ktot >= 32 * kRun) b128_tiles_of<B128, kOp, 4>(p, smem);
  else b128_tiles_of<B256N, kOp, 2>(p, smem);
}

template <class C, int kOp>
inline hipError_t run_b128(const Params& prm, hipStream_t s) {
  if (prm.ntiles <= 0) return hipSuccess;
  b128_kernel<C, kOp><<<dim3(takes_turns<C, kOp>(prm) ? kCUs : prm.ntiles * prm.splits), dim3(64 * C::NW * C::KW), 0, s>>>(prm);
  return hipGetLastError();
}

template <int kOp>
inline hipError_t run_b128_tail(const Params& prm, hipStream_t s) {
  b128_tail_kernel<kOp><<<dim3(kCUs), dim3(512), 0, s>>>(prm);
  return hipGetLastError();
}

}  // namespace gk
}  // namespace lp
