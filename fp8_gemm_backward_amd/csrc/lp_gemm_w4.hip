// Forward y = x @ W^T of few bf16 rows by a weight in 4 bits (MXFP4, NVFP4),
// dense and grouped.
//
// The weight is read once and everything else is small, so the call is a
// stream over W: it never goes through LDS.  Lane l of v_mfma_f32_16x16x32_bf16
// holds eight contraction elements of row l % 16; any order of the contraction
// will do as long as x has the same, so a lane takes 32 consecutive elements
// (16 bytes of codes) straight from global memory and decodes eight of them per
// MFMA, in registers, as lp_dequant does.  A wave owns 16 kNC columns of y (rows
// of W), 16 kRT rows of x and a part of the contraction; the sums of the kWK
// waves that share columns are added in wave order at the end, so the result
// does not depend on timing.
//
// What bounded it, step by step (96 rows over 31 of 64 experts of 2048 x 7168,
// NVFP4, 258 MB: 50 us at the rate of a large copy):
// * every lane loading its own scale bytes, 16 columns a wave        138 us
//   (2 bytes a lane from 16 rows: without these loads 74, without x's too 48)
// * the scales of six steps by one 16-byte load a lane, given out
//   through LDS                                                       70
// * x loaded once for the workgroup, through LDS                      68
// * the row tiles that have rows dealt first, counted with one group
//   a lane                                                            62
// * 16 rows by two column tiles a wave, x six steps at a time         55
// 512 rows over all 64 experts take 110 us (4.9 TB/s).  With more rows a tile the
// matrix cores' share grows: at 1000 x 4112 x 4128 every further 16 rows a workgroup
// add 0.10 us a step of 128, their MFMAs' own time, to 0.7 us for the weight's way
// into registers and the step's waits; deeper rings, four waves a SIMD and 64 columns
// a wave changed nothing there.
#include "lp_gemm_kernel.hpp"

namespace lp {
namespace gk {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kStep = 128;                      // contraction elements of a step: 32 a lane
constexpr int kSuper = 6;                       // steps whose scales are loaded together
constexpr int kPitch = 80;                      // LDS bytes of a row's scales: 64, and no two rows of a read on one bank

struct W4Args {
  Params p;
  int32_t row_tiles, col_tiles;                 // row_tiles: dense calls
};

// Row tiles (kRows rows of one group) of a grouped call.  Every wave looks at 64
// groups at a time, one a lane: their ends, starts and row tiles, and the row tiles
// up to each.
struct Groups64 {
  int end, start, tiles, upto;
};
template <int kRows>
__device__ __forceinline__ Groups64 groups64(const int32_t* offsets, int groups, int M, int base, int end0, int seen) {
  const int lane = threadIdx.x & 63;
  Groups64 s;
  int e = base + lane < groups ? offsets[base + lane] : 0;
  e = e > M ? M : e;
  e = e < end0 ? end0 : e;
  s.end = wave_scan(e, [](int a, int b) { return a > b ? a : b; });
  s.start = __shfl_up(s.end, 1);
  s.start = lane == 0 ? end0 : s.start;
  s.tiles = (s.end - s.start + kRows - 1) / kRows;
  s.upto = seen + wave_scan(s.tiles, [](int a, int b) { return a + b; });
  return s;
}

// How many there are.
template <int kRows>
__device__ __forceinline__ int live_tiles(const int32_t* offsets, int groups, int M) {
  int end0 = 0, seen = 0;
  for (int base = 0; base < groups; base += 64) {
    const Groups64 s = groups64<kRows>(offsets, groups, M, base, end0, seen);
    end0 = __builtin_amdgcn_readlane(s.end, 63);
    seen = __builtin_amdgcn_readlane(s.upto, 63);
  }
  return seen;
}

// The rt-th of them (rt below their number).
struct RowTile {
  int g, start, end;
};
template <int kRows>
__device__ __forceinline__ RowTile row_tile(const int32_t* offsets, int groups, int M, int rt) {
  int end0 = 0, seen = 0;
  for (int base = 0; base < groups; base += 64) {
    const Groups64 s = groups64<kRows>(offsets, groups, M, base, end0, seen);
    const uint64_t own = __ballot(s.upto > rt);
    if (own != 0) {
      const int l = __builtin_ctzll(own);
      const int before = __builtin_amdgcn_readlane(s.upto, l) - __builtin_amdgcn_readlane(s.tiles, l);
      return RowTile{base + l, __builtin_amdgcn_readlane(s.start, l) + (rt - before) * kRows, __builtin_amdgcn_readlane(s.end, l)};
    }
    end0 = __builtin_amdgcn_readlane(s.end, 63);
    seen = __builtin_amdgcn_readlane(s.upto, 63);
  }
  return RowTile{0, 0, 0};
}

// Where the 16-byte chunk 4 h + q (of the 16 of a step) of row r lies in LDS:
// the 16 lanes that a 16-byte read serves together (rows 0-3 and 12-15 of one h,
// 4-11 of its neighbour) get distinct slots of 256 bytes.
__device__ __forceinline__ int x_slot(int r, int h, int q) {
  return ((((h & 1) * 3) ^ (h >> 1)) * 4 + q) ^ r;
}

// kWK: waves that share 16 kNC columns, each with its part of the contraction;
// kNC, kRT: column and row tiles of a wave; kDepth: steps in flight; kXS: 0 for x
// straight into registers, else by way of LDS, loaded once for the workgroup, kXS
// steps at a time into two buffers in turn.
template <int F, int kWK, int kNC, int kRT, int kDepth, int kXS, int kEu = 2>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(kEu))) void w4_kernel(W4Args a) {
  constexpr int kRows = 16 * kRT, WN = kWaves / kWK;
  constexpr int kByte = F == NVFP4 ? 16 : 32;                    // elements of a scale byte
  using Scales = std::conditional_t<F == NVFP4, u32x4, u32x2>;   // a lane's part of a row's kSuper steps
  constexpr bool kShare = kXS > 0;
  constexpr int kRowBytes = (kShare ? kXS : 1) * kStep * 2, kXBytes = kWK * kRows * kRowBytes;   // LDS: a row's x, a buffer
  constexpr int kPieces = kShare ? kXBytes / 16 / kThreads : 1;
  static_assert(!kShare || (kXBytes / 16 % kThreads == 0 && kSuper % kXS == 0), "x divides among the threads");
  static_assert(kSuper % kDepth == 0 && kSuper * (kStep / kByte) + 3 <= 4 * (int)sizeof(Scales), "a lane's part of the scales");
  const Params& p = a.p;
  __shared__ __attribute__((aligned(256))) union {               // in turn, barriers between
    uint8_t x[kShare ? 2 * kXBytes : 16];
    f32x4 sum[kWK == 1 ? 1 : kWaves - WN][kNC * kRT][64];
  } sh;
  __shared__ __attribute__((aligned(16))) uint8_t s_scales[kWaves][kNC][16 * kPitch];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave % kWK, wn = wave / kWK;
  // Tiles in the order of columns, then row tiles.  Workgroups are dealt to the 8
  // XCDs in turn; XCD x takes the x-th eighth of the tiles, so that the row tiles
  // of a column share its L2, which then serves the weight's second reads.
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  int live = a.row_tiles;
  if (p.offsets != nullptr) live = live_tiles<kRows>(p.offsets, p.groups, p.Ptot);
  const int tiles = live * a.col_tiles, eighth = (tiles + 7) / 8, tile = xcd * eighth + at;
  if (at >= eighth || tile >= tiles) return;
  const int col = tile / live, rt = tile - col * live, n0 = (col * WN + wn) * 16 * kNC;
  int g = 0, p0 = rt * kRows, pend = p.Ptot;
  if (p.offsets != nullptr) {
    const RowTile t = row_tile<kRows>(p.offsets, p.groups, p.Ptot, rt);
    g = t.g;
    p0 = t.start;
    pend = t.end;
  }

  const int K = p.Ktot, N = p.Qtot;
  const int r = lane & 15, h = lane >> 4;
  // The wave's steps of the contraction; none for columns past the end.
  const int all = (K + kStep - 1) / kStep, per = (all + kWK - 1) / kWK;
  const int first = wk * per, last = n0 >= N ? 0 : first + per < all ? first + per : all;
  // Rows of W past the last read as zero: the range ends with them.
  const int64_t wrows = N - n0 < 16 * kNC ? N - n0 : 16 * kNC;
  const Rsrc wr = make_rsrc(p.Q.codes + (int64_t)g * p.Q.code_batch + (int64_t)n0 * p.Q.code_ld, wrows * p.Q.code_ld);
  const Rsrc sr = make_rsrc(p.Q.scales + (int64_t)g * p.Q.scale_batch + (int64_t)n0 * p.Q.scale_ld, wrows * p.Q.scale_ld);
  const Rsrc xr = make_rsrc(p.P.codes + (int64_t)p0 * p.P.code_ld, (int64_t)(pend - p0) * p.P.code_ld);
  float ts = 0.0f;
  if constexpr (F == NVFP4) ts = *p.Q.tensor_scale;

  // Step i's codes, and its x unless that comes by way of LDS; what lies past
  // the end reads as zero.
  struct Ring {
    u32x4 w[kNC], x[kShare ? 1 : kRT][4];
  } ring[kDepth];
  auto load = [&](Ring& b, int i) __attribute__((always_inline)) {
    const int k0 = i * kStep + 32 * h;                           // K % 32 == 0: all 32 are in, or none
    const bool in = i < last && k0 < K;
#pragma unroll
    for (int c = 0; c < kNC; ++c) b.w[c] = bload16(wr, in ? (r + 16 * c) * p.Q.code_ld + k0 / 2 : kOOB);
    if constexpr (!kShare) {
#pragma unroll
      for (int t = 0; t < kRT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) b.x[t][q] = bload16(xr, in ? (r + 16 * t) * p.P.code_ld + 2 * k0 + 16 * q : kOOB);
    }
  };
  // The scales of steps i .. i + kSuper - 1, a quarter of each row's a lane, from
  // the last multiple of four bytes on.
  Scales next[kNC];
  auto load_scales = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      const int at = (r + 16 * c) * p.Q.scale_ld + i * (kStep / kByte);
      const int off = i < last ? (at & ~3) + (int)sizeof(Scales) * h : kOOB;
      if constexpr (F == NVFP4) next[c] = bload16(sr, off);
      else next[c] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(sr, off, 0, 0));
    }
  };
  // x of the workgroup's steps v kXS .. of every part of the contraction.
  u32x4 xnext[kPieces];
  auto load_x = [&](int v) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = tid + i * kThreads, chunk = piece % (kRowBytes / 16), row = piece / (kRowBytes / 16);
      const int k0 = ((row / kRows) * per + v * kXS) * kStep + 8 * chunk;
      xnext[i] = bload16(xr, k0 < K && v * kXS < per ? row % kRows * p.P.code_ld + 2 * k0 : kOOB);
    }
  };
  auto store_x = [&](int v) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = tid + i * kThreads, chunk = piece % (kRowBytes / 16), row = piece / (kRowBytes / 16);
      *reinterpret_cast<u32x4*>(sh.x + (v & 1) * kXBytes + row * kRowBytes + chunk / 16 * 256 + 16 * x_slot(row & 15, chunk / 4 % 4, chunk % 4)) =
          xnext[i];
    }
  };

  f32x4 acc[kNC][kRT] = {};
  // A row's scales begin at (its address) % 4 in LDS; s: the step's place among its kSuper.
  const uint8_t* const scale_at = s_scales[wave][0] + r * kPitch + ((r * p.Q.scale_ld) & 3) + h * (32 / kByte);
  const uint8_t* const x_at = sh.x + (wk * kRows + r) * kRowBytes;
  auto multiply = [&](const Ring& b, int i, int s, int v) __attribute__((always_inline)) {
    Raw<F, -1> w[kNC];
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
      w[c].c = b.w[c];
      w[c].s = *reinterpret_cast<const typename Raw<F, -1>::S*>(scale_at + c * 16 * kPitch + s * (kStep / kByte));
      if (i * kStep + 32 * h >= K) w[c].s = 0;                   // the next row's
    }
    static_for<4>([&](auto piece) __attribute__((always_inline)) {
      constexpr int J = decltype(piece)::value;
      u32x4 x[kRT];
#pragma unroll
      for (int t = 0; t < kRT; ++t) {
        if constexpr (kShare) x[t] = *reinterpret_cast<const u32x4*>(x_at + (v & 1) * kXBytes + t * 16 * kRowBytes + s % (kShare ? kXS : 1) * 256 + 16 * x_slot(r, h, J));
        else x[t] = b.x[t][J];
      }
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        float sc;
        u32x4 v;
        v[0] = decode_quarter<F, -1, J, 0>(w[c], ts, sc);
        v[1] = decode_quarter<F, -1, J, 1>(w[c], ts, sc);
        v[2] = decode_quarter<F, -1, J, 2>(w[c], ts, sc);
        v[3] = decode_quarter<F, -1, J, 3>(w[c], ts, sc);
#pragma unroll
        for (int t = 0; t < kRT; ++t)
          acc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v), __builtin_bit_cast(bf16x8, x[t]), acc[c][t], 0, 0, 0);
      }
    });
  };

  load_scales(first);
  if constexpr (kShare) load_x(0);
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    load(ring[i], first + i);
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (kShare) {
    store_x(0);
    load_x(1);
  }
  // (Loads keep their order, so that waiting for a step leaves the later ones in flight.)
  for (int u = 0; u * kSuper < per; ++u) {
    __builtin_amdgcn_wave_barrier();                             // the last steps' scales (the wave's own) are read
#pragma unroll
    for (int c = 0; c < kNC; ++c)
      *reinterpret_cast<Scales*>(s_scales[wave][c] + r * kPitch + (int)sizeof(Scales) * h) = next[c];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    load_scales(first + (u + 1) * kSuper);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < kSuper; ++s) {
      const int i = first + u * kSuper + s, v = kShare ? u * (kSuper / (kShare ? kXS : 1)) + s / (kShare ? kXS : 1) : 0;
      if (u * kSuper + s >= per) break;
      if (kShare && s % (kShare ? kXS : 1) == 0) {
        __syncthreads();                                         // buffer v is written, the other one read
        store_x(v + 1);
        load_x(v + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
      multiply(ring[s % kDepth], i, s, v);
      __builtin_amdgcn_sched_barrier(0);
      load(ring[s % kDepth], i + kDepth);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  if constexpr (kWK > 1) {
    __syncthreads();                                             // x is read
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < kNC * kRT; ++i) sh.sum[wn * (kWK - 1) + wk - 1][i][lane] = acc[i / kRT][i % kRT];
    }
    __syncthreads();
    if (wk != 0) return;
#pragma unroll
    for (int w = 0; w < kWK - 1; ++w) {
#pragma unroll
      for (int i = 0; i < kNC * kRT; ++i) {
        const f32x4 o = sh.sum[wn * (kWK - 1) + w][i][lane];
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[i / kRT][i % kRT][d] += o[d];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kNC; ++c)
#pragma unroll
    for (int t = 0; t < kRT; ++t)
      if (p0 + r + 16 * t < pend && n0 + 16 * c < N)
        *reinterpret_cast<u32x2*>(p.C + (int64_t)(p0 + r + 16 * t) * p.ldc + n0 + 16 * c + 4 * h) =
            u32x2{pack_bf16x2(acc[c][t][0], acc[c][t][1]), pack_bf16x2(acc[c][t][2], acc[c][t][3])};
}

// The instantiated shapes of a workgroup, and their times in units of 10 ns:
// fixed, and for every round of 256 workgroups (the first one, each further one) a
// step of a wave's part of the contraction and, each further one, a fixed time too.
// Fitted to 2500 measured problems (1 to 4096 rows, dense and up to 64 groups,
// weights from HBM, both formats) with 7 to 18% of scatter: the shape they choose
// is within 3% of the fastest on average, within 1.4 times in 99 of 100 (the grouped
// ones' row tiles known only as a bound).  64 rows by one
// column tile a wave ({2, 1, 4}, {1, 1, 4}) serve some hundred rows of middling
// weights: 212 x 3488 x 4992 23 us (34.5 without them), 171 x 3616 x 1984 12.5 (18.9);
// 80 rows ({1, 2, 5}) 1000 x 4112 x 4128, whose tiles of 112 left a third of the CUs
// without any: 41 us (48).
struct Shape {
  int8_t wk, nc, rt;
  int16_t fixed, step, more, round;
};
constexpr Shape kShapes[] = {
    {8, 1, 1, 320, 58, 76, 59},    {4, 1, 1, 412, 43, 62, 256},   {2, 1, 1, 425, 37, 48, 274},   {1, 2, 1, 347, 58, 52, 141},
    {4, 1, 2, 428, 69, 82, 260},   {2, 1, 2, 433, 51, 59, 280},   {2, 1, 4, 444, 86, 91, 316},   {4, 2, 3, 459, 120, 132, 307},
    {2, 2, 4, 522, 110, 123, 418}, {1, 2, 4, 404, 98, 96, 213},   {1, 1, 6, 382, 91, 68, 161},   {1, 2, 5, 498, 112, 136, 364},
    {1, 2, 8, 454, 162, 179, 494}, {1, 1, 4, 373, 67, 51, 160},   {1, 2, 3, 424, 82, 91, 189},  {2, 2, 5, 519, 128, 150, 379},
};
constexpr int kShapeCount = sizeof(kShapes) / sizeof(kShapes[0]);
// The same of the 256 x 256 tiles that decode into LDS; their matrix cores, busier,
// run at a lower clock when every CU has a tile.
constexpr int kTileFixed = 800, kTileStep = 280, kTileStepFull = 410;

// Row tiles of a call; a bound where rows are grouped: groups with rows have a tile
// each for their first row, and one for every further row tile's worth of rows (1 row
// over 48 groups launched 48 times the workgroups it needs by M / rows + groups, 19 us
// for 6).
int64_t row_tiles(const Params& p, int rows) {
  if (p.offsets == nullptr) return (p.Ptot + rows - 1) / rows;
  const int64_t used = p.Ptot < p.groups ? p.Ptot : p.groups;
  return used + (p.Ptot - used) / rows;
}

int64_t col_tiles(const Params& p, const Shape& s) {
  const int64_t cols = 16 * s.nc * kWaves / s.wk;
  return (p.Qtot + cols - 1) / cols;
}

// The shape of least estimated time; -1: the 256 x 256 tiles.
int choose(const Params& p) {
  const int64_t steps = (p.Ktot + kStep - 1) / kStep;
  int best = -1;
  int64_t least = INT64_MAX;
  for (int i = 0; i < kShapeCount; ++i) {
    const Shape& s = kShapes[i];
    // (a launch has fewer than 2^32 threads)
    if (row_tiles(p, 16 * s.rt) * col_tiles(p, s) + 8 > (int64_t)1 << 23) continue;
    const int64_t rounds = (row_tiles(p, 16 * s.rt) * col_tiles(p, s) + kCUs - 1) / kCUs;
    const int64_t t = s.fixed + (rounds - 1) * s.round + (steps + s.wk - 1) / s.wk * (s.step + (rounds - 1) * s.more);
    if (t < least) {
      least = t;
      best = i;
    }
  }
  const int64_t tiles = row_tiles(p, 256) * ((p.Qtot + 255) / 256);
  const int64_t t = kTileFixed + steps * (tiles <= kCUs / 2 ? kTileStep : kTileStepFull * ((tiles + kCUs - 1) / kCUs));
  return best >= 0 && least <= t ? best : -1;
}

template <int F, int kIndex, int kDepth, int kXS, int kEu = 2>
hipError_t launch(W4Args a, hipStream_t s) {
  constexpr Shape kS = kShapes[kIndex];
  const int64_t rt = row_tiles(a.p, 16 * kS.rt), nt = col_tiles(a.p, kS);
  a.row_tiles = (int32_t)rt;
  a.col_tiles = (int32_t)nt;
  w4_kernel<F, kS.wk, kS.nc, kS.rt, kDepth, kXS, kEu><<<dim3((uint32_t)((rt * nt + 7) / 8 * 8)), dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

template <int F>
hipError_t launch_shape(const W4Args& a, int shape, hipStream_t s) {
  switch (shape) {
    case 0: return launch<F, 0, 2, 0>(a, s);
    case 1: return launch<F, 1, 2, 3>(a, s);
    case 2: return launch<F, 2, 3, 6>(a, s);
    case 3: return launch<F, 3, 2, 6>(a, s);
    case 4: return launch<F, 4, 2, 2>(a, s);
    case 5: return launch<F, 5, 3, 3>(a, s);
    case 6: return launch<F, 6, 2, 2>(a, s);
    case 7: return launch<F, 7, 2, 1>(a, s);
    case 8: return launch<F, 8, 2, 2>(a, s);
    case 9: return launch<F, 9, 2, 1, 4>(a, s);
    case 10: return launch<F, 10, 3, 1, 4>(a, s);
    case 11: return launch<F, 11, 2, 2>(a, s);
    case 12: return launch<F, 12, 2, 1>(a, s);
    case 13: return launch<F, 13, 2, 2>(a, s);
    case 14: return launch<F, 14, 2, 2>(a, s);
    default: return launch<F, 15, 2, 1>(a, s);
  }
}

}  // namespace

hipError_t w4_fwd(const Params& prm, int fmt_w, bool* done, hipStream_t s) {
  const int shape = choose(prm);
  *done = shape >= 0;
  if (shape < 0) return hipSuccess;
  const W4Args a{prm, 0, 0};
  return fmt_w == LP_MXFP4 ? launch_shape<MXFP4>(a, shape, s) : launch_shape<NVFP4>(a, shape, s);
}

}  // namespace gk
}  // namespace lp
