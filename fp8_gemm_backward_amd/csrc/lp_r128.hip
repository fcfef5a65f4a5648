// Quantization of bf16 to E4M3 with an fp32 scale per run of 128 (along the
// columns, along the rows, or both from one read) or per 128 x 128 block
// (HBM-bound, bit-exact; the arithmetic is in lp_r128.hpp).
#include <type_traits>

#include "lp_internal.hpp"
#include "lp_r128.hpp"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kRunLen = 128;

// f(0), f(1), f(2), f(3), each with a constant.
template <class F>
__device__ __forceinline__ void static_for4(F&& f) {
  f(std::integral_constant<int, 0>{});
  f(std::integral_constant<int, 1>{});
  f(std::integral_constant<int, 2>{});
  f(std::integral_constant<int, 3>{});
}

// Runs along the columns.  Sixteen lanes hold a run, eight values each, and
// take its largest magnitude with lane-row rotations.  A workgroup takes 16
// rows x 4 runs: a row's four runs are 1 KiB in a line, and the 16 rows'
// scales of one run index are 64 bytes in a line ([run][row]).  8192 x 4096 in
// 17.1 us (5.9 TB/s), 24 x 2048 in 2.7 us (a launch).
constexpr int kRunRows = 16, kRunCols = 4;

__global__ __launch_bounds__(kThreads) void r128_cols(const uint16_t* __restrict__ src, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales, int64_t total_rows, FastDiv rows,
                                                      int32_t cols, FastDiv col_tiles) {
  const uint32_t rt = fdiv(blockIdx.x, col_tiles);
  const uint32_t ct = blockIdx.x - rt * col_tiles.d;
  const int64_t row = (int64_t)rt * kRunRows + threadIdx.x / 16;          // over batch * rows
  if (row >= total_rows) return;
  const int lane = threadIdx.x & 15;
  const uint32_t b = fdiv((uint32_t)row, rows), r = (uint32_t)row - b * rows.d;
  const int nrun = (cols - 1) / kRunLen + 1;               // (cols may be the largest int less 15)
  u32x4 v[kRunCols];
#pragma unroll
  for (int j = 0; j < kRunCols; ++j) {
    const int c = (ct * kRunCols + j) * kRunLen + 8 * lane;
    v[j] = c < cols ? *reinterpret_cast<const u32x4*>(src + row * cols + c) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int j = 0; j < kRunCols; ++j) {
    const int run = ct * kRunCols + j, c = run * kRunLen + 8 * lane;
    const RunScale q = run_scale(row16_max(amax8(v[j])));
    if (run < nrun && lane == 0) scales[((int64_t)b * nrun + run) * rows.d + r] = q.s;
    if (c < cols) *reinterpret_cast<u32x2*>(codes + row * cols + c) = run_codes8(v[j], q);
  }
}

// The rows of token run `run` of a grouped tensor: group g's runs are
// start_g / 128 + g onwards, 128 rows each, the last one cut at the group's
// end.  Run indices between two groups' ranges have no rows.  Every wave
// looks at 64 groups at a time, one a lane (walking them one by one cost
// 32768 x 2048 in 64 groups 79 us along both axes, this 54 then and 45 now).
// kAhead: so many loads at once, for kernels where these loads show.
template <int kAhead = 1>
__device__ __forceinline__ void run_rows(const int32_t* __restrict__ offsets, int groups, int M, int run, int& r0,
                                         int& r1) {
  const int lane = threadIdx.x & 63;
  int end0 = 0;
  r0 = r1 = 0;
  for (int base0 = 0; base0 < groups; base0 += 64 * kAhead) {
    int ends[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int g = base0 + 64 * j + lane;
      if (base0 + 64 * j < groups) ends[j] = offsets[g < groups ? g : groups - 1];
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int base = base0 + 64 * j;
      if (base >= groups) return;
      int e = ends[j] > M ? M : ends[j];
      e = e < end0 ? end0 : e;
      e = wave_scan(e, [](int a, int b) { return a > b ? a : b; });
      int start = __shfl_up(e, 1);
      start = lane == 0 ? end0 : start;
      const int k = run - (start / kRunLen + base + lane);
      const uint64_t own = __ballot(base + lane < groups && k >= 0 && k < (e - start + kRunLen - 1) / kRunLen);
      if (own != 0) {
        const int i = __builtin_ctzll(own), end = __builtin_amdgcn_readlane(e, i);
        r0 = __builtin_amdgcn_readlane(start, i) + __builtin_amdgcn_readlane(k, i) * kRunLen;
        r1 = r0 + kRunLen < end ? r0 + kRunLen : end;
        return;
      }
      end0 = __builtin_amdgcn_readlane(e, 63);
    }
  }
}

// One 128 x 128 tile per workgroup, for runs along the rows (kRows), along
// both axes (kRows and kCols) or one scale for the tile (neither).  Thread
// 16 i + c holds rows i + 32 k (k = 0..3) of columns 8 c .. 8 c + 7, so that
// each load of 16 lanes is 256 bytes in a line; a row's largest magnitude is
// taken over its 16 lanes, a column's over the thread's four rows, the four
// lane rows of the wave and, through LDS, the eight waves.  One thread per
// column then makes its scale while the others go on with the runs along the
// columns.  Both axes of 1000 x 2064 in 4.6 us, of 8192 x 4096 in 23.0 (5.8 TB/s).
// Before the two-instruction quotients, 5.4 and 26.5, 256 threads took 1.2 and 0.5
// more, 1024 threads 0.1 less and 2.1 more, and every thread making the scales of
// its eight columns 0.4 and 0.8 more.
struct TileArgs {
  const uint16_t* src;
  uint8_t *codes_c, *codes_r;
  float *scales_c, *scales_r;
  const int32_t* offsets;
  int32_t groups, rows, cols;
  FastDiv col_tiles, row_tiles;            // row_tiles: runs (blocks) along the rows of one batch entry
};

constexpr int kTileThreads = 512, kTileWaves = kTileThreads / 64, kStep = kTileThreads / 16, kTileRows = kRunLen / kStep;

// kStream: past the caches, where the next kernel would not find them anyway.
template <bool kStream>
__device__ __forceinline__ void store_codes(uint8_t* to, u32x2 o) {
  if constexpr (kStream) __builtin_nontemporal_store(o, reinterpret_cast<u32x2*>(to));
  else *reinterpret_cast<u32x2*>(to) = o;
}

// 128 rows and columns, offsets inside which take 32 bits.
__device__ __forceinline__ bool is_full(const TileArgs& a, int rows, int ct) {
  return rows == kRunLen && ct < a.cols / kRunLen && a.cols < 1 << 25;
}

// What a tile's threads share.
struct TileLds {
  alignas(16) uint16_t max[kTileWaves][kRunLen];
  alignas(16) float r[kRunLen], l[kRunLen];                // of the runs along the rows (RunRecip)
  uint32_t bad[kRunLen / 64];                              // whether one of 64 columns has a bad run
  int rows[2];                                             // run_rows_once
};

// run_rows by the first wave, for all of a workgroup.
__device__ __forceinline__ void run_rows_once(const TileArgs& a, TileLds& sh, int run, int& r0, int& r1) {
  if (threadIdx.x < 64) {
    run_rows(a.offsets, a.groups, a.rows, run, r0, r1);
    if (threadIdx.x == 0) {
      sh.rows[0] = r0;
      sh.rows[1] = r1;
    }
  }
  __syncthreads();
  r0 = __builtin_amdgcn_readfirstlane(sh.rows[0]);
  r1 = __builtin_amdgcn_readfirstlane(sh.rows[1]);
}

__device__ __forceinline__ float bf16_at(u32x4 v, int e) { return e % 2 ? bf16_hi(v[e / 2]) : bf16_lo(v[e / 2]); }

// The values of lane k of each 16, in all of them.
template <int k>
__device__ __forceinline__ float row16_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x150 + k, 0xF, 0xF, true));   // row_newbcast:k
}
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true);      // quad_perm:[1,0,3,2]
}
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true);      // quad_perm:[2,3,0,1]
}

// Four maxima over 16 lanes: lane i gets the one of m[i % 4].
__device__ __forceinline__ uint32_t row16_max4(const uint32_t (&m)[4], int i) {
  const bool b0 = i & 1, b1 = i & 2;
  const uint32_t p = umax(b0 ? m[1] : m[0], quad_xor1(b0 ? m[0] : m[1]));
  const uint32_t q = umax(b0 ? m[3] : m[2], quad_xor1(b0 ? m[2] : m[3]));
  uint32_t t = umax(b1 ? q : p, quad_xor2(b1 ? p : q));
  t = umax(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0x128, 0xF, 0xF, true));   // row_ror:8
  return umax(t, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)t, 0x124, 0xF, 0xF, true));   // row_ror:4
}

// The tile of rows r0 .. r1 (at most 128; kFull, see is_full: 128 rows and columns) and column
// tile ct of batch entry b, whose run (block) along the rows is number rb; v: the
// thread's values.  The two ways of quantizing take 340 vector instructions for a
// thread's 32 values, which bounds tiles that come out of a cache; hence the
// four rows' scales made side by side in four lanes, a column's
// by one thread, and bad runs patched in a branch of their own.
template <bool kCols, bool kRows, bool kFull, bool kStream = false, int kTileThreads = lp::kTileThreads>
__device__ __forceinline__ void quant_tile(const TileArgs& a, TileLds& sh, u32x4 (&v)[kTileRows], int64_t b, int rb, int ct,
                                           int r0, int r1) {
  static_assert(kTileRows == 4, "a lane of four for each row");
  constexpr int kTileWaves = kTileThreads / 64, kStep = kTileThreads / 16;
  const int tid = threadIdx.x % kTileThreads, ci = tid & 15, ri = tid >> 4, wave = tid >> 6;
  const bool col_ok = kFull || ct * kRunLen + 8 * ci < a.cols;
  const int n = kFull ? kRunLen : r1 - r0;
  const int64_t corner = (b * a.rows + r0) * a.cols + ct * kRunLen;       // (uniform)
  using Off = std::conditional_t<kFull, uint32_t, uint64_t>;
  const Off off = (Off)ri * (Off)a.cols + 8 * ci, step = (Off)kStep * (Off)a.cols;
  auto stored = [&](int k) { return kFull || (col_ok && ri + kStep * k < n); };
  auto empty = [&](int k) { return !kFull && kStep * k >= n; };           // no row of the tile (uniform): groups of few rows
  // Magnitudes' maxima per column (bf16 pairs).
  u32x4 cm = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int k = 0; k < kTileRows; ++k)
#pragma unroll
    for (int d = 0; d < 4; ++d) cm[d] = pk_umax16(cm[d], v[k][d] & 0x7FFF7FFFu);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    cm[d] = pk_umax16(cm[d], (uint32_t)__shfl_xor((int)cm[d], 16));
    cm[d] = pk_umax16(cm[d], (uint32_t)__shfl_xor((int)cm[d], 32));
  }
  if ((tid & 63) < 16) *reinterpret_cast<u32x4*>(&sh.max[wave][8 * ci]) = cm;
  __syncthreads();
  if constexpr (kRows) {
    if (tid < kRunLen) {                                   // one column's scale per thread
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kTileWaves; ++w) m = umax(m, sh.max[w][tid]);
      const RunScale q = run_scale(m << 16);
      const RunRecip p = run_recip(q.s, q.r);
      sh.r[tid] = p.r;
      sh.l[tid] = q.bad ? __builtin_nanf("") : p.l;
      const bool any = __ballot(q.bad) != 0;
      if ((tid & 63) == 0) sh.bad[wave] = any;
      if (kFull || ct * kRunLen + tid < a.cols)
        a.scales_r[((int64_t)b * a.row_tiles.d + rb) * a.cols + ct * kRunLen + tid] = q.s;
    }
  }
  if constexpr (kCols || kRows) {
    if constexpr (kCols) {
      uint32_t m[kTileRows];
#pragma unroll
      for (int k = 0; k < kTileRows; ++k) m[k] = amax8(v[k]);
      const RunScale q = run_scale(row16_max4(m, ci));     // row ri + kStep (ci % 4)
      const RunRecip p = run_recip(q.s, q.r);
      if (ci < kTileRows && (kFull || (ri + kStep * ci < n && ct * kRunLen < a.cols)))
        a.scales_c[((int64_t)b * a.col_tiles.d + ct) * a.rows + r0 + ri + kStep * ci] = q.s;
      const bool any = __ballot(q.bad) != 0;
      uint8_t* const to = a.codes_c + corner;
      static_for4([&](auto kk) __attribute__((always_inline)) {
        constexpr int k = decltype(kk)::value;
        if (empty(k)) return;
        const RunRecip pk{row16_lane<k>(p.r), row16_lane<k>(p.l)};
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = run_div_bf16(bf16_at(v[k], e), pk);
        u32x2 o{codes4_unclamped(t[0], t[1], t[2], t[3]), codes4_unclamped(t[4], t[5], t[6], t[7])};
        if (__builtin_expect(any, false)) {
          if (row16_lane<k>(q.bad ? 1.0f : 0.0f) != 0.0f)
            o = u32x2{nan_e4m3x2(v[k][0]) | (nan_e4m3x2(v[k][1]) << 16), nan_e4m3x2(v[k][2]) | (nan_e4m3x2(v[k][3]) << 16)};
        }
        if (stored(k)) store_codes<kStream>(to + (off + k * step), o);
        __builtin_amdgcn_sched_barrier(0);                 // (a row at a time: fewer registers)
      });
    }
    if constexpr (kRows) {
      __syncthreads();
      // (The values are unpacked anew: kept unpacked they took 32 registers more, and
      // with them a workgroup less per CU.)
#pragma unroll
      for (int k = 0; k < kTileRows; ++k) asm volatile("" : "+v"(v[k]));
      RunRecip q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = RunRecip{sh.r[8 * ci + e], sh.l[8 * ci + e]};
      const bool any = (sh.bad[0] | sh.bad[1]) != 0;
      uint8_t* const to = a.codes_r + corner;
#pragma unroll
      for (int k = 0; k < kTileRows; ++k) {
        if (empty(k)) break;
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = run_div_bf16(bf16_at(v[k], e), q[e]);
        u32x2 o{codes4_unclamped(t[0], t[1], t[2], t[3]), codes4_unclamped(t[4], t[5], t[6], t[7])};
        if (__builtin_expect(any, false)) {
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const uint32_t nan = nan_e4m3x2(v[k][2 * d]) | (nan_e4m3x2(v[k][2 * d + 1]) << 16);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (__builtin_isnan(q[4 * d + e].l)) o[d] = (o[d] & ~(0xFFu << (8 * e))) | (nan & (0xFFu << (8 * e)));
          }
        }
        if (stored(k)) store_codes<kStream>(to + (off + k * step), o);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  } else {
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) {
      const u32x4 o = *reinterpret_cast<const u32x4*>(&sh.max[w][8 * ci]);
#pragma unroll
      for (int d = 0; d < 4; ++d) cm[d] = pk_umax16(cm[d], o[d]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) m = umax(m, umax(cm[d] & 0xFFFFu, cm[d] >> 16));
    const RunScale q = run_scale(row16_max(m) << 16);
    if (tid == 0) a.scales_c[((int64_t)b * a.row_tiles.d + rb) * a.col_tiles.d + ct] = q.s;
#pragma unroll
    for (int k = 0; k < kTileRows; ++k)
      if (stored(k)) *reinterpret_cast<u32x2*>(a.codes_c + corner + (off + k * step)) = run_codes8_bf16(v[k], q);
  }
}

template <bool kCols, bool kRows>
__global__ __launch_bounds__(kTileThreads) void r128_tile(TileArgs a) {
  __shared__ TileLds sh;
  const uint32_t rtile = fdiv(blockIdx.x, a.col_tiles);
  const int ct = blockIdx.x - rtile * a.col_tiles.d;
  const uint32_t b = fdiv(rtile, a.row_tiles);
  const int rb = rtile - b * a.row_tiles.d;
  int r0 = rb * kRunLen, r1 = r0 + kRunLen < a.rows ? r0 + kRunLen : a.rows;
  if (a.offsets != nullptr) {
    run_rows(a.offsets, a.groups, a.rows, rb, r0, r1);
    if (r1 == r0) return;
  }
  const int c = ct * kRunLen + 8 * (threadIdx.x & 15), ri = threadIdx.x >> 4;
  const int64_t base = ((int64_t)b * a.rows + r0) * a.cols + c;
  u32x4 v[kTileRows];
#pragma unroll
  for (int k = 0; k < kTileRows; ++k) {
    const int r = ri + kStep * k;
    v[k] = c < a.cols && r0 + r < r1 ? *reinterpret_cast<const u32x4*>(a.src + base + (int64_t)r * a.cols)
                                     : u32x4{0u, 0u, 0u, 0u};
  }
  if (is_full(a, r1 - r0, ct))
    quant_tile<kCols, kRows, true>(a, sh, v, b, rb, ct, r0, r1);
  else
    quant_tile<kCols, kRows, false>(a, sh, v, b, rb, ct, r0, r1);
}

// Results larger than a quarter of the 256 MB cache are stored past the caches: 4096
// tokens to 8 experts each, 7168 wide, read x (59 MB, each row k times) faster from a
// cache that 470 MB of codes do not wash through, 120 us in all (150); to 8 of 1024 experts,
// whose short runs go by fours (below), 267 (292), and 2048 of them to 4 of 256 57 (66).
constexpr int64_t kCacheBytes = (int64_t)64 << 20;

// Rows that come from elsewhere: row r is row order[r] / k of src, times
// weights[order[r]] when kWeighted, rounded to bf16; zeros when order[r] is no pair.
struct RowMap {
  const int32_t* order;
  const float* weights;
  FastDiv k;
  uint32_t pairs;
};

// The values of a thread, kTileThreads of which take a tile.
template <bool kWeighted, int kTileThreads>
__device__ __forceinline__ void mapped_values(const TileArgs& a, const RowMap& map, int ct, int r0, int r1, u32x4 (&v)[kTileRows]) {
  constexpr int kStep = kTileThreads / 16;
  const int tid = threadIdx.x % kTileThreads, c = ct * kRunLen + 8 * (tid & 15), r = r0 + (tid >> 4);
  uint32_t pair[kTileRows];
#pragma unroll
  for (int k = 0; k < kTileRows; ++k) {
    pair[k] = r + kStep * k < r1 ? (uint32_t)map.order[r + kStep * k] : ~0u;
    if (pair[k] >= map.pairs || c >= a.cols) pair[k] = ~0u;
  }
  // (each row into a variable of its own: into v[k] itself, one load waited for the last)
  float w[kTileRows];
#pragma unroll
  for (int k = 0; k < kTileRows; ++k) {
    u32x4 x = {0u, 0u, 0u, 0u};
    float y = 0.0f;
    if (pair[k] != ~0u) {
      x = *reinterpret_cast<const u32x4*>(a.src + (int64_t)fdiv(pair[k], map.k) * a.cols + c);
      if constexpr (kWeighted) y = map.weights[pair[k]];
    }
    v[k] = x;
    w[k] = y;
  }
  if constexpr (kWeighted) {
#pragma unroll
    for (int k = 0; k < kTileRows; ++k)
#pragma unroll
      for (int d = 0; d < 4; ++d) v[k][d] = pack_bf16x2(w[k] * bf16_lo(v[k][d]), w[k] * bf16_hi(v[k][d]));
  }
}

template <bool kWeighted, bool kStream>
__global__ __launch_bounds__(kTileThreads) void r128_mapped(TileArgs a, RowMap map) {
  __shared__ TileLds sh;
  const int rb = fdiv(blockIdx.x, a.col_tiles), ct = blockIdx.x - rb * a.col_tiles.d;
  int r0, r1;
  run_rows_once(a, sh, rb, r0, r1);
  if (r1 == r0) return;
  u32x4 v[kTileRows];
  mapped_values<kWeighted, kTileThreads>(a, map, ct, r0, r1, v);
  if (is_full(a, r1 - r0, ct))
    quant_tile<true, true, true, kStream>(a, sh, v, 0, rb, ct, r0, r1);
  else
    quant_tile<true, true, false, kStream>(a, sh, v, 0, rb, ct, r0, r1);
}

// For short runs: four column tiles to a workgroup (by_four: col_tiles / 4 of them, rounded
// up), side by side with 128 threads each where the run has up to 32 rows, else in turn.
// Of one tile each their number and the chain offsets, order, rows, scales bound them, whatever
// they hold: 128 tokens of 7168 to 8 of 64 experts 17.8 us, by fours 10.9; 500 of 4096 to
// 8 of 256 40.5 and 20; 32 rows an expert on average, even or by popularity: 20 and 21, 20
// and 16 (64 experts, 7168), 49 and 37, 49 and 29 (256, 4096).  With 96 28 and 37, 29 and 32
// (64); also lost where the tiles do not fill the GPU (1034 of 176 to 2 of 131: 4.7 and 5.0).
constexpr int kShortThreads = 128, kShortTiles = kTileThreads / kShortThreads, kShortRows = kRunLen / kShortTiles;

template <bool kWeighted, bool kStream>
__global__ __launch_bounds__(kTileThreads) void r128_mapped_short(TileArgs a, RowMap map, FastDiv by_four) {
  __shared__ TileLds sh[kShortTiles];
  const int rb = fdiv(blockIdx.x, by_four), ct0 = (blockIdx.x - rb * by_four.d) * kShortTiles;
  int r0, r1;
  run_rows<4>(a.offsets, a.groups, a.rows, rb, r0, r1);
  if (r1 == r0) return;
  u32x4 v[kTileRows];
  if (r1 - r0 <= kShortRows) {
    const int part = __builtin_amdgcn_readfirstlane(threadIdx.x / kShortThreads);
    mapped_values<kWeighted, kShortThreads>(a, map, ct0 + part, r0, r1, v);
    quant_tile<true, true, false, kStream, kShortThreads>(a, sh[part], v, 0, rb, ct0 + part, r0, r1);
    return;
  }
#pragma unroll 1
  for (int i = 0; i < kShortTiles && ct0 + i < (int)a.col_tiles.d; ++i) {
    mapped_values<kWeighted, kTileThreads>(a, map, ct0 + i, r0, r1, v);
    quant_tile<true, true, false, kStream>(a, sh[i], v, 0, rb, ct0 + i, r0, r1);
  }
}

}  // namespace

hipError_t launch_r128_cols(const void* src, int64_t batch, int64_t rows, int64_t cols, void* codes, void* scales,
                            hipStream_t stream) {
  const int64_t total = batch * rows, ct = (cols + kRunLen * kRunCols - 1) / (kRunLen * kRunCols);
  const int64_t grid = (total + kRunRows - 1) / kRunRows * ct;
  r128_cols<<<dim3((uint32_t)grid), dim3(kThreads), 0, stream>>>(
      static_cast<const uint16_t*>(src), static_cast<uint8_t*>(codes), static_cast<float*>(scales), total,
      make_fastdiv((uint32_t)rows), (int32_t)cols, make_fastdiv((uint32_t)ct));
  return hipGetLastError();
}

hipError_t launch_r128_tiles(const void* src, int64_t batch, int64_t rows, int64_t cols, const int32_t* offsets,
                             int64_t groups, void* codes_c, void* scales_c, void* codes_r, void* scales_r,
                             hipStream_t stream) {
  const int64_t ct = (cols + kRunLen - 1) / kRunLen;
  const int64_t rt = offsets ? rows / kRunLen + groups : (rows + kRunLen - 1) / kRunLen;
  const TileArgs a{static_cast<const uint16_t*>(src), static_cast<uint8_t*>(codes_c), static_cast<uint8_t*>(codes_r),
                   static_cast<float*>(scales_c), static_cast<float*>(scales_r), offsets, (int32_t)groups,
                   (int32_t)rows, (int32_t)cols, make_fastdiv((uint32_t)ct), make_fastdiv((uint32_t)rt)};
  const dim3 grid((uint32_t)(batch * rt * ct)), block(kTileThreads);
  if (codes_r == nullptr)
    r128_tile<false, false><<<grid, block, 0, stream>>>(a);
  else if (codes_c == nullptr)
    r128_tile<false, true><<<grid, block, 0, stream>>>(a);
  else
    r128_tile<true, true><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_moe_gather_quant(const void* x, int64_t tokens, int64_t topk, int64_t cols, const int32_t* order,
                                   const float* weights, const int32_t* offsets, int64_t groups, void* codes_c,
                                   void* scales_c, void* codes_r, void* scales_r, hipStream_t stream) {
  const int64_t rows = tokens * topk, ct = (cols + kRunLen - 1) / kRunLen, rt = rows / kRunLen + groups;
  const TileArgs a{static_cast<const uint16_t*>(x), static_cast<uint8_t*>(codes_c), static_cast<uint8_t*>(codes_r),
                   static_cast<float*>(scales_c), static_cast<float*>(scales_r), offsets, (int32_t)groups,
                   (int32_t)rows, (int32_t)cols, make_fastdiv((uint32_t)ct), make_fastdiv((uint32_t)rt)};
  const RowMap map{order, weights, make_fastdiv((uint32_t)topk), (uint32_t)rows};
  const dim3 grid((uint32_t)(rt * ct)), block(kTileThreads);
  const bool past = 2 * rows * cols > kCacheBytes;
  if (rows <= 32 * groups && rt * ct >= 1024) {
    const int64_t fours = (ct + kShortTiles - 1) / kShortTiles;
    const FastDiv by_four = make_fastdiv((uint32_t)fours);
    const dim3 few((uint32_t)(rt * fours));
    if (weights != nullptr)
      past ? r128_mapped_short<true, true><<<few, block, 0, stream>>>(a, map, by_four) : r128_mapped_short<true, false><<<few, block, 0, stream>>>(a, map, by_four);
    else
      past ? r128_mapped_short<false, true><<<few, block, 0, stream>>>(a, map, by_four) : r128_mapped_short<false, false><<<few, block, 0, stream>>>(a, map, by_four);
    return hipGetLastError();
  }
  if (weights != nullptr)
    past ? r128_mapped<true, true><<<grid, block, 0, stream>>>(a, map) : r128_mapped<true, false><<<grid, block, 0, stream>>>(a, map);
  else
    past ? r128_mapped<false, true><<<grid, block, 0, stream>>>(a, map) : r128_mapped<false, false><<<grid, block, 0, stream>>>(a, map);
  return hipGetLastError();
}

}  // namespace lp
