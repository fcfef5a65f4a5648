// Quantization of bf16 to E4M3 with an fp32 scale per run of 128 (along the
// columns, along the rows, or both from one read) or per 128 x 128 block
// (HBM-bound, bit-exact; the arithmetic is in lp_r128.hpp).
#include "lp_internal.hpp"
#include "lp_r128.hpp"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kRunLen = 128;

// Runs along the columns.  Sixteen lanes hold a run, eight values each, and
// take its largest magnitude with lane-row rotations.  A workgroup takes 16
// rows x 4 runs: a row's four runs are 1 KiB in a line, and the 16 rows'
// scales of one run index are 64 bytes in a line ([run][row]).  8192 x 4096 in
// 17.6 us (5.7 TB/s), 24 x 2048 in 3.2 us (a launch).
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
// 32768 x 2048 in 64 groups 79 us along both axes, this 54).
__device__ __forceinline__ void run_rows(const int32_t* __restrict__ offsets, int groups, int M, int run, int& r0,
                                         int& r1) {
  const int lane = threadIdx.x & 63;
  int end0 = 0;
  r0 = r1 = 0;
  for (int base = 0; base < groups; base += 64) {
    int e = base + lane < groups ? offsets[base + lane] : 0;
    e = e > M ? M : e;
    e = e < end0 ? end0 : e;
    e = wave_scan(e, [](int a, int b) { return a > b ? a : b; });
    int start = __shfl_up(e, 1);
    start = lane == 0 ? end0 : start;
    const int k = run - (start / kRunLen + base + lane);
    const uint64_t own = __ballot(k >= 0 && k < (e - start + kRunLen - 1) / kRunLen);
    if (own != 0) {
      const int j = __builtin_ctzll(own), end = __builtin_amdgcn_readlane(e, j);
      r0 = __builtin_amdgcn_readlane(start, j) + __builtin_amdgcn_readlane(k, j) * kRunLen;
      r1 = r0 + kRunLen < end ? r0 + kRunLen : end;
      return;
    }
    end0 = __builtin_amdgcn_readlane(e, 63);
  }
}

// One 128 x 128 tile per workgroup, for runs along the rows (kRows), along
// both axes (kRows and kCols) or one scale for the tile (neither).  Thread
// 16 i + c holds rows i + 32 k (k = 0..3) of columns 8 c .. 8 c + 7, so that
// each load of 16 lanes is 256 bytes in a line; a row's largest magnitude is
// taken over its 16 lanes, a column's over the thread's four rows, the four
// lane rows of the wave and, through LDS, the eight waves.  One thread per
// column then makes its scale while the others go on with the runs along the
// columns.  512 threads a tile: both axes of 1000 x 2064 in 5.8 us, 8192 x
// 4096 in 26.9 (5.0 TB/s); 256 threads 7.0 and 27.4, 1024 threads 5.7 and 29.0.
// With every thread making the scales of its eight columns: 6.2 and 27.7.
struct TileArgs {
  const uint16_t* src;
  uint8_t *codes_c, *codes_r;
  float *scales_c, *scales_r;
  const int32_t* offsets;
  int32_t groups, rows, cols;
  FastDiv col_tiles, row_tiles;            // row_tiles: runs (blocks) along the rows of one batch entry
};

constexpr int kTileThreads = 512, kTileWaves = kTileThreads / 64, kStep = kTileThreads / 16, kTileRows = kRunLen / kStep;

template <bool kCols, bool kRows>
__global__ __launch_bounds__(kTileThreads) void r128_tile(TileArgs a) {
  __shared__ alignas(16) uint16_t s_max[kTileWaves][kRunLen];
  __shared__ alignas(16) float s_scale[kRunLen], s_recip[kRunLen];
  const uint32_t rtile = fdiv(blockIdx.x, a.col_tiles);
  const int ct = blockIdx.x - rtile * a.col_tiles.d;
  const uint32_t b = fdiv(rtile, a.row_tiles);
  const int rb = rtile - b * a.row_tiles.d;
  int r0 = rb * kRunLen, r1 = r0 + kRunLen < a.rows ? r0 + kRunLen : a.rows;
  if (a.offsets != nullptr) {
    run_rows(a.offsets, a.groups, a.rows, rb, r0, r1);
    if (r1 == r0) return;
  }
  const int tid = threadIdx.x, ci = tid & 15, ri = tid >> 4, wave = tid >> 6;
  const int c = ct * kRunLen + 8 * ci;
  const bool col_ok = c < a.cols;
  const int64_t base = ((int64_t)b * a.rows + r0) * a.cols + c;
  u32x4 v[kTileRows];
#pragma unroll
  for (int k = 0; k < kTileRows; ++k) {
    const int r = ri + kStep * k;
    v[k] = col_ok && r0 + r < r1 ? *reinterpret_cast<const u32x4*>(a.src + base + (int64_t)r * a.cols)
                                 : u32x4{0u, 0u, 0u, 0u};
  }
  // Column maxima (bf16 magnitude pairs).
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
  if ((tid & 63) < 16) *reinterpret_cast<u32x4*>(&s_max[wave][8 * ci]) = cm;
  __syncthreads();
  if constexpr (kRows) {
    if (tid < kRunLen) {                                   // one column's scale per thread
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kTileWaves; ++w) m = umax(m, s_max[w][tid]);
      const RunScale q = run_scale(m << 16);
      s_scale[tid] = q.s;
      s_recip[tid] = q.r;
      if (ct * kRunLen + tid < a.cols)
        a.scales_r[((int64_t)b * a.row_tiles.d + rb) * a.cols + ct * kRunLen + tid] = q.s;
    }
  }
  if constexpr (kCols) {
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
      const int r = ri + kStep * k;
      const RunScale q = run_scale(row16_max(amax8(v[k])));
      if (r0 + r >= r1) continue;
      if (ci == 0) a.scales_c[((int64_t)b * a.col_tiles.d + ct) * a.rows + r0 + r] = q.s;
      if (col_ok) *reinterpret_cast<u32x2*>(a.codes_c + base + (int64_t)r * a.cols) = run_codes8(v[k], q);
    }
  }
  if constexpr (kRows) {
    __syncthreads();
    RunScale q[8];
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      q[e].s = s_scale[8 * ci + e];
      q[e].r = s_recip[8 * ci + e];
      q[e].bad = __builtin_isnan(q[e].s);
      bad |= q[e].bad;
    }
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
      const int r = ri + kStep * k;
      uint32_t o[2];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const uint32_t w0 = v[k][2 * d], w1 = v[k][2 * d + 1];
        o[d] = to_e4m3x2(run_div(bf16_lo(w0), q[4 * d]), run_div(bf16_hi(w0), q[4 * d + 1])) |
               (to_e4m3x2(run_div(bf16_lo(w1), q[4 * d + 2]), run_div(bf16_hi(w1), q[4 * d + 3])) << 16);
        if (__builtin_expect(bad, false)) {
          const uint32_t nan = nan_e4m3x2(w0) | (nan_e4m3x2(w1) << 16);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (q[4 * d + e].bad) o[d] = (o[d] & ~(0xFFu << (8 * e))) | (nan & (0xFFu << (8 * e)));
        }
      }
      if (col_ok && r0 + r < r1) *reinterpret_cast<u32x2*>(a.codes_r + base + (int64_t)r * a.cols) = u32x2{o[0], o[1]};
    }
  }
  if constexpr (!kCols && !kRows) {
#pragma unroll
    for (int w = 0; w < kTileWaves; ++w) {
      const u32x4 o = *reinterpret_cast<const u32x4*>(&s_max[w][8 * ci]);
#pragma unroll
      for (int d = 0; d < 4; ++d) cm[d] = pk_umax16(cm[d], o[d]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) m = umax(m, umax(cm[d] & 0xFFFFu, cm[d] >> 16));
    const RunScale q = run_scale(row16_max(m) << 16);
    if (tid == 0) a.scales_c[((int64_t)b * a.row_tiles.d + rb) * a.col_tiles.d + ct] = q.s;
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
      const int r = ri + kStep * k;
      if (col_ok && r0 + r < r1)
        *reinterpret_cast<u32x2*>(a.codes_c + base + (int64_t)r * a.cols) = run_codes8(v[k], q);
    }
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

}  // namespace lp
