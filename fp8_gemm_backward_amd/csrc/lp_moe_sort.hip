// (Token, slot) pairs sorted stably by expert: a counting sort.
//
//   row(i) = start(e_i) + number of pairs before i with the same expert
//
// A workgroup takes kChunk consecutive pairs, each of its waves kPer groups of
// 64 in a line.  In a wave, the lanes with the same expert find each other by
// one ballot per bit of the expert's number; a pair's rank is the wave's
// running count of its expert (LDS, one row of counters per wave) plus the lanes
// before it.  Then one thread per expert turns the waves' counts into where
// each wave begins.  What lies before the workgroup's pairs it counts itself (LDS
// additions of integers, whose order changes nothing), or, where the pairs are
// many, takes from two launches that count every chunk's experts and add them up.
#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64, kPer = 8, kChunk = kThreads * kPer;
constexpr int kMaxExperts = 1024;
// Up to so many chunks every workgroup counts all pairs itself, in one launch without
// a workspace (32768 pairs of 64 experts: 10.8 us, 18 by three launches).
constexpr int kCountChunks = 16;

struct SortArgs {
  const int32_t* experts;
  int64_t pairs;
  int32_t E, bits;
  int32_t chunks;
  int32_t* offsets;
  int32_t* rows;
  int32_t* order;
  int32_t* counts;             // [E][chunks]: per chunk, then (scanned) the pairs of the expert before the chunk
  int32_t* totals;             // [E]
};

// Sum over the wave's lanes up to each lane.
__device__ __forceinline__ int wave_prefix(int v) {
  return wave_scan(v, [](int a, int b) { return a + b; });
}

__global__ __launch_bounds__(kThreads) void sort_count(SortArgs a) {
  __shared__ int32_t count[kMaxExperts];
  for (int e = threadIdx.x; e < a.E; e += kThreads) count[e] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kChunk;
  for (int i = threadIdx.x; i < kChunk; i += kThreads) {
    const int e = base + i < a.pairs ? a.experts[base + i] : -1;
    if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&count[e], 1);    // (LDS; sums of integers)
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) a.counts[(int64_t)e * a.chunks + blockIdx.x] = count[e];
}

// One workgroup per expert: its chunks' counts become what lies before them.
__global__ __launch_bounds__(kThreads) void sort_scan(SortArgs a) {
  __shared__ int32_t part[kWaves];
  int32_t* c = a.counts + (int64_t)blockIdx.x * a.chunks;
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  int before = 0;
  for (int base = 0; base < a.chunks; base += kThreads) {
    const int i = base + threadIdx.x, v = i < a.chunks ? c[i] : 0, s = wave_prefix(v);
    if (lane == 63) part[wave] = s;
    __syncthreads();
    int mine = before + s - v;
    for (int w = 0; w < kWaves; ++w) {
      mine += w < wave ? part[w] : 0;
      before += part[w];
    }
    if (i < a.chunks) c[i] = mine;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.totals[blockIdx.x] = before;
}

enum class Before { kNothing, kCounted, kScanned };             // what lies before the workgroup's pairs

template <Before kBefore>
__global__ __launch_bounds__(kThreads) void sort_place(SortArgs a) {
  __shared__ int32_t start[kMaxExperts];                         // first row of this workgroup's pairs
  __shared__ int32_t part[kWaves];
  extern __shared__ int32_t count[];                             // [kWaves][E]; kCounted: and [2][E], before and from there on
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  int32_t* const other = count + kWaves * a.E;
  for (int i = threadIdx.x; i < (kWaves + (kBefore == Before::kCounted ? 2 : 0)) * a.E; i += kThreads) count[i] = 0;
  __syncthreads();
  if constexpr (kBefore == Before::kCounted) {
    const int pairs = (int)a.pairs, mine0 = blockIdx.x * kChunk;
    for (int i0 = threadIdx.x; i0 < pairs; i0 += kPer * kThreads) {
      int e[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) e[i] = i0 + i * kThreads < pairs ? a.experts[i0 + i * kThreads] : -1;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if ((uint32_t)e[i] < (uint32_t)a.E) atomicAdd(&other[e[i] + (i0 + i * kThreads < mine0 ? 0 : a.E)], 1);
    }
  }

  const int64_t first = (int64_t)blockIdx.x * kChunk + wave * (64 * kPer);
  int32_t* const mine = count + wave * a.E;
  int e[kPer], rank[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = first + 64 * i + lane;
    e[i] = p < a.pairs ? a.experts[p] : -1;
    if ((uint32_t)e[i] >= (uint32_t)a.E) e[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    uint64_t same = __ballot(e[i] >= 0);
    for (int b = 0; b < a.bits; ++b) {
      const bool bit = (e[i] >> b) & 1;
      const uint64_t set = __ballot(bit);
      same &= bit ? set : ~set;
    }
    int seen = 0;
    if (e[i] >= 0) seen = mine[e[i]];
    const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
    rank[i] = seen + before;
    wave_sync();
    if (e[i] >= 0 && before == 0) mine[e[i]] = seen + __builtin_popcountll(same);
    wave_sync();
  }
  __syncthreads();

  // Per expert: the waves' counts become what lies before them, and the
  // experts' totals their first rows.
  int carry = 0;
  for (int base = 0; base < a.E; base += kThreads) {
    const int x = base + threadIdx.x;
    int total = 0;
    if (x < a.E) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int n = count[w * a.E + x];
        count[w * a.E + x] = total;
        total += n;
      }
      if constexpr (kBefore == Before::kCounted) total = other[x] + other[a.E + x];
      if constexpr (kBefore == Before::kScanned) total = a.totals[x];
    }
    const int s = wave_prefix(total);
    if (lane == 63) part[wave] = s;
    __syncthreads();
    int at = carry + s - total;
    for (int w = 0; w < kWaves; ++w) {
      at += w < wave ? part[w] : 0;
      carry += part[w];
    }
    if (x < a.E) {
      if (blockIdx.x == 0) a.offsets[x] = at + total;
      if constexpr (kBefore == Before::kCounted) at += other[x];
      if constexpr (kBefore == Before::kScanned) at += a.counts[(int64_t)x * a.chunks + blockIdx.x];
      start[x] = at;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = first + 64 * i + lane;
    if (p >= a.pairs) continue;
    const int row = e[i] < 0 ? -1 : start[e[i]] + mine[e[i]] + rank[i];
    a.rows[p] = row;
    if (row >= 0) a.order[row] = (int32_t)p;
  }
}

}  // namespace

size_t moe_sort_workspace(int64_t pairs, int64_t experts) {
  const int64_t chunks = (pairs + kChunk - 1) / kChunk;
  return chunks <= kCountChunks ? 0 : (size_t)(experts * (chunks + 1)) * 4;
}

hipError_t launch_moe_sort(const int32_t* experts, int64_t pairs, int32_t groups, int32_t* offsets, int32_t* rows,
                           int32_t* order, void* ws, hipStream_t s) {
  SortArgs a{experts, pairs, groups, 0, (int32_t)((pairs + kChunk - 1) / kChunk), offsets, rows, order, nullptr, nullptr};
  while ((1 << a.bits) < groups) ++a.bits;
  const size_t lds = (size_t)kWaves * groups * 4;
  if (a.chunks <= 1) {
    sort_place<Before::kNothing><<<dim3(1), dim3(kThreads), lds, s>>>(a);
    return hipGetLastError();
  }
  if (a.chunks <= kCountChunks) {
    sort_place<Before::kCounted><<<dim3((uint32_t)a.chunks), dim3(kThreads), lds + 8 * (size_t)groups, s>>>(a);
    return hipGetLastError();
  }
  a.totals = static_cast<int32_t*>(ws);
  a.counts = a.totals + groups;
  sort_count<<<dim3((uint32_t)a.chunks), dim3(kThreads), 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sort_scan<<<dim3((uint32_t)groups), dim3(kThreads), 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  sort_place<Before::kScanned><<<dim3((uint32_t)a.chunks), dim3(kThreads), lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace lp
