// (Token, slot) pairs sorted stably by expert: a counting sort.
//
//   row(i) = start(e_i) + number of pairs before i with the same expert
//
// A workgroup takes kChunk consecutive pairs, each of its waves kPer groups of
// 64 in a line.  In a wave, the lanes with the same expert find each other by
// one ballot per bit of the expert's number; a pair's rank is the wave's
// running count of its expert (LDS, one row of counters per wave) plus the lanes
// before it.  Then one thread per expert turns the waves' counts into where
// each wave begins.  What lies before the workgroup's pairs comes from a
// first launch that counts every chunk's experts.
#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64, kPer = 8, kChunk = kThreads * kPer;
constexpr int kMaxExperts = 1024;

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

// Orders the wave's LDS accesses before it ahead of those after it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

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

template <bool kAlone>
__global__ __launch_bounds__(kThreads) void sort_place(SortArgs a) {
  __shared__ int32_t start[kMaxExperts];                         // first row of this workgroup's pairs
  __shared__ int32_t part[kWaves];
  extern __shared__ int32_t count[];                             // [kWaves][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  for (int i = threadIdx.x; i < kWaves * a.E; i += kThreads) count[i] = 0;
  __syncthreads();

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
      if constexpr (!kAlone) total = a.totals[x];
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
      start[x] = kAlone ? at : at + a.counts[(int64_t)x * a.chunks + blockIdx.x];
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
  return chunks <= 1 ? 0 : (size_t)(experts * (chunks + 1)) * 4;
}

hipError_t launch_moe_sort(const int32_t* experts, int64_t pairs, int32_t groups, int32_t* offsets, int32_t* rows,
                           int32_t* order, void* ws, hipStream_t s) {
  SortArgs a{experts, pairs, groups, 0, (int32_t)((pairs + kChunk - 1) / kChunk), offsets, rows, order, nullptr, nullptr};
  while ((1 << a.bits) < groups) ++a.bits;
  const size_t lds = (size_t)kWaves * groups * 4;
  if (a.chunks <= 1) {
    sort_place<true><<<dim3(1), dim3(kThreads), lds, s>>>(a);
    return hipGetLastError();
  }
  a.totals = static_cast<int32_t*>(ws);
  a.counts = a.totals + groups;
  sort_count<<<dim3((uint32_t)a.chunks), dim3(kThreads), 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  sort_scan<<<dim3((uint32_t)groups), dim3(kThreads), 0, s>>>(a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  sort_place<false><<<dim3((uint32_t)a.chunks), dim3(kThreads), lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace lp
