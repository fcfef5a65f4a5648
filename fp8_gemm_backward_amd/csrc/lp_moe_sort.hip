// (Token, slot) pairs sorted stably by expert: a counting sort.
//
//   row(i) = start(e_i) + number of pairs before i with the same expert
//
// A workgroup takes consecutive pairs, each of its waves up to kPer groups of 64 in
// a line.  In a wave, the lanes with the same expert find each other by one
// ballot per bit of the expert's number; a pair's rank is the wave's running
// count of its expert (LDS, one row of counters per wave) plus the lanes before it.
// Then one thread per expert turns the waves' counts into where each wave begins.
// What lies before the workgroup's pairs it counts itself (LDS additions of
// integers, whose order changes nothing), or, where the pairs are many, takes
// from two launches that count every chunk's experts and add them up.
//
// 96 pairs 3.3 us, 32768 of 64 experts 7.5, 2^20 15: a launch and a chain of
// dependent steps, then the counting of all pairs by every workgroup.
#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kPer = 4, kChunk = kThreads * kPer;
constexpr int kAhead = 32;             // pairs a thread loads before it counts them
constexpr int kMaxExperts = 1024;
// Up to so many pairs every workgroup counts them all itself, in one launch without a
// workspace (65536 pairs of 64 experts: 10.1 us; 131072 by three launches 11.4, and
// what three launches cost the host).  With 512 threads and eight groups a wave 32768 took 11.8 us for 7.1.
constexpr int64_t kCountedPairs = 65536;

struct SortArgs {
  const int32_t* experts;
  int64_t pairs;
  int32_t E, bits;
  int32_t chunks, per;         // workgroups, and how many groups of 64 pairs each of their waves takes
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

// Copies of the counters of what lies before and after a workgroup's pairs.
__host__ __device__ constexpr int copies_of(int experts) { return experts <= 256 ? 8 : 2; }

enum class Before { kNothing, kCounted, kScanned };             // what lies before the workgroup's pairs

template <Before kBefore>
__global__ __launch_bounds__(kThreads) void sort_place(SortArgs a) {
  __shared__ int32_t start[kMaxExperts];                         // first row of this workgroup's pairs
  __shared__ int32_t part[kWaves];
  extern __shared__ int32_t count[];                             // [kWaves][E]; kCounted: and [2][copies][odd], before and from there on
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  // Lanes that add to one address wait for one another, so neighbours add to copies.
  const int odd = a.E | 1, copies = copies_of(a.E);
  int32_t* const other = count + kWaves * a.E;
  for (int i = threadIdx.x; i < kWaves * a.E + (kBefore == Before::kCounted ? 2 * copies * odd : 0); i += kThreads) count[i] = 0;
  __syncthreads();
  if constexpr (kBefore == Before::kCounted) {
    const int pairs = (int)a.pairs, mine0 = blockIdx.x * kThreads * a.per, copy = (lane & (copies - 1)) * odd;
    for (int i0 = threadIdx.x; i0 < pairs; i0 += kAhead * kThreads) {
      int e[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) e[i] = i0 + i * kThreads < pairs ? a.experts[i0 + i * kThreads] : -1;
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if ((uint32_t)e[i] < (uint32_t)a.E) atomicAdd(&other[copy + e[i] + (i0 + i * kThreads < mine0 ? 0 : copies * odd)], 1);
    }
  }

  const int per = kBefore == Before::kCounted ? 1 : a.per;
  const int64_t first = ((int64_t)blockIdx.x * kWaves + wave) * (64 * per);
  int32_t* const mine = count + wave * a.E;
  int e[kPer], rank[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = first + 64 * i + lane;
    e[i] = i < per && p < a.pairs ? a.experts[p] : -1;
    if ((uint32_t)e[i] >= (uint32_t)a.E) e[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i >= per) break;
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
    int total = 0, earlier = 0;
    if (x < a.E) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int n = count[w * a.E + x];
        count[w * a.E + x] = total;
        total += n;
      }
      if constexpr (kBefore == Before::kCounted) {
        total = 0;
        for (int c = 0; c < copies; ++c) {
          earlier += other[c * odd + x];
          total += other[(copies + c) * odd + x];
        }
        total += earlier;
      }
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
      if constexpr (kBefore == Before::kCounted) at += earlier;
      if constexpr (kBefore == Before::kScanned) at += a.counts[(int64_t)x * a.chunks + blockIdx.x];
      start[x] = at;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = first + 64 * i + lane;
    if (i >= per || p >= a.pairs) continue;
    const int row = e[i] < 0 ? -1 : start[e[i]] + mine[e[i]] + rank[i];
    a.rows[p] = row;
    if (row >= 0) a.order[row] = (int32_t)p;
  }
}

}  // namespace

size_t moe_sort_workspace(int64_t pairs, int64_t experts) {
  return pairs <= kCountedPairs ? 0 : (size_t)(experts * ((pairs + kChunk - 1) / kChunk + 1)) * 4;
}

hipError_t launch_moe_sort(const int32_t* experts, int64_t pairs, int32_t groups, int32_t* offsets, int32_t* rows,
                           int32_t* order, void* ws, hipStream_t s) {
  SortArgs a{experts, pairs, groups, 0, 1, kPer, offsets, rows, order, nullptr, nullptr};
  while ((1 << a.bits) < groups) ++a.bits;
  const size_t lds = (size_t)kWaves * groups * 4;
  if (pairs <= 2 * kThreads) {           // (4096 pairs by one workgroup 6.2 us, by four 5.5)
    a.per = (int32_t)((pairs + kThreads - 1) / kThreads);
    sort_place<Before::kNothing><<<dim3(1), dim3(kThreads), lds, s>>>(a);
    return hipGetLastError();
  }
  if (pairs <= kCountedPairs) {
    a.per = 1;
    a.chunks = (int32_t)((pairs + kThreads - 1) / kThreads);
    sort_place<Before::kCounted><<<dim3((uint32_t)a.chunks), dim3(kThreads), lds + 8 * (size_t)copies_of(groups) * (groups | 1), s>>>(a);
    return hipGetLastError();
  }
  a.chunks = (int32_t)((pairs + kChunk - 1) / kChunk);
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
