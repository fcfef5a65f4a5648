// The router's gate: softmax over a token's expert logits, its k largest, and
// the gradient.
//
//   p = softmax(l), S = chosen;  w_j = p_{e_j}, or p_{e_j} / sum_S p
//   dl_i = p_i ([i in S] g_i - sum_S w g), or w_i (g_i - sum_S w g) on S
//
// Up to 256 experts 16 lanes own a token (four a wave), else a wave does; a lane
// holds up to 16 logits.  Every logit gets a key that orders as it does and
// carries its index, lower indices higher, so that no two are equal: 32 bits for
// bf16 logits, 64 for fp32.  A lane sorts its keys once (Batcher's odd-even
// merges); then the largest of the lanes' first keys is the next choice, k times,
// and its lane moves its keys up.  The first choice is the softmax's largest
// logit.  No logit is read twice; sums are fp32.  The gradient adds the chosen
// slots' parts to the softmax's in LDS.
//
// 32768 tokens of 256 bf16 logits, 8 chosen: 10.2 us, the gradient 9.4 after it, 11.3 of
// logits out of the caches (17 and 36 MB, 3.3 and 7.0 us of copying; with a wave to a
// token and the lane's best logit sought anew for each choice 32.4 and 22.0).  fp32:
// 17.0 and 16.4 (34 and 69 MB, 6.7 and 13.5 us).  The choice is bound by instructions,
// 554 a wave of four bf16 tokens: 7.6 us of every SIMD, 73% of the kernel's time with its
// launch and its last waves; the gradient by its bytes.
#include <math.h>

#include <type_traits>

#include "lp_device.hpp"
#include "lp_internal.hpp"

namespace lp {

namespace {

constexpr int kWaves = 4;
constexpr int64_t kMaxBlocks = 1 << 20;

struct GateArgs {
  const void* logits;
  const float* grad_w;
  float* weights;
  int32_t* chosen;
  const float* weights_in;
  const int32_t* chosen_in;
  void* grad_l;
  int64_t tokens;
  int32_t E, k;
  bool renorm;
};

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {            // (a lane without a source gets 0)
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}
template <int kCtrl>
__device__ __forceinline__ int32_t dpp(int32_t v) {
  return (int32_t)dpp<kCtrl>((uint32_t)v);
}
template <int kCtrl>
__device__ __forceinline__ uint64_t dpp(uint64_t v) {
  return (uint64_t)dpp<kCtrl>((uint32_t)(v >> 32)) << 32 | dpp<kCtrl>((uint32_t)v);
}
template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<kCtrl>(__builtin_bit_cast(uint32_t, v)));
}

template <int kLane>
__device__ __forceinline__ uint32_t of_lane(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, kLane); }
template <int kLane>
__device__ __forceinline__ int32_t of_lane(int32_t v) { return __builtin_amdgcn_readlane(v, kLane); }
template <int kLane>
__device__ __forceinline__ uint64_t of_lane(uint64_t v) {
  return (uint64_t)of_lane<kLane>((uint32_t)(v >> 32)) << 32 | of_lane<kLane>((uint32_t)v);
}
template <int kLane>
__device__ __forceinline__ float of_lane(float v) {
  return __builtin_bit_cast(float, of_lane<kLane>(__builtin_bit_cast(uint32_t, v)));
}

// Reduction over the token's lanes, in all of them.
template <int kLanes, class T, class F>
__device__ __forceinline__ T over_lanes(T v, F op) {
  v = op(v, dpp<0x128>(v));                                      // row_ror:8
  v = op(v, dpp<0x124>(v));
  v = op(v, dpp<0x122>(v));
  v = op(v, dpp<0x121>(v));
  if constexpr (kLanes == 64) {
    v = op(v, dpp<0x142>(v));                                    // row_bcast:15: the last 16 lanes get the 16 before
    v = op(v, dpp<0x143>(v));                                    // row_bcast:31: and the first 32
    v = of_lane<63>(v);
  }
  return v;
}
template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
  return over_lanes<kLanes>(v, [](float a, float b) { return a + b; });
}
template <class T>
__device__ __forceinline__ T larger(T a, T b) { return a > b ? a : b; }

template <class T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 2) return __builtin_bit_cast(float, (uint32_t)v << 16);
  else return v;
}
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, v); }

// e^d for d <= 0 (NaN for NaN and infinity): 2^t with t = d log2 e split into a
// rounded part and its residual, relative error below 2^-22 whatever d; 0 where the
// result is no normal number.
__device__ __forceinline__ float exp_of(float d) {
  constexpr float kLog2e = 0x1.715476p+0f, kLow = 0x1.4ae0bep-26f;        // log2 e = kLog2e + kLow
  const float t = d * kLog2e;
  const float e = __builtin_amdgcn_exp2f(t);
  const float r = __builtin_fmaf(d, kLow, __builtin_fmaf(d, kLog2e, -t));
  return t < -126.0f ? 0.0f : __builtin_fmaf(e, r * 0x1.62e43p-1f, e);
}

// The same as a term of a softmax's sum: without the residual e^d is off by |d| 2^-24 of
// itself, the sum by the softmax's mean of |d|, which is below ln E (its entropy is),
// times 2^-24.
__device__ __forceinline__ float exp_in_sum(float d) { return __builtin_amdgcn_exp2f(d * 0x1.715476p+0f); }

// m (all ones or none): a, else b.  By bits (one instruction of 32): as selections by
// condition the moves of 16 keys compared anew for each of them, 52 us a gate for 13.
__device__ __forceinline__ uint32_t pick(uint32_t m, uint32_t a, uint32_t b) { return (a & m) | (b & ~m); }
__device__ __forceinline__ int32_t pick(uint32_t m, int32_t a, int32_t b) { return (int32_t)pick(m, (uint32_t)a, (uint32_t)b); }
__device__ __forceinline__ uint64_t pick(uint32_t m, uint64_t a, uint64_t b) {
  return (uint64_t)pick(m, (uint32_t)(a >> 32), (uint32_t)(b >> 32)) << 32 | pick(m, (uint32_t)a, (uint32_t)b);
}
__device__ __forceinline__ uint32_t mask_of(bool c) {
  uint32_t m = c ? ~0u : 0u;
  asm volatile("" : "+v"(m));                                    // (kept a mask)
  return m;
}

// The lane's logits: numbers kItems lane + i where the row divides into aligned pieces
// (kWide: wide loads), else kLanes i + lane.
template <class T, int kItems>
constexpr int piece_of() { return kItems < 16 / (int)sizeof(T) ? kItems : 16 / (int)sizeof(T); }
template <int kLanes, int kItems, bool kWide>
__device__ __forceinline__ int logit_index(int lane, int i) { return kWide ? kItems * lane + i : kLanes * i + lane; }

// A logit's key: above all keys of smaller logits and of equal ones (0 and -0 are) with
// a higher index; below kNone, or at it, for -inf and past the last expert.  NaN counts
// as +inf.  Of bf16 32 bits: the signed magnitude in two's complement, then the index
// downwards, whose part by lane (lane_code) is added to the lane's first key only.
template <class T>
using Key = std::conditional_t<sizeof(T) == 2, int32_t, uint64_t>;
template <class T>
constexpr Key<T> kNone = sizeof(T) == 2 ? (Key<T>)0x8080FFFF : 0;           // (-0x7F80: -inf)
template <class T>
constexpr Key<T> kLast = sizeof(T) == 2 ? (Key<T>)0x80000000 : 0;
template <class T, int kLanes, int kItems, bool kWide>
__device__ __forceinline__ Key<T> key_of(float v, int lane, int i) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    return (int32_t)(pick((uint32_t)((int32_t)b >> 31), 0x80000000u - b, b) | (kWide ? kItems - 1 - i : (kItems - 1 - i) * kLanes));
  } else {
    v += 0.0f;                                                   // (-0 equals 0)
    const uint32_t b = __builtin_bit_cast(uint32_t, v), up = (int32_t)b < 0 ? ~b : b | 0x80000000u;
    if (v == -INFINITY) return 0;
    return (uint64_t)up << 32 | (0xFFFFFFFFu - (uint32_t)logit_index<kLanes, kItems, kWide>(lane, i));
  }
}
template <class T, int kLanes, int kItems, bool kWide>
__device__ __forceinline__ Key<T> lane_code(int lane) {
  if constexpr (sizeof(T) == 2) return kWide ? (kLanes - 1 - lane) * kItems : kLanes - 1 - lane;
  else return 0;
}
template <class T, int kLanes, int kItems>
__device__ __forceinline__ int index_of(Key<T> k) {
  if constexpr (sizeof(T) == 2) return kLanes * kItems - 1 - (k & 0xFFFF);
  else return (int)(0xFFFFFFFFu - (uint32_t)k);
}
template <class T>
__device__ __forceinline__ float value_of(Key<T> k) {
  uint32_t b;
  if constexpr (sizeof(T) == 2) {
    b = (uint32_t)k & 0xFFFF0000u;
    b = k < 0 ? 0x80000000u - b : b;
  } else {
    b = (uint32_t)(k >> 32);
    b = (int32_t)b < 0 ? b ^ 0x80000000u : ~b;
  }
  return __builtin_bit_cast(float, b);
}

template <class K>
__device__ __forceinline__ void in_order(K& a, K& b) {           // larger first
  const K x = a, y = b;
  a = larger(x, y);
  b = x > y ? y : x;
}

// Largest first.
template <int kN, class K>
__device__ __forceinline__ void sort_items(K* a) {
#pragma unroll
  for (int p = 1; p < kN; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < kN; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < kN && (i + j) / (2 * p) == (i + j + q) / (2 * p)) in_order(a[i + j], a[i + j + q]);
}

// The kKeep largest of kItems first, largest first.  Half of them: both halves sorted,
// the larger of each one's i-th and the other's i-th from the end kept (which rises,
// then falls), and that sorted by halving distances.
template <int kItems, int kKeep, class K>
__device__ __forceinline__ void sort_largest(K (&a)[kItems]) {
  if constexpr (kKeep == kItems) {
    sort_items<kItems>(a);
  } else {
    static_assert(2 * kKeep == kItems);
    sort_items<kKeep>(a);
    sort_items<kKeep>(a + kKeep);
#pragma unroll
    for (int i = 0; i < kKeep; ++i) a[i] = larger(a[i], a[kItems - 1 - i]);
#pragma unroll
    for (int q = kKeep / 2; q >= 1; q /= 2)
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if ((i & q) == 0) in_order(a[i], a[i + q]);
  }
}

template <class T, int kLanes, int kItems, bool kWide>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, float (&v)[kItems]) {
  if constexpr (kWide) {
    constexpr int kPiece = piece_of<T, kItems>();
    struct alignas(kPiece * sizeof(T)) Piece {
      T t[kPiece];
    };
    const Piece* const from = reinterpret_cast<const Piece*>(row + kItems * lane);
    Piece w[kItems / kPiece] = {};
    if (E == kLanes * kItems) {                                  // (32768 rows of 256 bf16: 9.9 us, 11.6 by the branches below)
#pragma unroll
      for (int p = 0; p < kItems / kPiece; ++p) w[p] = from[p];
    } else {
#pragma unroll
      for (int p = 0; p < kItems / kPiece; ++p)
        if (kItems * lane + p * kPiece < E) w[p] = from[p];
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      v[i] = kItems * lane + i / kPiece * kPiece < E ? to_f32(w[i / kPiece].t[i % kPiece]) : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      const int e = kLanes * i + lane;
      v[i] = e < E ? to_f32(row[e]) : -INFINITY;
    }
  }
}

// kKeep: of a lane's logits, at least min(k, kItems).
template <class T, int kLanes, int kItems, bool kWide, int kKeep>
__global__ __launch_bounds__(64 * kWaves) void gate_kernel(GateArgs a) {
  constexpr int kPer = 64 / kLanes, kOut = 64 / kLanes;          // tokens of a wave; slots of a lane (k <= 64)
  const int lane = threadIdx.x % kLanes, group = threadIdx.x % 64 / kLanes * kLanes;
  const Key<T> code = lane_code<T, kLanes, kItems, kWide>(lane);
  for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + threadIdx.x / 64) * kPer; t0 < a.tokens; t0 += (int64_t)gridDim.x * kWaves * kPer) {
    const int64_t t = t0 + group / kLanes, row = t < a.tokens ? t : a.tokens - 1;
    float v[kItems];
    load_logits<T, kLanes, kItems, kWide>(static_cast<const T*>(a.logits) + row * a.E, a.E, lane, v);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kItems; i += 2) nan |= __builtin_isunordered(v[i], v[i + 1 < kItems ? i + 1 : i]);
    const uint64_t nans = __ballot(nan);
    if (nans != 0) {
#pragma unroll
      for (int i = 0; i < kItems; ++i) v[i] = v[i] != v[i] ? INFINITY : v[i];
    }
    nan = (nans >> group & (kLanes == 64 ? ~0ull : (1ull << kLanes) - 1)) != 0;
    Key<T> left[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      left[i] = key_of<T, kLanes, kItems, kWide>(v[i], lane, i);
      if (!kWide && logit_index<kLanes, kItems, kWide>(lane, i) >= a.E) left[i] = kLast<T>;
    }
    sort_largest<kItems, kKeep>(left);
    Key<T> mine[kOut], first = 0;
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      mine[o] = kLast<T>;
      for (int j = o * kLanes; j < a.k && j < (o + 1) * kLanes; ++j) {
        const Key<T> own = left[0] + code, best = over_lanes<kLanes>(own, [](Key<T> x, Key<T> y) { return larger(x, y); });
        if (o == 0) first = j == 0 ? best : first;
        mine[o] = pick(mask_of(lane == j - o * kLanes), best, mine[o]);
        const uint32_t taken = mask_of(own == best);             // (they differ but where nothing is left)
#pragma unroll
        for (int i = 0; i + 1 < kKeep; ++i) left[i] = pick(taken, left[i + 1], left[i]);
        left[kKeep - 1] = pick(taken, kLast<T>, left[kKeep - 1]);
      }
    }
    const float peak = first > kNone<T> ? value_of<T>(first) : 0.0f;
    float w[kOut], total = 0.0f;
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      w[o] = mine[o] > kNone<T> ? exp_of(value_of<T>(mine[o]) - peak) : 0.0f;
      total += w[o];
    }
    if (!a.renorm) {
      total = 0.0f;
#pragma unroll
      for (int i = 0; i < kItems; ++i) total += exp_in_sum(v[i] - peak);
    }
    total = sum_lanes<kLanes>(total);
    if (t >= a.tokens) continue;
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      const int j = o * kLanes + lane;
      if (j >= a.k) continue;
      const bool some = mine[o] > kNone<T>;
      a.weights[t * a.k + j] = !some ? 0.0f : nan ? NAN : w[o] / total;
      a.chosen[t * a.k + j] = some ? index_of<T, kLanes, kItems>(mine[o]) : -1;
    }
  }
}

template <class T, int kLanes, int kItems, bool kWide>
__global__ __launch_bounds__(64 * kWaves) void gate_bwd_kernel(GateArgs a) {
  constexpr int kPer = 64 / kLanes, kOut = 64 / kLanes, kRow = kLanes * kItems;
  __shared__ __attribute__((aligned(16))) float s_grad[kWaves * kPer][kRow];
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x % 64 / kLanes;
  float* const d = s_grad[threadIdx.x / 64 * kPer + sub];       // the token's gradient
  for (int64_t t0 = ((int64_t)blockIdx.x * kWaves + threadIdx.x / 64) * kPer; t0 < a.tokens; t0 += (int64_t)gridDim.x * kWaves * kPer) {
    const int64_t t = t0 + sub, row = t < a.tokens ? t : a.tokens - 1;
    int e[kOut];
    float v[kItems], w[kOut], g[kOut], inner = 0.0f;
    if (!a.renorm) load_logits<T, kLanes, kItems, kWide>(static_cast<const T*>(a.logits) + row * a.E, a.E, lane, v);
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      const int j = o * kLanes + lane;
      e[o] = j < a.k ? a.chosen_in[row * a.k + j] : -1;
      if ((uint32_t)e[o] >= (uint32_t)a.E) e[o] = -1;
      w[o] = e[o] >= 0 ? a.weights_in[row * a.k + j] : 0.0f;
      g[o] = e[o] >= 0 ? a.grad_w[row * a.k + j] : 0.0f;
      inner += w[o] * g[o];
    }
    inner = sum_lanes<kLanes>(inner);
    if (!a.renorm) {
      float peak = -INFINITY, total = 0.0f;
#pragma unroll
      for (int i = 0; i < kItems; ++i) peak = __builtin_fmaxf(peak, v[i]);
      peak = over_lanes<kLanes>(peak, [](float x, float y) { return __builtin_fmaxf(x, y); });
      peak = peak == -INFINITY ? 0.0f : peak;                    // (then every exponential is 0)
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        // (beside a bf16 gradient's rounding |d| 2^-24 is nothing)
        v[i] = sizeof(T) == 2 ? exp_in_sum(v[i] - peak) : exp_of(v[i] - peak);
        total += v[i];
      }
      total = sum_lanes<kLanes>(total);
      const float scale = total == 0.0f ? 0.0f : -inner / total;
#pragma unroll
      for (int i = 0; i < kItems; ++i) v[i] *= scale;
    } else {
#pragma unroll
      for (int i = 0; i < kItems; ++i) v[i] = 0.0f;
    }
    // The chosen ones' own part: all slots at once, or one after the other where an expert
    // comes twice, which shows in whose number its place keeps.
    uint32_t* const owner = reinterpret_cast<uint32_t*>(d);
    bool twice = false;
#pragma unroll
    for (int o = 0; o < kOut; ++o)
      if (e[o] >= 0) owner[e[o]] = o * kLanes + lane;
    wave_sync();
#pragma unroll
    for (int o = 0; o < kOut; ++o)
      if (e[o] >= 0) twice |= owner[e[o]] != (uint32_t)(o * kLanes + lane);
    const bool serial = __ballot(twice) != 0;
    wave_sync();
#pragma unroll
    for (int i = 0; i < kItems; ++i) d[logit_index<kLanes, kItems, kWide>(lane, i)] = v[i];
    wave_sync();
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      const float own = a.renorm ? w[o] * (g[o] - inner) : w[o] * g[o];
      if (!serial) {
        if (e[o] >= 0) d[e[o]] += own;
      } else {
#pragma unroll 1
        for (int j = 0; j < kLanes && o * kLanes + j < a.k; ++j) {
          if (lane == j && e[o] >= 0) d[e[o]] += own;
          wave_sync();
        }
      }
    }
    wave_sync();
    if (t < a.tokens) {
      T* const out = static_cast<T*>(a.grad_l) + t * a.E;
      if constexpr (kWide && sizeof(T) == 2 && kItems >= 2) {
        constexpr int kPiece = piece_of<T, kItems>();
        struct alignas(kPiece * sizeof(T)) Piece {
          uint32_t w[kPiece / 2];
        };
#pragma unroll
        for (int i = 0; i < kItems; i += kPiece) {
          const float* const g = d + kItems * lane + i;
          Piece o;
#pragma unroll
          for (int j = 0; j < kPiece / 2; ++j) o.w[j] = pack_bf16x2(g[2 * j], g[2 * j + 1]);
          if (kItems * lane + i < a.E) *reinterpret_cast<Piece*>(out + kItems * lane + i) = o;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
          const int x = kLanes * i + lane;
          if (x < a.E) store(out + x, d[x]);
        }
      }
    }
    wave_sync();                                                 // the next token's gradient goes there
  }
}

// Up to 8 chosen, 8 of a lane's 16 logits are enough (8 of 256 for 32768 tokens: 9.9 us,
// 11.6 with all kept).
template <class T, int kLanes, int kItems, bool kWide>
void launch_gate(const GateArgs& a, dim3 grid, dim3 block, hipStream_t s) {
  if (kItems == 16 && a.k <= 8) gate_kernel<T, kLanes, kItems, kWide, kItems == 16 ? 8 : kItems><<<grid, block, 0, s>>>(a);
  else gate_kernel<T, kLanes, kItems, kWide, kItems><<<grid, block, 0, s>>>(a);
}

template <class T, int kLanes, int kItems>
void launch(const GateArgs& a, bool bwd, hipStream_t s) {
  const int64_t per = kWaves * (64 / kLanes), blocks = (a.tokens + per - 1) / per;
  const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), block(64 * kWaves);
  constexpr uintptr_t kPiece = piece_of<T, kItems>(), kWord = kPiece * sizeof(T);
  const bool wide = a.E % kPiece == 0 && reinterpret_cast<uintptr_t>(a.logits) % kWord == 0 &&
                    reinterpret_cast<uintptr_t>(a.grad_l) % kWord == 0;
  if (bwd)
    wide ? gate_bwd_kernel<T, kLanes, kItems, true><<<grid, block, 0, s>>>(a)
         : gate_bwd_kernel<T, kLanes, kItems, false><<<grid, block, 0, s>>>(a);
  else
    wide ? launch_gate<T, kLanes, kItems, true>(a, grid, block, s) : launch_gate<T, kLanes, kItems, false>(a, grid, block, s);
}

template <class T>
hipError_t dispatch(const GateArgs& a, bool bwd, hipStream_t s) {
  if (a.E <= 16) launch<T, 16, 1>(a, bwd, s);
  else if (a.E <= 32) launch<T, 16, 2>(a, bwd, s);
  else if (a.E <= 64) launch<T, 16, 4>(a, bwd, s);
  else if (a.E <= 128) launch<T, 16, 8>(a, bwd, s);
  else if (a.E <= 256) launch<T, 16, 16>(a, bwd, s);
  else if (a.E <= 512) launch<T, 64, 8>(a, bwd, s);
  else launch<T, 64, 16>(a, bwd, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_gate(const void* logits, bool bf16, int64_t tokens, int32_t experts, int32_t topk, bool renorm,
                           float* weights, int32_t* chosen, hipStream_t s) {
  const GateArgs a{logits, nullptr, weights, chosen, nullptr, nullptr, nullptr, tokens, experts, topk, renorm};
  return bf16 ? dispatch<uint16_t>(a, false, s) : dispatch<float>(a, false, s);
}

hipError_t launch_moe_gate_bwd(const float* grad_w, const void* logits, bool bf16, int64_t tokens, int32_t experts,
                               int32_t topk, bool renorm, const float* weights, const int32_t* chosen, void* grad_l,
                               hipStream_t s) {
  const GateArgs a{logits, grad_w, nullptr, nullptr, weights, chosen, grad_l, tokens, experts, topk, renorm};
  return bf16 ? dispatch<uint16_t>(a, true, s) : dispatch<float>(a, true, s);
}

}  // namespace lp
