// The router's gate: softmax over a token's expert logits, its k largest, and
// the gradient.
//
// A wave owns a token.  Lane l holds the logits kItems l .. kItems (l + 1) - 1,
// so that the lowest lane, then the lowest of its items, is the lowest index
// of equal logits.  Per slot: the wave's maximum of the lanes' largest items
// left (DPP), one ballot for the lane, and that lane looks for its next one.
// No logit is read twice; sums are fp32.
//
//   p = softmax(l), S = chosen;  w_j = p_{e_j}, or p_{e_j} / sum_S p
//   dl_i = p_i ([i in S] g_i - sum_S w g), or w_i (g_i - sum_S w g) on S
#include <math.h>

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

template <class F>
__device__ __forceinline__ float wave_all(float v, F op) {       // over all 64 lanes, in all of them
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = op(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_all(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_all(v, [](float a, float b) { return a + b; });
}

template <class T>
__device__ __forceinline__ float to_f32(T v) {
  if constexpr (sizeof(T) == 2) return __builtin_bit_cast(float, (uint32_t)v << 16);
  else return v;
}
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, v); }

template <class T, int kItems>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, float (&v)[kItems]) {
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int e = lane * kItems + i;
    v[i] = e < E ? to_f32(row[e]) : -INFINITY;
  }
}

// The largest logit (0 for a row of -inf, so that the exponentials are 0).
template <int kItems>
__device__ __forceinline__ float row_peak(const float (&v)[kItems]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kItems; ++i) m = __builtin_fmaxf(m, v[i]);
  m = wave_max(m);
  return m == -INFINITY ? 0.0f : m;
}
template <int kItems>
__device__ __forceinline__ float row_total(const float (&v)[kItems], float peak) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kItems; ++i) s += expf(v[i] - peak);
  return wave_sum(s);
}

template <class T, int kItems>
__global__ __launch_bounds__(64 * kWaves) void gate_kernel(GateArgs a) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64; t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
    float v[kItems];
    load_row(static_cast<const T*>(a.logits) + t * a.E, a.E, lane, v);
    const float peak = row_peak(v), total = a.renorm ? 0.0f : row_total(v, peak);
    // What is left to choose from: a NaN ranks as +inf, which peak - peak below
    // turns into NaN weights as the softmax does.
    float left[kItems];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      nan |= v[i] != v[i];
      left[i] = v[i] != v[i] ? INFINITY : v[i];
    }
    nan = __ballot(nan) != 0;
    auto best = [&](int& at) __attribute__((always_inline)) {
      float m = left[0];
      at = 0;
#pragma unroll
      for (int i = 1; i < kItems; ++i) {
        if (left[i] > m) {
          m = left[i];
          at = i;
        }
      }
      return m;
    };
    int at = 0, mine_e = -1;
    float cur = best(at), mine = -INFINITY;                      // lane j: slot j
    for (int j = 0; j < a.k; ++j) {
      const float m = wave_max(cur);
      if (m == -INFINITY) break;
      const int owner = __builtin_ctzll(__ballot(cur == m));
      const int e = __shfl(lane * kItems + at, owner);
      if (lane == j) {
        mine = m;
        mine_e = e;
      }
      if (lane == owner) {
#pragma unroll
        for (int i = 0; i < kItems; ++i)
          if (i == at) left[i] = -INFINITY;
        cur = best(at);
      }
    }
    float w = expf(mine - peak);
    const float den = a.renorm ? wave_sum(mine_e < 0 ? 0.0f : w) : total;
    w = mine_e < 0 ? 0.0f : nan ? NAN : w / den;
    if (lane < a.k) {
      a.weights[t * a.k + lane] = w;
      a.chosen[t * a.k + lane] = mine_e;
    }
  }
}

template <class T, int kItems>
__global__ __launch_bounds__(64 * kWaves) void gate_bwd_kernel(GateArgs a) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / 64; t < a.tokens; t += (int64_t)gridDim.x * kWaves) {
    int e = -1;
    float w = 0.0f, g = 0.0f;
    if (lane < a.k) {
      e = a.chosen_in[t * a.k + lane];
      if ((uint32_t)e >= (uint32_t)a.E) e = -1;
      if (e >= 0) {
        w = a.weights_in[t * a.k + lane];
        g = a.grad_w[t * a.k + lane];
      }
    }
    const float inner = wave_sum(w * g);
    float d[kItems] = {};
    if (!a.renorm) {
      float v[kItems];
      load_row(static_cast<const T*>(a.logits) + t * a.E, a.E, lane, v);
      const float peak = row_peak(v), total = row_total(v, peak);
      const float scale = total == 0.0f ? 0.0f : -inner / total;
#pragma unroll
      for (int i = 0; i < kItems; ++i) d[i] = expf(v[i] - peak) * scale;
    }
    const float own = a.renorm ? w * (g - inner) : w * g;
    for (int j = 0; j < a.k; ++j) {
      const int ej = __builtin_amdgcn_readlane(e, j);
      const float dj = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, own), j));
      if (ej < 0) continue;
#pragma unroll
      for (int i = 0; i < kItems; ++i)
        if (lane * kItems + i == ej) d[i] += dj;
    }
    T* out = static_cast<T*>(a.grad_l) + t * a.E;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      if (lane * kItems + i < a.E) store(out + lane * kItems + i, d[i]);
  }
}

template <class T, int kItems>
void launch(const GateArgs& a, bool bwd, hipStream_t s) {
  const int64_t blocks = (a.tokens + kWaves - 1) / kWaves;
  const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
  if (bwd)
    gate_bwd_kernel<T, kItems><<<grid, dim3(64 * kWaves), 0, s>>>(a);
  else
    gate_kernel<T, kItems><<<grid, dim3(64 * kWaves), 0, s>>>(a);
}

template <class T>
hipError_t dispatch(const GateArgs& a, bool bwd, hipStream_t s) {
  if (a.E <= 64) launch<T, 1>(a, bwd, s);
  else if (a.E <= 128) launch<T, 2>(a, bwd, s);
  else if (a.E <= 256) launch<T, 4>(a, bwd, s);
  else if (a.E <= 512) launch<T, 8>(a, bwd, s);
  else launch<T, 16>(a, bwd, s);
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
