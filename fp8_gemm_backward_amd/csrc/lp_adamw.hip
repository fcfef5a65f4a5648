// One AdamW step over many tensors (HBM-bound), moments in fp32 or in E4M3
// with an fp32 scale per run of 128 elements.
//
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g            v = b2 v + (1 - b2) g^2
//   p = (1 - lr wd) p - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Every operation is an fp32 operation of its own, in this order, with no
// multiply-add contraction, so that the result does not depend on how the
// compiler fuses them.  The factors that depend on the step and the tensor only
// are computed in double, then rounded to fp32.  The moments and masters stay
// fp32 inside; 8-bit moments and bf16 copies are rounded once, at the end.
//
// 8-bit moments: m, and sqrt(v) in place of v (its range in powers of two is
// half of v's), are quantized per run of 128 by the rule of lp_r128.hpp;
// a positive sqrt(v) is never stored as 0 (at least code 1), or the next step
// would divide by eps alone.
//
// A table in device memory, made once (lp_adamw_plan), lists the tensors and
// the tensor of each chunk of kChunk elements, so that a step is one launch
// whatever the number of tensors, with one lookup per workgroup.  A lane holds
// four consecutive elements (16 bytes of fp32, so every access of a wave is
// one contiguous KiB), kUnits times, with all loads issued first; 32 lanes
// hold a run.  96 small tensors (1.6 M elements) 10.5 us; with the tensors in the
// kernel arguments, two launches and a search per workgroup, 18.7.  67 M
// parameters with bf16 gradients and copies: 354 us with fp32 moments (1.88 GB,
// 5.3 TB/s), 206 us with 8-bit ones (1.08 GB, 5.3 TB/s): the rate of memory.
#include "lp_internal.hpp"
#include "lp_r128.hpp"

#pragma clang fp contract(off)

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;
constexpr int kChunk = kThreads * 4 * kUnits;

struct Entry {
  void* p;
  const void* g;
  void *m, *v;
  float *ms, *vs;
  uint16_t* copy;
  int64_t n;
  float lr_scale, weight_decay;
  uint32_t first;        // the tensor's first chunk
  int32_t vec;           // every pointer is aligned for four-element accesses
};

struct Args {
  const Entry* e;
  const uint32_t* tensor;                // of each chunk
  float b1, c1, b2, c2, inv_bc2, eps;    // c = 1 - b; inv_bc2 = 1 / sqrt(1 - b2^t)
  double lr, bc1;                        // bc1 = 1 - b1^t
  const float* grad_scale;
};

__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

// Elements i .. i + 3 of a tensor of n, as fp32; those past the end are 0.
template <bool kBf16>
__device__ __forceinline__ f32x4 load4(const void* base, int64_t i, int64_t n, bool vec) {
  f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (kBf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if (vec && i + 4 <= n) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(p);
      r = f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (i + d < n) r[d] = bf16_lo(p[d]);
    }
  } else {
    const float* p = static_cast<const float*>(base) + i;
    if (vec && i + 4 <= n) {
      r = *reinterpret_cast<const f32x4*>(p);
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (i + d < n) r[d] = p[d];
    }
  }
  return r;
}

template <bool kBf16>
__device__ __forceinline__ void store4(void* base, int64_t i, int64_t n, bool vec, f32x4 v) {
  if constexpr (kBf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + i;
    if (vec && i + 4 <= n) {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (i + d < n) p[d] = bf16_bits(v[d]);
    }
  } else {
    float* p = static_cast<float*>(base) + i;
    if (vec && i + 4 <= n) {
      *reinterpret_cast<f32x4*>(p) = v;
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d)
        if (i + d < n) p[d] = v[d];
    }
  }
}

__device__ __forceinline__ uint32_t load4_codes(const void* base, int64_t i, int64_t n, bool vec) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  if (vec && i + 4 <= n) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int d = 0; d < 4; ++d)
    if (i + d < n) w |= (uint32_t)p[d] << (8 * d);
  return w;
}

__device__ __forceinline__ void store4_codes(void* base, int64_t i, int64_t n, bool vec, uint32_t w) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  if (vec && i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(p) = w;
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (i + d < n) p[d] = (uint8_t)(w >> (8 * d));
  }
}

// (A bit cast of a vector's element itself would take the vector's first.)
__device__ __forceinline__ uint32_t f32_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

__device__ __forceinline__ f32x4 decode4(uint32_t w, float s) {
  const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, false);
  const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, 1.0f, true);
  return f32x4{lo[0] * s, lo[1] * s, hi[0] * s, hi[1] * s};
}

// The scale of the run that the 32 lanes of this half wave hold.
__device__ __forceinline__ RunScale half_wave_scale(f32x4 x) {
  uint32_t m = 0;
#pragma unroll
  for (int d = 0; d < 4; ++d) m = umax(m, f32_bits(x[d]) & 0x7FFFFFFFu);
  m = row16_max(m);
  m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
  return run_scale(m);
}

// Codes of four values; kKeep: a positive value is at least code 1 (2^-9).
template <bool kKeep>
__device__ __forceinline__ uint32_t quant4(f32x4 x, const RunScale& q) {
  f32x4 t;
  uint32_t nan = 0;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    t[d] = run_div(x[d], q);
    if (kKeep && x[d] > 0.0f && t[d] < 0x1p-9f) t[d] = 0x1p-9f;
    nan |= (0x7Fu | ((f32_bits(x[d]) >> 24) & 0x80u)) << (8 * d);
  }
  return q.bad ? nan : to_e4m3x2(t[0], t[1]) | (to_e4m3x2(t[2], t[3]) << 16);
}

template <bool kBf16P, bool kBf16G, bool k8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Args a) {
  const Entry e = a.e[__builtin_amdgcn_readfirstlane((int)a.tensor[blockIdx.x])];
  const double lr = a.lr * (double)e.lr_scale;
  const float decay = (float)(1.0 - lr * (double)e.weight_decay), step = (float)(lr / a.bc1);
  const int64_t n = e.n, i0 = (int64_t)(blockIdx.x - e.first) * kChunk + 4 * threadIdx.x;
  const bool vec = e.vec != 0;
  f32x4 p[kUnits], g[kUnits], m[kUnits], v[kUnits];
  uint32_t mc[kUnits], vc[kUnits];
  float ms[kUnits], vs[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t i = i0 + u * kThreads * 4;
    p[u] = load4<kBf16P>(e.p, i, n, vec);
    g[u] = load4<kBf16G>(e.g, i, n, vec);
    if constexpr (k8) {
      mc[u] = load4_codes(e.m, i, n, vec);
      vc[u] = load4_codes(e.v, i, n, vec);
      ms[u] = i < n ? e.ms[i >> 7] : 0.0f;
      vs[u] = i < n ? e.vs[i >> 7] : 0.0f;
    } else {
      m[u] = load4<false>(e.m, i, n, vec);
      v[u] = load4<false>(e.v, i, n, vec);
    }
  }
  const float gs = a.grad_scale != nullptr ? *a.grad_scale : 1.0f;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int64_t i = i0 + u * kThreads * 4;
    if constexpr (k8) {
      m[u] = decode4(mc[u], ms[u]);
      v[u] = decode4(vc[u], vs[u]);
#pragma unroll
      for (int d = 0; d < 4; ++d) v[u][d] = v[u][d] * v[u][d];
    }
    f32x4 r;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const float gg = g[u][d] * gs;
      const float mm = m[u][d] * a.b1 + gg * a.c1;
      const float vv = v[u][d] * a.b2 + (gg * gg) * a.c2;
      r[d] = __builtin_sqrtf(vv);
      m[u][d] = mm;
      v[u][d] = vv;
      p[u][d] = p[u][d] * decay - mm / (r[d] * a.inv_bc2 + a.eps) * step;
    }
    store4<kBf16P>(e.p, i, n, vec, p[u]);
    if (!kBf16P && e.copy != nullptr) store4<true>(e.copy, i, n, vec, p[u]);
    if constexpr (k8) {
      const RunScale qm = half_wave_scale(m[u]), qr = half_wave_scale(r);
      if ((threadIdx.x & 31) == 0 && i < n) {
        e.ms[i >> 7] = qm.s;
        e.vs[i >> 7] = qr.s;
      }
      store4_codes(e.m, i, n, vec, quant4<false>(m[u], qm));
      store4_codes(e.v, i, n, vec, quant4<true>(r, qr));
    } else {
      store4<false>(e.m, i, n, vec, m[u]);
      store4<false>(e.v, i, n, vec, v[u]);
    }
  }
}

template <bool kBf16P, bool kBf16G>
void launch(const Args& a, uint32_t chunks, bool bits8, hipStream_t s) {
  if (bits8)
    adamw_kernel<kBf16P, kBf16G, true><<<dim3(chunks), dim3(kThreads), 0, s>>>(a);
  else
    adamw_kernel<kBf16P, kBf16G, false><<<dim3(chunks), dim3(kThreads), 0, s>>>(a);
}

bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }
size_t map_offset(int64_t count) { return (size_t)count * sizeof(Entry); }

}  // namespace

int64_t adamw_chunks(const lp_adamw_tensor* tensors, int64_t count) {
  int64_t chunks = 0;
  for (int64_t k = 0; k < count; ++k) chunks += chunks_of(tensors[k].n);
  return chunks;
}

size_t adamw_table_bytes(int64_t count, int64_t chunks) { return map_offset(count) + (size_t)chunks * 4; }

void adamw_fill(const lp_adamw_tensor* tensors, int64_t count, bool bf16_param, bool bf16_grad, bool bits8, void* table) {
  Entry* const entries = static_cast<Entry*>(table);
  uint32_t* map = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(table) + map_offset(count));
  uint32_t first = 0;
  for (int64_t k = 0; k < count; ++k) {
    const lp_adamw_tensor& t = tensors[k];
    const uintptr_t state = bits8 ? 4 : 16;
    const bool vec = is_aligned(t.param, bf16_param ? 8 : 16) && is_aligned(t.grad, bf16_grad ? 8 : 16) &&
                     is_aligned(t.exp_avg, state) && is_aligned(t.exp_avg_sq, state) && is_aligned(t.param_copy, 8);
    entries[k] = Entry{t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.exp_avg_scales, t.exp_avg_sq_scales,
                       static_cast<uint16_t*>(t.param_copy), t.n, t.lr_scale, t.weight_decay, first, vec};
    for (int64_t c = chunks_of(t.n); c > 0; --c, ++first) *map++ = (uint32_t)k;
  }
}

hipError_t launch_adamw(const AdamwCall& c, hipStream_t stream) {
  const uint8_t* const table = static_cast<const uint8_t*>(c.table);
  const Args a{reinterpret_cast<const Entry*>(table),
               reinterpret_cast<const uint32_t*>(table + map_offset(c.count)),
               (float)c.beta1,
               (float)(1.0 - c.beta1),
               (float)c.beta2,
               (float)(1.0 - c.beta2),
               (float)(1.0 / __builtin_sqrt(1.0 - __builtin_pow(c.beta2, (double)c.step))),
               (float)c.eps,
               c.lr,
               1.0 - __builtin_pow(c.beta1, (double)c.step),
               c.grad_scale};
  const uint32_t chunks = (uint32_t)c.chunks;
  if (c.bf16_param)
    c.bf16_grad ? launch<true, true>(a, chunks, c.bits8, stream) : launch<true, false>(a, chunks, c.bits8, stream);
  else
    c.bf16_grad ? launch<false, true>(a, chunks, c.bits8, stream) : launch<false, false>(a, chunks, c.bits8, stream);
  return hipGetLastError();
}

}  // namespace lp
