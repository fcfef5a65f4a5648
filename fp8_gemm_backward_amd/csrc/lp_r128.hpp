// Quantization to E4M3 with an fp32 scale per 128 elements: the arithmetic
// shared by the quantizers, the products that quantize their own input and
// the optimizer's 8-bit moments.
//
// For a set of values with largest magnitude a:
//   s = fp32(max(a, 2^-64) / 448),   code = E4M3(fp32(v / s)),
// nearest even and saturating.  The floor keeps s and 1 / s normal numbers
// (an all-zero set needs no case of its own); sets that small are far below
// what a bf16 training step resolves.  A NaN or an infinity makes s a NaN and
// every code of the set 0x7F with its element's sign, so that it cannot be
// mistaken for a finite result later.
#pragma once

#include "lp_mxq.hpp"

namespace lp {

constexpr float kE4M3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-64f;

struct RunScale {
  float s;       // decode multiplier (NaN for a bad set)
  float r;       // 1 / s, correctly rounded
  bool bad;
};

// Both quotients by one exact residual each instead of the general division,
// whose scaling for subnormal numbers these cannot need; equal to the divided
// a / 448 and 1 / s for every significand (all 2^23 compared at four
// exponents, the lowest and highest among them).  Quantizing along both axes
// took 16 of these a thread: 8192 x 4096 in 28.4 us, 30.2 with divisions.
// amax: magnitude bits of the largest |v| as fp32 (bits >= 0x7F800000: NaN
// or infinity, which the integer maximum keeps).
__device__ __forceinline__ RunScale run_scale(uint32_t amax) {
  RunScale q;
  q.bad = amax >= 0x7F800000u;
  const float a = q.bad ? 1.0f : __builtin_fmaxf(__builtin_bit_cast(float, amax), kAmaxFloor);
  const float t = a * (1.0f / kE4M3Max);
  const float s = __builtin_fmaf(__builtin_fmaf(-t, kE4M3Max, a), 1.0f / kE4M3Max, t);
  const float r = __builtin_amdgcn_rcpf(s);
  q.r = __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
  q.s = q.bad ? __builtin_bit_cast(float, 0x7FC00000u) : s;
  return q;
}

// fp32(v / s), correctly rounded: the quotient by the rounded reciprocal is
// within one unit in the last place, and one exact residual corrects it
// (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  s >= 2^-73 keeps the residual of every
// quotient that does not round to code 0 out of the subnormal range.  The
// residual is taken as t s - v: an exact zero then leaves a negative zero's
// sign alone.
__device__ __forceinline__ float run_div(float v, const RunScale& q) {
  const float t = v * q.r;
  return __builtin_fmaf(-__builtin_fmaf(t, q.s, -v), q.r, t);
}

// Four values -> four codes (first in the low byte).
__device__ __forceinline__ uint32_t run_codes4(float a, float b, float c, float d, const RunScale& q) {
  return to_e4m3x2(run_div(a, q), run_div(b, q)) | (to_e4m3x2(run_div(c, q), run_div(d, q)) << 16);
}

// Maximum over the 16 lanes of a lane row.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));   // row_ror:8
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));   // row_ror:4
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));   // row_ror:2
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));   // row_ror:1
  return v;
}

// Largest magnitude of the eight bf16 of a 16-byte piece, as fp32 bits.
__device__ __forceinline__ uint32_t amax8(u32x4 v) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = pk_umax16(m, v[k] & 0x7FFF7FFFu);
  return umax(m & 0xFFFFu, m >> 16) << 16;
}

// Codes of the eight bf16 of a piece under one scale.
__device__ __forceinline__ u32x2 run_codes8(u32x4 v, const RunScale& q) {
  if (q.bad) return u32x2{nan_e4m3x2(v[0]) | (nan_e4m3x2(v[1]) << 16), nan_e4m3x2(v[2]) | (nan_e4m3x2(v[3]) << 16)};
  return u32x2{run_codes4(bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1]), q),
               run_codes4(bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3]), q)};
}

}  // namespace lp
