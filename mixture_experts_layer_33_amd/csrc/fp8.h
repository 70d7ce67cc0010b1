// FP8 with one fp32 scale per block of 128: E4M3 codes, value = code * scale,
// scale = max(amax, 2^-100) / 448 (the largest magnitude of a block becomes E4M3's largest
// value, 448; the floor keeps the scale of a block of zeros a normal number).  Included by
// common.h users that quantise (norm, dispatch, quantiser, the gate/up epilogue).
#pragma once

#include "common.h"

namespace moe {

constexpr float FP8_MAX = 448.0f;

// Largest magnitude of the 8 values of each of G consecutive lanes.  Taken on the bit
// patterns, where a NaN is above every number, so that it is not lost as in fmaxf: the
// result is then a NaN (or an infinity), not less than INFINITY.
template <int G>
__device__ __forceinline__ float lanes_amax(float a) {
  static_assert(G >= 2 && G <= 64 && (G & (G - 1)) == 0, "groups of 2 .. 64 lanes");
  int v = __float_as_int(a) & 0x7fffffff;
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, false));
  if constexpr (G >= 4) v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, false));
  if constexpr (G >= 8) v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, false));
  if constexpr (G >= 16) v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, false));
  if constexpr (G >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((int)s[0], (int)s[1]);
  }
  if constexpr (G >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((int)s[0], (int)s[1]);
  }
  return __int_as_float(v);
}
__device__ __forceinline__ float amax2(float a, float b) {
  return __int_as_float(max(__float_as_int(a) & 0x7fffffff, __float_as_int(b) & 0x7fffffff));
}
template <int G>
__device__ __forceinline__ float block_amax(const float (&v)[8]) {
  float a = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) a = amax2(a, v[q]);
  return lanes_amax<G>(a);
}

// NaN for a block that holds a NaN or an infinity.
__device__ __forceinline__ float fp8_scale(float amax) {
  return amax < INFINITY ? fmaxf(amax, 0x1p-100f) / FP8_MAX : NAN;
}

// E4M3 of v / scale, v over the scale being divided as written (IEEE), clamped against the last
// bit of the quotient of the block's largest value.
__device__ __forceinline__ uint32_t fp8_encode4(float a, float b, float c, float d, float s) {
  auto q = [s](float v) { return __builtin_amdgcn_fmed3f(v / s, -FP8_MAX, FP8_MAX); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q(a), q(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q(c), q(d), lo, true);
}
__device__ __forceinline__ u32x2 fp8_encode8(const float (&v)[8], float s) {
  return u32x2{fp8_encode4(v[0], v[1], v[2], v[3], s), fp8_encode4(v[4], v[5], v[6], v[7], s)};
}

// H's codes: the same quotient, from the scale's rounded reciprocal r and one correction by the exact remainder of v r
// (Markstein's theorem: the result is the rounded v / s).  As plain divisions, some ten instructions each, a
// gate/up tile's epilogue took 6 % of a call (4,096 rows over 16 experts, d 1024, f 2048: 150 -> 159 us; so 145), and v r
// alone takes values that lie within a last bit of a rounding border to its other side.
__device__ __forceinline__ uint32_t h_encode4(float a, float b, float c, float d, float s) {
  const float r = 1.0f / s;
  auto quotient = [r, s](float v) {
    const float q = v * r;
    return fmaf(fmaf(-q, s, v), r, q);
  };
  auto q = [&](float v) { return __builtin_amdgcn_fmed3f(quotient(v), -FP8_MAX, FP8_MAX); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q(a), q(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q(c), q(d), lo, true);
}

}  // namespace moe
