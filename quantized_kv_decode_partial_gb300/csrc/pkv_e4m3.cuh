// Codes of e4m3 pages with one power-of-two scale per (block, KV head): the scale that a
// block's values need, values to codes, codes under a grown scale. Used by both appends
// into such pages, so that they write the same bits.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

// Elementwise maximum of the magnitudes of bf16 pairs (the values are finite).
__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t w) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&m), __habs2(*reinterpret_cast<__nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_abs(uint32_t m, const uint4& v) {
  return max_abs(max_abs(max_abs(max_abs(m, v.x), v.y), v.z), v.w);
}

// The smallest power of two s (at least 2^-126) with a <= 448 s, for a > 0; 0 for a = 0.
__device__ __forceinline__ float pow2_scale(float a) {
  const uint32_t u = __float_as_uint(a);
  if (u == 0u) return 0.f;
  // 448 = 1.75 * 2^8: the exponent of a less 8, one more when a's significand exceeds 1.75
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Codes of 8 bf16 values over s (s > 0): times its exact reciprocal when s is a power of
// two (EXACT, as the append makes it), else by division (a scale the caller chose).
template <bool EXACT>
__device__ __forceinline__ uint2 quantize8(const uint4& v, float s, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
    c[i] = EXACT ? e4m3x2(lo * inv, hi * inv) : e4m3x2(__fdiv_rn(lo, s), __fdiv_rn(hi, s));
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// The four codes of a word times `ratio`, as codes.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return e4m3x2(a.x * ratio, a.y * ratio) | (e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

}  // namespace pkv
