// Codes of quantised pages to 16-bit values, sixteen at a time, and packed f32 arithmetic.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

// Pairs of f32 values in one register pair: packed arithmetic, each lane of it rounded as the scalar one.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Sixteen codes of a row as pairs of 16-bit values: e4m3 times their scale, in bf16; affine scale * code + bias, in
// fp16. In f32, rounded once.
template <int FMT>
__device__ __forceinline__ void codes_to_values(const uint4& v, float scale, float bias, uint32_t (&out)[8]) {
  if constexpr (FMT == kFmtE4m3) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2(w[i], lo, hi);
      float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      unpair(mul2(pair(a.x, a.y), pair(scale, scale)), a.x, a.y);
      unpair(mul2(pair(b.x, b.y), pair(scale, scale)), b.x, b.y);
      out[2 * i] = pack_bf16x2(a.x, a.y);
      out[2 * i + 1] = pack_bf16x2(b.x, b.y);
    }
  } else {
    // codes as halves: 1024 + code has the code in its last bits
    const __half2 k1024 = __floats2half2_rn(1024.f, 1024.f);
    auto floats = [&](uint32_t bits) {
      return __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&bits), k1024));
    };
    if constexpr (FMT == 8) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = floats(__byte_perm(w[i], 0x64646464u, 0x4140)), b = floats(__byte_perm(w[i], 0x64646464u, 0x4342));
        out[2 * i] = pack_f16x2(fmaf(a.x, scale, bias), fmaf(a.y, scale, bias));
        out[2 * i + 1] = pack_f16x2(fmaf(b.x, scale, bias), fmaf(b.y, scale, bias));
      }
    } else {
      const uint32_t w[2] = {v.x, v.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float2 n[4];  // codes k and k + 4
#pragma unroll
        for (int k = 0; k < 4; ++k) n[k] = floats((w[i] >> (4 * k) & 0x000F000Fu) | 0x64006400u);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          out[4 * i + k] = pack_f16x2(fmaf(n[2 * k].x, scale, bias), fmaf(n[2 * k + 1].x, scale, bias));
          out[4 * i + 2 + k] = pack_f16x2(fmaf(n[2 * k].y, scale, bias), fmaf(n[2 * k + 1].y, scale, bias));
        }
      }
    }
  }
}

}  // namespace pkv
