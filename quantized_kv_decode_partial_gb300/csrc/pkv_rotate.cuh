// One head's row on its way to attention: RMS norm over the head dim, weight, rotation of
// pairs of values by the row's position, one rounding to bf16.
//
// Lanes. DPL = 8 values per lane, so a row takes D / 8 lanes (8 at D = 64, 16 at 128, 32 at
// 256, 24 of 32 at 192) and a warp 32 / lanes rows at once. A lane holds both members of its
// pairs, whatever the pairing, so rotating needs no exchange: two runs of four values, at u*4
// and R/2 + u*4 of the rotated part (halves), or at u*8 and u*8 + 4 (adjacent pairs and the
// part that does not turn). Each run is one 8-byte load; a row's runs fill whole sectors.
//
// Angles. position * frequency is reduced in fixed point: a frequency becomes the fraction of
// a turn it makes per position, times 2^64, and the product with the position wraps at whole
// turns by itself. For |frequency| < 2 and any 32-bit position it is off by less than 2^-31
// turns; nothing of it runs in f64, whose rate here is two FMAs per clock and SM.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

template <int D>
struct RowLanes {
  static constexpr int kLanes = D == 64 ? 8 : D == 128 ? 16 : 32;  // lanes a row takes, a power of two
  static constexpr int kUsed = D / 8;                              // of which hold values
  static constexpr int kRows = 32 / kLanes;                        // rows a warp takes at once
};

// 2^64 times the fraction of a turn that an angle of f makes (f mod 2 pi).
__device__ __forceinline__ uint64_t turn_step(float f) {
  constexpr uint64_t kInvTau = 2935890503282001226ull;  // floor(2^64 / (2 pi))
  const uint32_t u = __float_as_uint(f);
  const int e8 = (u >> 23) & 255;
  const uint64_t m = (u & 0x7FFFFFu) | (e8 ? 0x800000u : 0u);  // f = m * 2^(e8 - 150)
  const uint64_t hi = __umul64hi(m << 40, kInvTau);            // m / (2 pi) * 2^40
  const int sh = (e8 ? e8 : 1) - 126;
  const uint64_t c = sh >= 0 ? (sh < 64 ? hi << sh : 0ull) : (sh > -64 ? hi >> -sh : 0ull);
  return (u >> 31) ? 0ull - c : c;
}

__device__ __forceinline__ void turn_at(uint64_t step, int position, float amplitude, float& c, float& s) {
  const uint64_t turns = step * static_cast<uint64_t>(static_cast<int64_t>(position));
  // the upper 32 bits as half turns in [-1, 1)
  sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &s, &c);
  c = __fmul_rn(c, amplitude);
  s = __fmul_rn(s, amplitude);
}

// The axis whose position turns frequency i.
__device__ __forceinline__ int axis_of(const RotationShape& r, int i) {
  if (r.num_axes == 1) return 0;
  if (r.cycle) {
    const int a = i % r.num_axes;
    return i < r.num_axes * r.sections[a] ? a : 0;
  }
  int a = 0, edge = r.sections[0];
  while (a + 1 < r.num_axes && i >= edge) edge += r.sections[++a];
  return a;
}

// Where lane u's two runs of four values begin.
__device__ __forceinline__ void run_offsets(const RotationShape& r, int u, int& off0, int& off1) {
  const bool halves = !r.adjacent && u * 8 < r.rot;
  off0 = halves ? u * 4 : u * 8;
  off1 = halves ? r.rot / 2 + u * 4 : u * 8 + 4;
}

// A norm weight's four values from index i on (plus the offset), f32 or bf16.
__device__ __forceinline__ void load_weight4(const void* w, bool f32, int i, float offset, float* out) {
  if (f32) {
    const float* p = static_cast<const float*>(w) + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = __fadd_rn(p[j], offset);
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w) + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = __fadd_rn(__bfloat162float(p[j]), offset);
  }
}

// Norm and rotation of a lane's eight values (a: the run at off0, b: at off1). Every lane of the
// warp takes part; lanes without values pass zeros. Fused multiply-adds are spelled out, so
// that every kernel that includes this gives the same bits.
//   normed     the row is divided by its root mean square and multiplied by w
//   turned     the lane's values turn; cs, sn: of its four pairs
template <int D>
__device__ __forceinline__ void turn_row(uint2& a, uint2& b, bool any_norm, bool normed, const float (&w)[8], float eps,
                                         bool turned, bool adjacent, const float (&cs)[4], const float (&sn)[4]) {
  float x[8];
  const uint32_t v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
  if (any_norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x[i], x[i], ss);
#pragma unroll
    for (int off = 1; off < RowLanes<D>::kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = __frsqrt_rn(__fmaf_rn(ss, 1.f / D, eps));
    if (normed) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
    }
  }
  auto turn = [&](float& p, float& q, int i) {
    const float x0 = p, x1 = q;
    p = __fmaf_rn(x0, cs[i], -__fmul_rn(x1, sn[i]));
    q = __fmaf_rn(x1, cs[i], __fmul_rn(x0, sn[i]));
  };
  if (turned) {
    if (adjacent) {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], i);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) turn(x[i], x[i + 4], i);
    }
  }
  a = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  b = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// The last b in [0, n) with key(b) <= x, for keys that do not fall; 0 when there is none. Asked
// by a whole warp: 32 probes a round.
template <typename Key>
__device__ __forceinline__ int find_last(int n, long long x, const Key& key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const long long at = lo + static_cast<long long>(lane) * step;
    const bool le = at < hi && (lane == 0 || key(static_cast<int>(at)) <= x);
    const int count = __popc(__ballot_sync(0xffffffffu, le));  // at least lane 0
    lo += (count - 1) * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

}  // namespace pkv
