// One head's row on its way to attention: RMS norm over the head dim, weight, rotation of
// pairs of values by the row's position, one rounding to bf16.
//
// Lanes. A unit is eight values of a row, D / 8 of them in all, which hold both members of their pairs, whatever the
// pairing, so that rotating needs no exchange: two runs of four values, at u*4 and R/2 + u*4 of the rotated part
// (halves), or at u*8 and u*8 + 4 (adjacent pairs and the part that does not turn). Each run is one 8-byte access; a row's
// runs fill whole sectors. A lane has one unit of its row, or two, kHalf apart.
//
// Angles. position * frequency is reduced in fixed point: a frequency becomes the fraction of
// a turn it makes per position, times 2^64, and the product with the position wraps at whole
// turns by itself. For |frequency| < 2 and any 32-bit position it is off by less than 2^-31
// turns; nothing of it runs in f64, whose rate here is two FMAs per clock and SM.
#pragma once

#include "pkv_codes.cuh"
#include "pkv_common.cuh"

namespace pkv {

template <int D>
struct RowLanes {
  static constexpr int kLanes = D == 64 ? 8 : D == 128 ? 16 : 32;  // lanes a row takes, a power of two
  static constexpr int kUsed = D / 8;                              // of which hold values
  static constexpr int kRows = 32 / kLanes;                        // rows a warp takes at once
  static constexpr int kHalf = kLanes / 2, kRows2 = 2 * kRows;     // with two units per lane
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

// cos and sin (times amplitude) of `position` steps. The angle is brought to the nearest quarter turn, f of a turn away
// (|f| <= 1/8): there their Taylor series in f^2 are off by less than 2^-28.
__device__ __forceinline__ void turn_at(uint64_t step, int position, float amplitude, float& c, float& s) {
  const uint64_t turns = step * static_cast<uint64_t>(static_cast<int64_t>(position));
  const uint32_t u = static_cast<uint32_t>(turns >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const float f = static_cast<float>(static_cast<int32_t>(u - (quarter << 30))) * 0x1p-32f;
  const float z = __fmul_rn(f, f);
  // (2 pi)^n / n!
  float sn = __fmaf_rn(__fmaf_rn(__fmaf_rn(__fmaf_rn(42.0586939f, z, -76.7058597f), z, 81.6052492f), z, -41.3417022f), z,
                       6.28318531f);
  sn = __fmul_rn(sn, f);
  float cn = __fmaf_rn(__fmaf_rn(-26.4262567f, z, 60.2446413f), z, -85.4568172f);
  cn = __fmaf_rn(__fmaf_rn(__fmaf_rn(cn, z, 64.9393940f), z, -19.7392088f), z, 1.f);
  const bool odd = quarter & 1;
  const float x = odd ? sn : cn, y = odd ? cn : sn;
  c = __fmul_rn(__uint_as_float(__float_as_uint(x) ^ ((quarter + 1 & 2) << 30)), amplitude);
  s = __fmul_rn(__uint_as_float(__float_as_uint(y) ^ ((quarter & 2) << 30)), amplitude);
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

// What does not change from token to token, in shared memory: each frequency's step and axis, and the norm weights
// (plus their offset; ones where there is no norm).
template <int D>
struct __align__(16) RotateTables {
  uint64_t step[D / 2];
  float weight[2][D];  // queries', keys'
  uint8_t axis[D / 2];
};

// Filled by the whole block of at least 128 threads, which then synchronises: the words are asked for first and
// used when something else has had its time.
template <int D>
struct TablesAhead {
  static constexpr int kWeights = 2 * D / 128;  // of a thread, at most
  float freq, weight[kWeights];
  __device__ __forceinline__ void load(const RotateParams& p) {
    const int t = threadIdx.x;
    freq = t < p.turn.rot / 2 ? p.inv_freq[t] : 0.f;
#pragma unroll
    for (int k = 0; k < kWeights; ++k) {
      const int i = t + k * blockDim.x;
      const void* w = i < D ? p.q_weight : p.k_weight;
      const int d = i < D ? i : i - D;
      weight[k] = 0.f;
      if (i < 2 * D && w)
        weight[k] = p.weight_f32 ? static_cast<const float*>(w)[d] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[d]);
    }
  }
  __device__ __forceinline__ void store(RotateTables<D>& tab, const RotateParams& p) const {
    const int t = threadIdx.x;
    if (t < p.turn.rot / 2) {
      tab.step[t] = turn_step(freq);
      tab.axis[t] = static_cast<uint8_t>(axis_of(p.turn, t));
    }
#pragma unroll
    for (int k = 0; k < kWeights; ++k) {
      const int i = t + k * blockDim.x;
      if (i < 2 * D) (&tab.weight[0][0])[i] = (i < D ? p.q_weight : p.k_weight) ? __fadd_rn(weight[k], p.weight_offset) : 1.f;
    }
  }
};

// What a lane's eight values are multiplied by: value v of a pair becomes r * (v * own + partner * other), r
// the row's norm. own and other hold the norm weight times cos and sin, so a token's heads share them.
struct LaneTurn {
  uint64_t own[4], other[4];  // of the values (0, 1), (2, 3) of the first run, then of the second
};

// w: the eight weights (ones without a norm); cs, sn: of the lane's four pairs. Products are spelled out here and below,
// so that every kernel that includes this gives the same bits. SIMPLE: whole heads turn, in halves (then `turned` and
// `adjacent` are not looked at): the usual form, without the branches of the others.
template <bool SIMPLE>
__device__ __forceinline__ LaneTurn make_turn(const float (&w)[8], const float (&cs)[4], const float (&sn)[4], bool turned,
                                              bool adjacent) {
  LaneTurn t;
  if (SIMPLE) adjacent = false;
  if (!SIMPLE && !turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.own[i] = pair(w[2 * i], w[2 * i + 1]);
      t.other[i] = 0ull;
    }
    return t;
  }
  float p[8], q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // pair i: the values a and b
    const float wa = adjacent ? w[2 * i] : w[i], wb = adjacent ? w[2 * i + 1] : w[4 + i];
    const float pa = __fmul_rn(wa, cs[i]), pb = __fmul_rn(wb, cs[i]), qa = -__fmul_rn(wb, sn[i]), qb = __fmul_rn(wa, sn[i]);
    if (adjacent) {
      p[2 * i] = pa;
      p[2 * i + 1] = pb;
      q[2 * i] = qa;
      q[2 * i + 1] = qb;
    } else {
      p[i] = pa;
      p[4 + i] = pb;
      q[i] = qa;
      q[4 + i] = qb;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.own[i] = pair(p[2 * i], p[2 * i + 1]);
    t.other[i] = pair(q[2 * i], q[2 * i + 1]);
  }
  return t;
}

// Eight values of a row: a is the run at off0, b the run at off1.
struct Unit {
  uint64_t x[4];  // as f32 pairs
  __device__ __forceinline__ Unit(const uint2& a, const uint2& b) {
    const uint32_t v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ float squares() const {
    uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s2 = fma2(x[i], x[i], s2);
    float s0, s1;
    unpair(s2, s0, s1);
    return __fadd_rn(s0, s1);
  }
  // Rotation and weights, times r where there is a norm; back to bf16.
  template <bool SIMPLE>
  __device__ __forceinline__ void turn(bool normed, float r, bool turned, bool adjacent, const LaneTurn& t, uint2& a,
                                       uint2& b) const {
    uint64_t y[4];
    if (!SIMPLE && !turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mul2(x[i], t.own[i]);
    } else if (!SIMPLE && adjacent) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpair(x[i], lo, hi);
        y[i] = fma2(x[i], t.own[i], mul2(pair(hi, lo), t.other[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fma2(x[i], t.own[i], mul2(x[i ^ 2], t.other[i]));
    }
    if (normed) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mul2(y[i], pair(r, r));
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpair(y[i], lo, hi);
      w[i] = pack_bf16x2(lo, hi);
    }
    a = make_uint2(w[0], w[1]);
    b = make_uint2(w[2], w[3]);
  }
};

__device__ __forceinline__ float inverse_rms(float squares, int dim, float eps) {
  return rsqrtf(__fmaf_rn(squares, 1.f / dim, eps));
}

// Norm and rotation of a row that has one unit in each of RowLanes<D>::kLanes lanes. Every lane of the warp takes
// part; lanes without values pass zeros.
template <int D, bool SIMPLE>
__device__ __forceinline__ void turn_row(uint2& a, uint2& b, bool normed, float eps, bool turned, bool adjacent,
                                         const LaneTurn& t) {
  const Unit v(a, b);
  float r = 1.f;
  if (normed) {
    float ss = v.squares();
#pragma unroll
    for (int off = 1; off < RowLanes<D>::kLanes; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    r = inverse_rms(ss, D, eps);
  }
  v.turn<SIMPLE>(normed, r, turned, adjacent, t, a, b);
}

// The same with two units per lane, u and u + kHalf, for half as many lanes and as much of everything that is done once
// per row and lane. The squares are added up in the same order.
template <int D, bool SIMPLE>
__device__ __forceinline__ void turn_row2(uint2 (&a)[2], uint2 (&b)[2], bool normed, float eps, const bool (&turned)[2],
                                          bool adjacent, const LaneTurn (&t)[2]) {
  const Unit v0(a[0], b[0]), v1(a[1], b[1]);
  float r = 1.f;
  if (normed) {
    float s0 = v0.squares(), s1 = v1.squares();
#pragma unroll
    for (int off = 1; off < RowLanes<D>::kLanes / 2; off <<= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, off);
      s1 += __shfl_xor_sync(0xffffffffu, s1, off);
    }
    r = inverse_rms(s0 + s1, D, eps);
  }
  v0.turn<SIMPLE>(normed, r, turned[0], adjacent, t[0], a[0], b[0]);
  v1.turn<SIMPLE>(normed, r, turned[1], adjacent, t[1], a[1], b[1]);
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

// Packed tokens' starts, looked through by one warp: flags those that fall or leave [0, tokens].
__device__ __forceinline__ void check_starts(const int32_t* starts, int num_seqs, int tokens, int32_t* error_flag) {
  bool bad = false;
  for (int i = threadIdx.x & 31; i <= num_seqs; i += 32) {
    const int s = starts[i];
    bad = bad || s < 0 || s > tokens || (i > 0 && s < starts[i - 1]);
  }
  if (bad && error_flag) atomicOr(error_flag, kDevErrBadSeqLen);
}

}  // namespace pkv
