// Sparse decode attention over a paged cache: which blocks of each (sequence, KV head) a
// step reads.
//
// Each (block, KV head) carries the bounds of its stored keys, k_bounds [NB, HK, 2, D]: the
// elementwise smallest (row 0) and largest (row 1) value, rounded outward to bf16. For a
// query row q no key of block j scores above
//     u_j(q) = sum_d max(q_d lo_jd, q_d hi_jd) = <max(q, 0), hi_j> + <min(q, 0), lo_j>
// and the block's score for a KV head is the largest u_j over its query rows. The step then
// attends over `first` blocks at the start, `last` at the end and the best-scored others,
// top_k in all, through the decode kernels: the pool seen as NB * HK blocks of one head, and
// every (sequence, KV head) as a sequence of its chosen blocks in order.
//
// The bounds' upkeep after an append is one kernel. Scores and choice are two, or one where
// a cluster per (sequence, KV head) scores every block in one step and the GPU holds all
// clusters at once.
#include <algorithm>
#include <atomic>

#include "pkv_launch.h"

namespace pkv {

namespace {

// ------------------------------------------------------------------------------ bounds' upkeep
// One warp per (sequence, touched block, KV head). A lane holds the same 16 bytes of every
// kRowsPerPass-th row, so each pass is one coalesced 16-byte load per lane, and keeps the
// running bounds of its dims in registers. Bound by HBM for bf16 and e4m3 pages (packed
// min/max, 2 values per instruction; 8 x 32768 bf16 rows, 8 KV heads, D=128: 86.2 us, 0.98 of a
// copy's rate); affine codes cost an FMA, a minimum and a maximum per
// value, which 4-bit pages are bound by.
template <int FMT, int D>
struct BoundsCfg {
  static constexpr int kBits = FMT == kFmtE4m3 ? 8 : FMT;
  static constexpr int kRowBytes = D * kBits / 8;
  static constexpr int kLanes = kRowBytes / 16;        // lanes per row
  static constexpr int kRowsPerPass = 32 / kLanes;     // rows per warp-wide load
  static constexpr int kVals = 128 / kBits;            // values per lane
  static constexpr bool kAffine = FMT == 4 || FMT == 8;
  static constexpr int kUnroll = kAffine ? 4 : 8;      // loads in flight per lane
};

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t w) {  // m, |w|
  const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&m), __habs2(*reinterpret_cast<__nv_bfloat162*>(&w)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// max(a, 0) and min(a, 0), NaN for NaN
__device__ __forceinline__ uint32_t positive_bf16x2(uint32_t a) {
  const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), __float2bfloat162_rn(0.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t negative_bf16x2(uint32_t a) {
  const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), __float2bfloat162_rn(0.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t min_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int FMT, int D>
__global__ void __launch_bounds__(128) pkv_bounds_kernel(const __grid_constant__ BoundsParams p) {
  using C = BoundsCfg<FMT, D>;
  wait_for_prerequisite_grids();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const int unit = blockIdx.x * 4 + warp;
  if (unit >= p.blocks * p.num_kv_heads) return;
  const int t = unit / p.num_kv_heads, h = unit - t * p.num_kv_heads;
  const int len = p.seq_lens[b];
  if (len < 0 || static_cast<long long>(len) > static_cast<long long>(p.max_blocks) * p.block_size) {
    if (lane == 0 && unit == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadSeqLen);
    return;
  }
  const int begin = len > p.n_new ? len - p.n_new : 0;
  const int blk = begin / p.block_size + t;
  const long long row0 = static_cast<long long>(blk) * p.block_size;
  if (row0 >= len) return;
  const int phys = p.block_tables[static_cast<size_t>(b) * p.max_blocks + blk];
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
    if (lane == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
    return;
  }
  // rows [r0, r1) of the block are new; earlier ones are in the stored bounds already, but
  // for e4m3 pages, whose scale may have grown with the new rows: those are taken whole
  const int r1 = static_cast<int>(min(len - row0, static_cast<long long>(p.block_size)));
  const bool held = row0 < begin && FMT != kFmtE4m3;
  const int r0 = held ? static_cast<int>(begin - row0) : 0;
  const size_t cell = static_cast<size_t>(phys) * p.num_kv_heads + h;
  const int sub = lane / C::kLanes, col = lane % C::kLanes;  // row within a pass, 16-byte column
  const bool on = sub < C::kRowsPerPass;
  const char* base = static_cast<const char*>(p.k_pool) + (cell * p.block_size) * C::kRowBytes + col * 16;

  // this lane's dims: [col * kVals, col * kVals + kVals)
  constexpr int kWords = C::kAffine ? C::kVals : C::kVals / 2;  // f32 values, or 16-bit pairs
  uint32_t lo[kWords], hi[kWords];
  constexpr uint32_t kInf = C::kAffine ? 0x7F800000u : FMT == 16 ? 0x7F807F80u : 0x7C007C00u;
  constexpr uint32_t kNegInf = C::kAffine ? 0xFF800000u : FMT == 16 ? 0xFF80FF80u : 0xFC00FC00u;
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    lo[i] = kInf;
    hi[i] = kNegInf;
  }
  for (int r = r0; r < r1; r += C::kRowsPerPass * C::kUnroll) {
    uint4 v[C::kUnroll];
    float sc[C::kUnroll], bi[C::kUnroll];
#pragma unroll
    for (int u = 0; u < C::kUnroll; ++u) {
      const int row = r + u * C::kRowsPerPass + sub;
      const bool in = on && row < r1;
      // a row past the end repeats the first one, which changes no bound
      const int rr = in ? row : r0;
      v[u] = *reinterpret_cast<const uint4*>(base + static_cast<size_t>(rr) * C::kRowBytes);
      if constexpr (C::kAffine) {
        const size_t g = (cell * p.block_size + rr) * (D / 64) + col * C::kVals / 64;
        sc[u] = __bfloat162float(p.k_scales[g]);
        bi[u] = __bfloat162float(p.k_biases[g]);
      }
    }
#pragma unroll
    for (int u = 0; u < C::kUnroll; ++u) {
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (FMT == 16) {
          lo[k] = min_bf16x2(lo[k], w[k]);
          hi[k] = max_bf16x2(hi[k], w[k]);
        } else if constexpr (FMT == kFmtE4m3) {
          uint32_t a, c;
          e4m3x4_to_f16x2(w[k], a, c);
          lo[2 * k] = min_f16x2(lo[2 * k], a);
          hi[2 * k] = max_f16x2(hi[2 * k], a);
          lo[2 * k + 1] = min_f16x2(lo[2 * k + 1], c);
          hi[2 * k + 1] = max_f16x2(hi[2 * k + 1], c);
        } else {
          constexpr int kPer = 32 / FMT;  // codes per word
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            // each bound's roundings all go outward: to the nearest f32 a key could end inside
            const float c = static_cast<float>((w[k] >> (FMT * j)) & ((1u << FMT) - 1u));
            const int i = k * kPer + j;
            lo[i] = __float_as_uint(fminf(__uint_as_float(lo[i]), __fmaf_rd(sc[u], c, bi[u])));
            hi[i] = __float_as_uint(fmaxf(__uint_as_float(hi[i]), __fmaf_ru(sc[u], c, bi[u])));
          }
        }
      }
    }
  }
  // the row groups of the pass, into the first
  auto merge = [&](int i, uint32_t l, uint32_t m) {
    if constexpr (FMT == 16) {
      lo[i] = min_bf16x2(lo[i], l);
      hi[i] = max_bf16x2(hi[i], m);
    } else if constexpr (FMT == kFmtE4m3) {
      lo[i] = min_f16x2(lo[i], l);
      hi[i] = max_f16x2(hi[i], m);
    } else {
      lo[i] = __float_as_uint(fminf(__uint_as_float(lo[i]), __uint_as_float(l)));
      hi[i] = __float_as_uint(fmaxf(__uint_as_float(hi[i]), __uint_as_float(m)));
    }
  };
  if constexpr ((C::kLanes & (C::kLanes - 1)) == 0) {
#pragma unroll
    for (int d = C::kLanes; d < 32; d <<= 1)
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        merge(i, __shfl_xor_sync(0xffffffffu, lo[i], d), __shfl_xor_sync(0xffffffffu, hi[i], d));
  } else {
#pragma unroll
    for (int s = 1; s < C::kRowsPerPass; ++s)
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        merge(i, __shfl_down_sync(0xffffffffu, lo[i], s * C::kLanes), __shfl_down_sync(0xffffffffu, hi[i], s * C::kLanes));
  }
  if (lane >= C::kLanes) return;
  // 2 rows of D bf16: the lane's kVals values of each
  uint32_t* const out_lo = reinterpret_cast<uint32_t*>(p.k_bounds + cell * 2 * D + col * C::kVals);
  uint32_t* const out_hi = out_lo + D / 2;
  const float scale = FMT == kFmtE4m3 ? p.k_block_scales[cell] : 1.f;
#pragma unroll
  for (int q = 0; q < C::kVals / 8; ++q) {  // 8 values, one 16-byte store, at a time
    uint32_t l4[4], h4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (FMT == 16) {
        l4[i] = lo[4 * q + i];
        h4[i] = hi[4 * q + i];
      } else {
        float2 a, c;
        if constexpr (FMT == kFmtE4m3) {
          a = __half22float2(*reinterpret_cast<__half2*>(&lo[4 * q + i]));
          c = __half22float2(*reinterpret_cast<__half2*>(&hi[4 * q + i]));
          a = make_float2(__fmul_rd(a.x, scale), __fmul_rd(a.y, scale));
          c = make_float2(__fmul_ru(c.x, scale), __fmul_ru(c.y, scale));
        } else {
          a = make_float2(__uint_as_float(lo[8 * q + 2 * i]), __uint_as_float(lo[8 * q + 2 * i + 1]));
          c = make_float2(__uint_as_float(hi[8 * q + 2 * i]), __uint_as_float(hi[8 * q + 2 * i + 1]));
        }
        const __nv_bfloat162 l = __halves2bfloat162(__float2bfloat16_rd(a.x), __float2bfloat16_rd(a.y));
        const __nv_bfloat162 m = __halves2bfloat162(__float2bfloat16_ru(c.x), __float2bfloat16_ru(c.y));
        l4[i] = *reinterpret_cast<const uint32_t*>(&l);
        h4[i] = *reinterpret_cast<const uint32_t*>(&m);
      }
    }
    if (held) {
      const uint4 l = reinterpret_cast<const uint4*>(out_lo)[q], m = reinterpret_cast<const uint4*>(out_hi)[q];
      const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, mw[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l4[i] = min_bf16x2(l4[i], lw[i]);
        h4[i] = max_bf16x2(h4[i], mw[i]);
      }
    }
    reinterpret_cast<uint4*>(out_lo)[q] = make_uint4(l4[0], l4[1], l4[2], l4[3]);
    reinterpret_cast<uint4*>(out_hi)[q] = make_uint4(h4[0], h4[1], h4[2], h4[3]);
  }
}

template <int FMT, int D>
cudaError_t launch_bounds_of(const BoundsParams& p, int num_seqs, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((p.blocks * p.num_kv_heads + 3) / 4, num_seqs);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits before it touches memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pkv_bounds_kernel<FMT, D>, p);
}

// -------------------------------------------------------------------------------------- scores
// A warp scores 16 blocks at a time against all query rows of its KV head (up to 64) with
// m16n8k16 MMAs: blocks on M, query rows on N, and the products of the two bounds summed
// over 2 D. The order of the dims within the contraction is free, so the A fragments are the
// 16-byte loads themselves (each lane 8 dims of two blocks per load, four lanes a 64-byte
// run) and no bound passes through shared memory; the B fragment of the same dims is 16
// bytes of a query row. Bound by HBM: 4 D bytes per (block, KV head); 64 units of 8192 blocks,
// D=128, 16 query rows: 49 us, 0.81 of a copy's rate, ramp-up and tail included. The registers of each
// bound take the next tile's values as soon as the MMAs have read them, so that the 16 warps
// they leave room for keep loads in flight throughout. Bulk copies of a block's two rows (512
// bytes) into rings in shared memory were slower (64 units of 8192 blocks, D=128, scores and
// choice: 61.6 -> 70.2 us), and so were equal runs of all units' tiles over one wave of CTAs
// (64 sequences of 1024 to 32768 rows: 37.3 -> 42.5); half the registers for twice the warps
// changed nothing.
//
// Scores are stored as integers of the same order, NaN as -infinity.
constexpr uint32_t kLowestScore = 0x007FFFFFu;  // of -infinity, and of NaN
__device__ __forceinline__ uint32_t order_key(float s) {
  if (!(s == s)) return kLowestScore;
  const uint32_t u = __float_as_uint(s + 0.f);  // -0 as 0
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

constexpr int kScoreWarps = 4;  // of the kernel that scores alone
constexpr int kScoreTile = 16;  // blocks per warp and step

// Bytes of a staged query row: max(q, 0), min(q, 0), padded so that rows g, g + 1 meet in no bank.
constexpr __host__ __device__ int query_row_bytes(int D) { return D * 4 + 64; }

// Scores this warp's tiles first_tile, first_tile + step, ... (`count` of them, the same for
// every warp of the CTA) of unit (b, h) with n blocks; sq: space for the query rows. ready()
// runs once, in every thread, before the first result; put(j, key) and put_tile(tile, m) take
// a block's score and the bits of a tile's largest |bound|.
// NT: most tiles of 8 query rows (nq <= 8 NT).
template <int D, int NT, int WARPS, typename Ready, typename Put, typename PutTile>
__device__ __forceinline__ void score_tiles(const SelectParams& p, size_t unit, int h, const int32_t* table, int n,
                                            int first_tile, int step, int count, uint8_t* sq, Ready ready, Put put,
                                            PutTile put_tile) {
  constexpr int kSteps = D / 32;  // 16-byte loads per bound row and lane
  constexpr int kStride = query_row_bytes(D);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ntiles = (p.nq + 7) / 8;  // tiles of 8 query rows

  // a tile's block ids, one per lane of the first 16; -1 past the last block
  auto ids_of = [&](int it) {
    const int j = (first_tile + it * step) * kScoreTile + lane;
    return it < count && lane < kScoreTile && j < n ? table[j] : -1;
  };
  auto good = [&](int ph) { return static_cast<unsigned>(ph) < static_cast<unsigned>(p.num_blocks); };
  // one bound (0: lo, 1: hi) of blocks ph0 and ph1, in fragment order; zeros for a bad block
  auto load = [&](int ph0, int ph1, int bound, uint4 (&a)[kSteps], uint4 (&b)[kSteps]) {
    const __nv_bfloat16* r0 = p.k_bounds + (static_cast<size_t>(ph0 < 0 ? 0 : ph0) * p.num_kv_heads + h) * 2 * D + 8 * t;
    const __nv_bfloat16* r1 = p.k_bounds + (static_cast<size_t>(ph1 < 0 ? 0 : ph1) * p.num_kv_heads + h) * 2 * D + 8 * t;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      a[i] = ph0 >= 0 ? ld_nc_keep_v4(r0 + bound * D + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
      b[i] = ph1 >= 0 ? ld_nc_keep_v4(r1 + bound * D + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  // the blocks g and g + 8 of a tile, -1 where there is none
  auto pick = [&](int ids, int& ph0, int& ph1) {
    const int ph = good(ids) ? ids : -1;
    ph0 = __shfl_sync(0xffffffffu, ph, g);
    ph1 = __shfl_sync(0xffffffffu, ph, g + 8);
  };

  int ids = ids_of(0), ids_next = ids_of(1);
  uint4 lo0[kSteps], hi0[kSteps], lo1[kSteps], hi1[kSteps];
  int ph0, ph1;
  pick(ids, ph0, ph1);
  load(ph0, ph1, 1, hi0, hi1);
  load(ph0, ph1, 0, lo0, lo1);
  {  // the query rows, max(q, 0) then min(q, 0), staged while the first bounds are in flight; a
     // NaN stays one, so that its row's sums are NaN and no score of a block
    const uint4* q = reinterpret_cast<const uint4*>(p.q + unit * p.nq * D);
    for (int i = threadIdx.x; i < ntiles * 8 * (D / 8); i += WARPS * 32) {
      const int r = i / (D / 8), c = i - r * (D / 8);
      const uint4 v = r < p.nq ? q[i] : make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(sq + r * kStride + c * 16) =
          make_uint4(positive_bf16x2(v.x), positive_bf16x2(v.y), positive_bf16x2(v.z), positive_bf16x2(v.w));
      *reinterpret_cast<uint4*>(sq + r * kStride + D * 2 + c * 16) =
          make_uint4(negative_bf16x2(v.x), negative_bf16x2(v.y), negative_bf16x2(v.z), negative_bf16x2(v.w));
    }
    __syncthreads();
    ready();
  }
  for (int it = 0; it < count; ++it) {
    const int j0 = (first_tile + it * step) * kScoreTile;  // warp-uniform
    if (j0 >= n) break;
    if (!good(ids) && lane < kScoreTile && j0 + lane < n && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
    int next0, next1;
    pick(ids_next, next0, next1);
    const int ids_after = ids_of(it + 2);
    // Each bound's registers take the next tile's as soon as the MMAs have read them, so that
    // loads are in flight throughout. mm: the tile's largest magnitude, for the choice's E.
    uint32_t mm[4] = {0u, 0u, 0u, 0u};
    float acc[NT][2][4];  // <max(q, 0), hi> and <min(q, 0), lo>, apart for the sake of latency
    auto half = [&](int bound, uint4 (&a)[kSteps], uint4 (&b)[kSteps]) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        mm[0] = max_abs_bf16x2(max_abs_bf16x2(mm[0], a[i].x), b[i].x);
        mm[1] = max_abs_bf16x2(max_abs_bf16x2(mm[1], a[i].y), b[i].y);
        mm[2] = max_abs_bf16x2(max_abs_bf16x2(mm[2], a[i].z), b[i].z);
        mm[3] = max_abs_bf16x2(max_abs_bf16x2(mm[3], a[i].w), b[i].w);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float (&c)[4] = acc[nt][bound];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = 0.f;
        if (nt >= ntiles) continue;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint4 q = *reinterpret_cast<const uint4*>(sq + (8 * nt + g) * kStride + (bound ? 0 : D * 2) +
                                                          (32 * i + 8 * t) * 2);
          mma_bf16(c, a[i].x, b[i].x, a[i].y, b[i].y, q.x, q.y);
          mma_bf16(c, a[i].z, b[i].z, a[i].w, b[i].w, q.z, q.w);
        }
      }
      load(next0, next1, bound, a, b);
    };
    half(1, hi0, hi1);
    half(0, lo0, lo1);
    uint32_t m = max_bf16x2(max_bf16x2(mm[0], mm[1]), max_bf16x2(mm[2], mm[3]));
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    put_tile(first_tile + it * step, m << 16);

    float best0 = -INFINITY, best1 = -INFINITY;  // blocks j0 + g and j0 + g + 8
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (8 * nt + 2 * t + e < p.nq) {
          best0 = fmaxf(best0, acc[nt][0][e] + acc[nt][1][e]);
          best1 = fmaxf(best1, acc[nt][0][e + 2] + acc[nt][1][e + 2]);
        }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      best0 = fmaxf(best0, __shfl_xor_sync(0xffffffffu, best0, d));
      best1 = fmaxf(best1, __shfl_xor_sync(0xffffffffu, best1, d));
    }
    if (t == 0) {
      if (j0 + g < n) put(j0 + g, order_key(ph0 >= 0 ? best0 : -INFINITY));
      if (j0 + g + 8 < n) put(j0 + g + 8, order_key(ph1 >= 0 ? best1 : -INFINITY));
    }
    ph0 = next0;
    ph1 = next1;
    ids = ids_next;
    ids_next = ids_after;
  }
}

// Scores alone, into the workspace.
template <int D, int NT>
__global__ void __launch_bounds__(kScoreWarps * 32) pkv_score_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) uint8_t sq[];
  wait_for_prerequisite_grids();
  allow_dependent_launch();  // the choice may take its place on the SMs; it waits for this grid's end
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the KV heads of a run of blocks are neighbours in the grid, as their bounds are in memory
  const int chunk = blockIdx.x / p.num_kv_heads, h = blockIdx.x - chunk * p.num_kv_heads, b = blockIdx.y;
  const size_t unit = static_cast<size_t>(b) * p.num_kv_heads + h;
  const int len = p.seq_lens[b];
  if (len < p.n_query || len > p.max_blocks * p.block_size) return;  // the choice flags it
  const int n = (len + p.block_size - 1) / p.block_size;
  const int cta_tile = chunk * kScoreWarps * p.tiles_per_warp;
  if (n <= p.top_k || cta_tile * kScoreTile >= n) return;  // every block is taken, or none is here
  score_tiles<D, NT, kScoreWarps>(
      p, unit, h, p.block_tables + static_cast<size_t>(b) * p.max_blocks, n, cta_tile + warp, kScoreWarps,
      p.tiles_per_warp, sq, [] {}, [&](int j, uint32_t key) { p.scores[unit * p.score_stride + j] = key; },
      [&](int tile, uint32_t m) {
        if (lane == 0) p.tile_abs[unit * p.tiles + tile] = __uint_as_float(m);
      });
}

// -------------------------------------------------------------------------------------- choice
// One CTA per (sequence, KV head). The blocks taken are those that exact sums would take,
// ties to the lower block: f32 scores decide all but the few within their error bound E of
// the last place, and those are summed again in pairs of f32 (48 bits; the products of bf16
// values are exact, and so is nearly every sum of up to 256 of them).
//
// With T the k-th largest of the candidates' f32 scores and |f32 - exact| <= E: a score
// above T + 2E is in (at most k - 1 scores lie above T, and a block below T cannot overtake
// it), one below T - 2E is out, the rest is ambiguous. E = 1.5 D 2^-25 |q|_1 max|bound|: an MMA
// adds 16 exact products and the f32 accumulator, each cut toward 0 below 2^-25 of the power of
// two that the largest addend reaches, and cuts the sum to 24 bits (2^-23), as sums made to show
// it do on this GPU. With A the magnitudes summed in an accumulator, an MMA is thus off by at most
// (17 + 4) 2^-25 A, the D / 16 MMAs of both accumulators by 21/16 D 2^-25 (A + A'), A + A' at most
// |q|_1 max|bound|, and their sum by 2^-24 of it: 1.35 D 2^-25 in all. Spread scores stay under a
// tenth of E.
//
// T comes from histograms of 2048 equal bins over [lowest, highest] key, narrowed to the bin
// that holds the k-th until that holds at most 32 keys, which every warp then ranks (one round
// as a rule): spread scores meet few bank conflicts, which radix digits of nearby floats would.
// The marks of 32 blocks at a time (ballots) and a prefix over their counts then give each taken
// block its place.
//
// The CTA's time is a chain of dependent steps (loads, barriers, prefixes), so it takes as
// few warps as its blocks need: 8 for tables of up to 2048 blocks, 32 above (8192 blocks: 8.6 us
// a CTA; with 8 scores per thread in registers 7.1 us, but no faster a step, for twice the code).
constexpr int kSelectBins = 2048;
constexpr int kSelectMostKeys = 24576;  // scores kept in shared memory; more are read again from L2
constexpr int kSelectAmbiguous = 256;   // ambiguous blocks ranked in shared memory; more by way of the workspace
constexpr uint32_t kForced = 0xFFFFFFFFu;  // key of a block that is always taken; no score has it

template <int T>
struct SelectShared {
  static constexpr int kSegment = 32 * T;  // blocks whose marks fit at once, a word per thread
  union {
    int hist[kSelectBins];
    unsigned long long pairs[T / 32][2];
    struct {
      uint32_t sure[T], amb[T];  // marks of 32 blocks: taken, ambiguous
    } marks;
  };
  uint32_t red[32];
  unsigned long long few[32];  // keys of the threshold's bin
  unsigned long long amb_key[kSelectAmbiguous];  // ambiguous blocks: the exact score's key
  int amb[kSelectAmbiguous];                     // and the block
  int bin, above, in_bin, few_count;
};

// Exclusive prefix over the block, in thread order, and the total.
template <int T>
__device__ __forceinline__ uint32_t block_prefix(SelectShared<T>& sh, uint32_t v, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  __syncthreads();  // red is free
  if (lane == 31) sh.red[warp] = incl;
  __syncthreads();
  uint32_t w = lane < T / 32 ? sh.red[lane] : 0u;  // every warp scans the warps' sums
  const uint32_t own = w;
#pragma unroll
  for (int d = 1; d < T / 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  total = __shfl_sync(0xffffffffu, w, T / 32 - 1);
  return __shfl_sync(0xffffffffu, w - own, warp) + incl - v;
}

// The need-th largest (need >= 1) of the keys in [lo, hi] that key_of(i, &key) yields for i
// in [0, n); `need` becomes its rank among the keys equal to it. Every thread gets it.
template <int T, typename Key, typename F>
__device__ __forceinline__ Key nth_largest(SelectShared<T>& sh, F key_of, int n, int& need, Key lo, Key hi) {
  for (;;) {
    const Key span = hi - lo;
    const int width = sizeof(Key) == 8 ? 64 - __clzll(static_cast<long long>(span)) : 32 - __clz(static_cast<int>(span));
    const int shift = width > 11 ? width - 11 : 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kSelectBins; i += T) sh.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += T) {
      Key k;
      if (key_of(i, k) && k >= lo && k <= hi) atomicAdd(&sh.hist[static_cast<int>((k - lo) >> shift)], 1);
    }
    __syncthreads();
    // bins from the top, a few per thread
    constexpr int kPer = kSelectBins / T;
    const int top = kSelectBins - 1 - kPer * threadIdx.x;
    int sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += sh.hist[top - j];
    uint32_t all;
    int above = static_cast<int>(block_prefix(sh, static_cast<uint32_t>(sum), all));
    if (above < need && above + sum >= need) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int c = sh.hist[top - j];
        if (above < need && above + c >= need) {
          sh.few_count = 0;
          sh.bin = top - j;
          sh.above = above;
          sh.in_bin = c;
        }
        above += c;
      }
    }
    __syncthreads();
    need -= sh.above;
    lo += static_cast<Key>(sh.bin) << shift;
    if (shift == 0) return lo;
    const Key end = lo + ((static_cast<Key>(1) << shift) - 1);
    hi = end < hi ? end : hi;
    const int in_bin = sh.in_bin;
    if (in_bin <= 32) {  // few in the bin: every warp ranks them, a lane each
      for (int i = threadIdx.x; i < n; i += T) {
        Key k;
        if (key_of(i, k) && k >= lo && k <= hi) sh.few[atomicAdd(&sh.few_count, 1) & 31] = static_cast<unsigned long long>(k);
      }
      __syncthreads();
      const int lane = threadIdx.x & 31;
      const Key mine = lane < in_bin ? static_cast<Key>(sh.few[lane]) : Key(0);
      int greater = 0, equal = 0;
      for (int i = 0; i < in_bin; ++i) {
        const Key o = __shfl_sync(0xffffffffu, mine, i);
        greater += o > mine;
        equal += o == mine;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, lane < in_bin && greater < need && need <= greater + equal);
      const int at = hit ? __ffs(hit) - 1 : 0;
      need -= __shfl_sync(0xffffffffu, greater, at);
      return __shfl_sync(0xffffffffu, mine, at);
    }
  }
}

// A sum kept as an unevaluated pair of f32 (hi + lo, |lo| at most half a step of hi): the
// rounding error of each addition is itself an f32 and joins lo, so the pair carries about
// 48 bits. The f64 unit is far slower on this GPU (2 lanes per clock and SM).
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  const float s = __fadd_rn(a.hi, b.hi), v = __fsub_rn(s, a.hi);
  if (!(fabsf(s) < INFINITY)) return Pair{s, 0.f};  // infinite or NaN: no error term
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, v)), __fsub_rn(b.hi, v));  // s + e = a.hi + b.hi exactly
  const float l = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  const float h = __fadd_rn(s, l);
  return Pair{h, __fsub_rn(l, __fsub_rn(h, s))};
}

// of a NaN score and of a bad block
constexpr unsigned long long kLowestKey = static_cast<unsigned long long>(kLowestScore) << 32;
constexpr int kExactRows = 4;  // query rows summed side by side, so that their chains of additions overlap

// The largest u_j of query rows r0 .. r0 + kExactRows - 1 (within nq) as an ordered integer,
// by one warp: the products of bf16 values are exact in f32 (above 2^-134). Pairs order by
// hi, then by lo.
__device__ __forceinline__ unsigned long long exact_key(const __nv_bfloat16* q, int r0, int nq,
                                                        const __nv_bfloat16* bounds, int D, int lane) {
  Pair s[kExactRows];
#pragma unroll
  for (int r = 0; r < kExactRows; ++r) s[r] = Pair{0.f, 0.f};
  for (int d = 2 * lane; d < D; d += 64) {
    const __nv_bfloat162 l = *reinterpret_cast<const __nv_bfloat162*>(bounds + d);
    const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(bounds + D + d);
#pragma unroll
    for (int r = 0; r < kExactRows; ++r) {
      const int row = r0 + r < nq ? r0 + r : nq - 1;
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(q + static_cast<size_t>(row) * D + d);
      const float x0 = __low2float(x), x1 = __high2float(x);
      s[r] = pair_add(s[r], Pair{fmaxf(x0 * __low2float(l), x0 * __low2float(h)), 0.f});
      s[r] = pair_add(s[r], Pair{fmaxf(x1 * __high2float(l), x1 * __high2float(h)), 0.f});
    }
  }
#pragma unroll
  for (int k = 16; k > 0; k >>= 1)
#pragma unroll
    for (int r = 0; r < kExactRows; ++r)
      s[r] = pair_add(s[r], Pair{__shfl_xor_sync(0xffffffffu, s[r].hi, k), __shfl_xor_sync(0xffffffffu, s[r].lo, k)});
  unsigned long long best = kLowestKey;
#pragma unroll
  for (int r = 0; r < kExactRows; ++r) {
    const uint32_t hi = order_key(s[r].hi);
    const unsigned long long key =
        hi == kLowestScore ? kLowestKey : (static_cast<unsigned long long>(hi) << 32) | order_key(s[r].lo);
    best = key > best ? key : best;
  }
  return best;
}

// The largest 1-norm of the unit's query rows this warp looks at.
template <int T>
__device__ __forceinline__ float query_norm(const SelectParams& p, int unit) {
  const __nv_bfloat16* q = p.q + static_cast<size_t>(unit) * p.nq * p.head_dim;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float q1 = 0.f;
  for (int r = warp; r < p.nq; r += T / 32) {  // a row's D / 8 <= 32 lanes hold 8 values each
    float s = 0.f;
    if (lane < p.head_dim / 8) {
      const uint4 v = ld_nc_keep_v4(q + static_cast<size_t>(r) * p.head_dim + 8 * lane);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s += fabsf(__uint_as_float(w[e] << 16)) + fabsf(__uint_as_float(w[e] & 0xFFFF0000u));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    q1 = fmaxf(q1, s);
  }
  return q1;
}

// Chooses the blocks of one unit. FUSED: sh_keys holds the scores of its n blocks and
// `mag_bits` the largest |bound| this thread knows of; else both are read from the workspace.
template <int T, bool FUSED>
__device__ __forceinline__ void select_unit(const SelectParams& p, SelectShared<T>& sh, uint32_t* sh_keys, int unit,
                                            int len, float q1, uint32_t mag_bits) {
  constexpr int kSegment = SelectShared<T>::kSegment;
  const int b = unit / p.num_kv_heads, h = unit - b * p.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const __nv_bfloat16* q = p.q + static_cast<size_t>(unit) * p.nq * p.head_dim;
  int32_t* const out_blocks = p.out_blocks ? p.out_blocks + static_cast<size_t>(unit) * p.top_k : nullptr;
  int32_t* const out_table = p.out_tables + static_cast<size_t>(unit) * p.table_width;
  const int32_t* table = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  const bool bad = len < p.n_query || len > p.max_blocks * p.block_size;
  const int n = bad ? 0 : (len + p.block_size - 1) / p.block_size;
  const int taken = n < p.top_k ? n : p.top_k;
  if (threadIdx.x == 0) {
    p.out_lens[unit] = bad ? 0 : (taken - 1) * p.block_size + (len - (n - 1) * p.block_size);
    if (bad && p.error_flag) atomicOr(p.error_flag, kDevErrBadSeqLen);
  }
  auto put = [&](int pos, int j) {  // block j at place pos of the choice
    const int ph = j < 0 ? -1 : table[j];
    const bool ok = static_cast<unsigned>(ph) < static_cast<unsigned>(p.num_blocks);
    if (out_blocks) out_blocks[pos] = j;
    if (pos < p.table_width) out_table[pos] = ok ? ph * p.num_kv_heads + h : -1;
    if (j >= 0 && !ok && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
  };
  for (int i = taken + threadIdx.x; i < p.top_k; i += T) put(i, -1);
  if (n <= p.top_k) {
    for (int j = threadIdx.x; j < n; j += T) put(j, j);
    return;
  }
  const uint32_t* scores = p.scores + static_cast<size_t>(unit) * p.score_stride;  // 16-byte aligned
  unsigned long long* const keys64 = p.keys64 + static_cast<size_t>(unit) * p.max_blocks;
  const bool staged = FUSED || n <= p.key_space;
  auto forced = [&](int j) { return j < p.first || j >= n - p.last; };
  auto key_at = [&](int j) { return staged ? sh_keys[j] : forced(j) ? kForced : __ldcg(scores + j); };

  // keys and the candidates' range; the bounds' largest magnitude
  uint32_t kmin = 0xFFFFFFFFu, kmax = 0u;
  if constexpr (FUSED) {
    for (int j = threadIdx.x; j < n; j += T) {
      if (forced(j)) {
        sh_keys[j] = kForced;
      } else {
        kmin = min(kmin, sh_keys[j]);
        kmax = max(kmax, sh_keys[j]);
      }
    }
  }
  float mag = __uint_as_float(mag_bits);
  const int tiles = (n + kScoreTile - 1) / kScoreTile;
  constexpr int kBatch = 2;
  for (int j0 = 4 * threadIdx.x, t0 = threadIdx.x; !FUSED && j0 < n; j0 += 4 * T * kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + 4 * T * u;
      v[u] = j < n ? __ldcg(reinterpret_cast<const uint4*>(scores + j)) : make_uint4(0u, 0u, 0u, 0u);
    }
    for (; t0 < tiles && t0 < j0 + 4 * T * kBatch; t0 += T)
      mag = fmaxf(mag, __ldcg(p.tile_abs + static_cast<size_t>(unit) * p.tiles + t0));
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + 4 * T * u;
      uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (j + e >= n) continue;
        if (forced(j + e)) {
          w[e] = kForced;
        } else {
          kmin = min(kmin, w[e]);
          kmax = max(kmax, w[e]);
        }
        if (staged) sh_keys[j + e] = w[e];
      }
    }
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  const uint32_t mag_u = __reduce_max_sync(0xffffffffu, __float_as_uint(mag));
  if (lane == 0) {
    sh.pairs[warp][0] = (static_cast<unsigned long long>(kmin) << 32) | kmax;
    sh.pairs[warp][1] = (static_cast<unsigned long long>(mag_u) << 32) | __float_as_uint(q1);
  }
  __syncthreads();
  uint32_t mu = 0u, qu = 0u;
  if (lane < T / 32) {
    const unsigned long long x = sh.pairs[lane][0], y = sh.pairs[lane][1];
    kmin = static_cast<uint32_t>(x >> 32);
    kmax = static_cast<uint32_t>(x);
    mu = static_cast<uint32_t>(y >> 32);
    qu = static_cast<uint32_t>(y);
  }
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  mu = __reduce_max_sync(0xffffffffu, mu);
  qu = __reduce_max_sync(0xffffffffu, qu);
  float err = static_cast<float>(p.head_dim) * 4.47034836e-8f * __uint_as_float(qu) * __uint_as_float(mu);  // E
  // Where E leaves the normal range so may the products, whose roundings E does not count: exact sums decide.
  if (qu != 0u && mu != 0u && err < 1.17549435e-38f) err = INFINITY;

  // keys over `above` are taken, under `below` not; the ones between are ambiguous
  uint32_t above = kForced - 1u, below = kForced;
  const int k = p.top_k - p.first - p.last;
  if (k > 0) {
    int rank = k;
    const float s = key_score(nth_largest<T, uint32_t>(
        sh, [&](int j, uint32_t& key) { key = key_at(j); return key != kForced; }, n, rank, kmin, kmax));
    const float hi = s + 2.f * err, lo = s - 2.f * err;  // NaN past infinity: then every score is ambiguous
    above = hi == hi ? order_key(hi) : kForced - 1u;
    below = lo == lo ? order_key(lo) : 0u;
  }
  auto is_amb = [&](uint32_t key) { return key <= above && key >= below; };
  // marks of the 32 blocks of each word of a segment: taken, ambiguous
  auto mark = [&](int seg) {
    __syncthreads();
    for (int w = warp; w < T && seg + 32 * w < n; w += T / 32) {
      const int j = seg + 32 * w + lane;
      const uint32_t key = j < n ? key_at(j) : 0u;
      const uint32_t ms = __ballot_sync(0xffffffffu, j < n && key > above);
      const uint32_t ma = __ballot_sync(0xffffffffu, j < n && is_amb(key));
      if (lane == 0) {
        sh.marks.sure[w] = ms;
        sh.marks.amb[w] = ma;
      }
    }
    __syncthreads();
  };
  // this thread's word of a segment, and the counts before it: taken in the high half,
  // ambiguous in the low half (a segment holds at most 2^15 blocks)
  uint32_t my_sure = 0u, my_amb = 0u;
  auto count = [&](int seg, uint32_t& total) {
    const bool on = seg + 32 * static_cast<int>(threadIdx.x) < n;
    my_sure = on ? sh.marks.sure[threadIdx.x] : 0u;
    my_amb = on ? sh.marks.amb[threadIdx.x] : 0u;
    return block_prefix(sh, (static_cast<uint32_t>(__popc(my_sure)) << 16) | __popc(my_amb), total);
  };
  int sure = 0, ambiguous = 0;
  uint32_t before = 0u, total = 0u;
  for (int seg = 0; seg < n; seg += kSegment) {
    mark(seg);
    before = count(seg, total);
    int at = ambiguous + static_cast<int>(before & 0xFFFFu);
    for (uint32_t m = my_amb; m && at < kSelectAmbiguous; m &= m - 1)
      sh.amb[at++] = seg + 32 * threadIdx.x + __ffs(m) - 1;
    sure += static_cast<int>(total >> 16);
    ambiguous += static_cast<int>(total & 0xFFFFu);
  }
  int ties = p.top_k - sure;  // how many ambiguous blocks are taken, in order where exact sums tie
  unsigned long long t64 = 0ull;
  const bool exact = ambiguous > ties && err != 0.f;  // err = 0: every product is 0, the scores are exact
  const bool few = ambiguous <= kSelectAmbiguous;
  bool remark = n > kSegment, recount = remark || exact;
  const int row_groups = (p.nq + kExactRows - 1) / kExactRows;
  // rank of ambiguous block i among them; the list is in block order
  auto rank_of = [&](int i) {
    int rank = 0;
    for (int o = 0; o < ambiguous; ++o)
      rank += sh.amb_key[o] > sh.amb_key[i] || (sh.amb_key[o] == sh.amb_key[i] && o < i);
    return rank;
  };
  if (exact) {
    auto bounds_of = [&](int j) -> const __nv_bfloat16* {  // nullptr for a bad block
      const int ph = table[j];
      if (static_cast<unsigned>(ph) >= static_cast<unsigned>(p.num_blocks)) return nullptr;
      return p.k_bounds + (static_cast<size_t>(ph) * p.num_kv_heads + h) * 2 * p.head_dim;
    };
    if (few) {  // as a rule: a warp per (block, query rows), then a rank by counting
      for (int i = threadIdx.x; i < ambiguous; i += T) sh.amb_key[i] = 0ull;
      __syncthreads();
      for (int w = warp; w < ambiguous * row_groups; w += T / 32) {
        const int at = w / row_groups, r = w - at * row_groups;
        const __nv_bfloat16* bd = bounds_of(sh.amb[at]);
        const unsigned long long key = bd ? exact_key(q, r * kExactRows, p.nq, bd, p.head_dim, lane) : kLowestKey;
        if (lane == 0) atomicMax(&sh.amb_key[at], key);
      }
      __syncthreads();
      if (!remark) {  // unmark those that are not taken
        for (int i = threadIdx.x; i < ambiguous; i += T)
          if (rank_of(i) >= ties) atomicAnd(&sh.marks.amb[sh.amb[i] / 32], ~(1u << (sh.amb[i] & 31)));
        __syncthreads();
      }
    } else {
      unsigned long long lo64 = ~0ull, hi64 = 0ull;  // range of this warp's keys
      for (int i0 = warp * 32; i0 < n; i0 += T) {
        uint32_t todo = __ballot_sync(0xffffffffu, i0 + lane < n && is_amb(key_at(min(i0 + lane, n - 1))));
        while (todo) {
          const int j = i0 + __ffs(todo) - 1;
          todo &= todo - 1;
          const __nv_bfloat16* bd = bounds_of(j);
          unsigned long long key = kLowestKey;
          for (int r = 0; bd && r < p.nq; r += kExactRows) {
            const unsigned long long of = exact_key(q, r, p.nq, bd, p.head_dim, lane);
            key = of > key ? of : key;
          }
          if (lane == 0) keys64[j] = key;
          lo64 = key < lo64 ? key : lo64;
          hi64 = key > hi64 ? key : hi64;
        }
      }
      __syncthreads();  // the keys are written, the marks' space is free
      if (lane == 0) {
        sh.pairs[warp][0] = lo64;
        sh.pairs[warp][1] = hi64;
      }
      __syncthreads();
      for (int i = 0; i < T / 32; ++i) {
        lo64 = sh.pairs[i][0] < lo64 ? sh.pairs[i][0] : lo64;
        hi64 = sh.pairs[i][1] > hi64 ? sh.pairs[i][1] : hi64;
      }
      t64 = nth_largest<T, unsigned long long>(
          sh,
          [&](int j, unsigned long long& key) {
            if (!is_amb(key_at(j))) return false;
            key = keys64[j];
            return true;
          },
          n, ties, lo64, hi64);
      remark = true;
    }
  }
  // Places: each thread its word of a segment. The chosen go to a list first where it fits,
  // so that their table entries are read all at once.
  const bool listed = p.top_k <= p.key_space;
  int* const list = reinterpret_cast<int*>(sh_keys);
  int placed = 0, tied = 0;  // taken and ambiguous blocks of earlier segments
  for (int seg = 0; seg < n; seg += kSegment) {
    if (remark) {
      mark(seg);
      if (exact && few) {  // several segments: unmark this one's
        for (int i = threadIdx.x; i < ambiguous; i += T) {
          const int j = sh.amb[i] - seg;
          if (j >= 0 && j < kSegment && rank_of(i) >= ties) atomicAnd(&sh.marks.amb[j / 32], ~(1u << (j & 31)));
        }
      } else if (exact) {  // above the threshold: taken; at it: in order; below: not
        for (int w = threadIdx.x; w < T && seg + 32 * w < n; w += T) {
          for (uint32_t m = sh.marks.amb[w]; m; m &= m - 1) {
            const uint32_t bit = m & (0u - m);
            const unsigned long long key = keys64[seg + 32 * w + __ffs(m) - 1];
            if (key > t64) sh.marks.sure[w] |= bit;
            if (key != t64) sh.marks.amb[w] &= ~bit;
          }
        }
      }
      __syncthreads();
    }
    if (recount) {
      before = count(seg, total);
    } else {
      __syncthreads();  // the keys' last reader is done: the list takes their place
    }
    int s = placed + static_cast<int>(before >> 16), a = tied + static_cast<int>(before & 0xFFFFu);
    for (uint32_t m = my_sure | my_amb; m; m &= m - 1) {
      const uint32_t bit = m & (0u - m);
      const int j = seg + 32 * threadIdx.x + __ffs(m) - 1;
      const bool is_sure = (my_sure & bit) != 0u;
      if (is_sure || a < ties) {
        const int pos = s + min(a, ties);
        if (listed) {
          list[pos] = j;
        } else {
          put(pos, j);
        }
      }
      s += is_sure;
      a += !is_sure;
    }
    placed += static_cast<int>(total >> 16);
    tied += static_cast<int>(total & 0xFFFFu);
  }
  if (!listed) return;
  __syncthreads();
  for (int i = threadIdx.x; i < p.top_k; i += T) put(i, list[i]);
}

// The choice alone, from the workspace's scores.
template <int T>
__global__ void __launch_bounds__(T, 1024 / T) pkv_select_kernel(const __grid_constant__ SelectParams p) {
  __shared__ SelectShared<T> sh;
  extern __shared__ __align__(16) uint32_t sh_keys[];  // [key_space]: the scores, later the chosen blocks
  // Behind the scores, this grid starts once every CTA of theirs has seen the work before
  // them complete: the inputs may be read before the scores are waited for.
  if (!p.after_scores) wait_for_prerequisite_grids();
  const int unit = blockIdx.x;
  const int len = p.seq_lens[unit / p.num_kv_heads];
  const float q1 = query_norm<T>(p, unit);
  if (p.after_scores) wait_for_prerequisite_grids();
  allow_dependent_launch();  // the attention may take its place on the SMs; it waits for this grid's end
  select_unit<T, false>(p, sh, sh_keys, unit, len, q1, 0u);
}

// Scores and choice of one unit by a cluster of 1 to 8 CTAs: each scores its share of the
// tiles, one per warp, into the first CTA's shared memory, and that one chooses. One launch
// less, and no trip of the scores through L2: 8 units of 1024 blocks (D=128, 4 query rows)
// 11.4 -> 10.9 us on the GPU (7.9 where no unit has blocks to sum exactly) and 2.7 us less per call
// from the host. With several tiles per
// warp or more than one wave of clusters the two kernels were faster (fused -> two: 64 units
// of 626 blocks, D=256, 17.4 -> 15.7 us; 512 of up to 1024, 43.2 -> 39.8; 64 of 8192,
// 64.6 -> 61.6).
constexpr int kFusedThreads = 256;
constexpr int kFusedCluster = 8;
constexpr int kFusedBlocks = kFusedCluster * kFusedThreads / 32 * kScoreTile;  // 1024

template <int D, int NT>
__global__ void __launch_bounds__(kFusedThreads)
    pkv_choose_kernel(const __grid_constant__ SelectParams p) {
  __shared__ SelectShared<kFusedThreads> sh;
  __shared__ uint32_t mags[kFusedCluster * kFusedThreads / 32];  // largest |bound| per warp of the cluster
  extern __shared__ __align__(16) uint32_t sh_keys[];  // [key_space]: scores, later the chosen blocks; then query rows
  wait_for_prerequisite_grids();
  allow_dependent_launch();  // the attention may take its place on the SMs; it waits for this grid's end
  const int rank = blockIdx.x, ctas = gridDim.x, unit = blockIdx.y;
  const int b = unit / p.num_kv_heads, h = unit - b * p.num_kv_heads;
  const int len = p.seq_lens[b];
  const float q1 = rank == 0 ? query_norm<kFusedThreads>(p, unit) : 0.f;
  const int n = len < p.n_query || len > p.max_blocks * p.block_size ? 0 : (len + p.block_size - 1) / p.block_size;
  uint32_t mag = 0u;
  if (n > p.top_k) {  // the same for the whole cluster
    constexpr int kWarps = kFusedThreads / 32;
    const int warp = threadIdx.x >> 5, tiles = (n + kScoreTile - 1) / kScoreTile;
    cluster_arrive_relaxed();  // tells that this CTA runs; the first CTA's memory is written after all have
    score_tiles<D, NT, kWarps>(
        p, unit, h, p.block_tables + static_cast<size_t>(b) * p.max_blocks, n, rank * kWarps + warp, ctas * kWarps,
        (tiles + ctas * kWarps - 1) / (ctas * kWarps), reinterpret_cast<uint8_t*>(sh_keys + p.key_space),
        [] { cluster_wait(); }, [&](int j, uint32_t key) { st_cluster_u32(smem_addr(sh_keys + j), 0, key); },
        [&](int, uint32_t m) { mag = max(mag, m); });
    if ((threadIdx.x & 31) == 0) st_cluster_u32(smem_addr(mags + rank * kWarps + warp), 0, mag);
    cluster_sync();
    if (rank != 0) return;
    mag = threadIdx.x < ctas * kWarps ? mags[threadIdx.x] : 0u;
  } else if (rank != 0) {
    return;
  }
  select_unit<kFusedThreads, true>(p, sh, sh_keys, unit, len, q1, mag);
}

// Raises a kernel's dynamic shared memory limit once per device.
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& configured, int device) {
  const unsigned long long bit = device >= 0 && device < 64 ? 1ull << device : 0ull;  // a bit per device < 64
  if (bit && (configured.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <int T>
cudaError_t launch_select_of(const SelectParams& p, int num_seqs, int device, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = allow_smem(pkv_select_kernel<T>, kSelectMostKeys * sizeof(uint32_t), configured, device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(num_seqs) * p.num_kv_heads);
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = p.key_space * sizeof(uint32_t);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits before it touches memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pkv_select_kernel<T>, p);
}

template <int D, int NT>
cudaError_t launch_score_of(const SelectParams& p, int num_seqs, int device, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e = allow_smem(pkv_score_kernel<D, NT>, 64 * query_row_bytes(D), configured, device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const int per_cta = kScoreWarps * p.tiles_per_warp;
  const long long ctas = static_cast<long long>((p.tiles + per_cta - 1) / per_cta) * p.num_kv_heads;
  if (ctas >= (1ll << 31)) return cudaErrorInvalidValue;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), num_seqs);
  cfg.blockDim = dim3(kScoreWarps * 32);
  cfg.dynamicSmemBytes = (p.nq + 7) / 8 * 8 * query_row_bytes(D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits before it touches memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pkv_score_kernel<D, NT>, p);
}

template <int D, int NT>
cudaError_t launch_choose_of(const SelectParams& p, int units, int cluster, int device, cudaStream_t stream) {
  static std::atomic<unsigned long long> configured{0};
  const cudaError_t e =
      allow_smem(pkv_choose_kernel<D, NT>, kFusedBlocks * 4 + 64 * query_row_bytes(D), configured, device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cluster, units);
  cfg.blockDim = dim3(kFusedThreads);
  cfg.dynamicSmemBytes = p.key_space * sizeof(uint32_t) + (p.nq + 7) / 8 * 8 * query_row_bytes(D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits before it touches memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pkv_choose_kernel<D, NT>, p);
}

}  // namespace

cudaError_t launch_bounds(const BoundsParams& p, int fmt, int head_dim, int num_seqs, cudaStream_t stream) {
#define X(F_, D_) \
  if (fmt == F_ && head_dim == D_) return launch_bounds_of<F_, D_>(p, num_seqs, stream);
  X(16, 64) X(16, 128) X(16, 192) X(16, 256) X(8, 128) X(8, 256) X(4, 128) X(4, 256)
  X(kFmtE4m3, 64) X(kFmtE4m3, 128) X(kFmtE4m3, 192) X(kFmtE4m3, 256)
#undef X
  return cudaErrorInvalidValue;
}

int select_tiles(int max_blocks) { return (max_blocks + kScoreTile - 1) / kScoreTile; }

cudaError_t launch_select(SelectParams p, int num_seqs, int sm_count, int device, cudaStream_t stream) {
  p.tiles = select_tiles(p.max_blocks);
  if (p.max_blocks <= kFusedBlocks) {
    const int units = num_seqs * p.num_kv_heads;  // at most 65535
    int cluster = 1;
    while (cluster * (kFusedThreads / 32) < p.tiles) cluster *= 2;
    if (units * cluster <= sm_count) {
      p.key_space = (p.max_blocks + 3) / 4 * 4;
#define X(D_, NT_) \
  if (p.head_dim == D_ && p.nq <= 8 * NT_) return launch_choose_of<D_, NT_>(p, units, cluster, device, stream);
      X(64, 1) X(128, 1) X(192, 1) X(256, 1) X(64, 8) X(128, 8) X(192, 8) X(256, 8)
#undef X
      return cudaErrorInvalidValue;
    }
  }
  if (p.max_blocks > p.top_k) {  // else every block is taken
    // A warp takes one tile while that fills the GPU about four times over, then up to 8, so
    // that the query rows are staged for more of them.
    const long long tiles = static_cast<long long>(p.tiles) * p.num_kv_heads * num_seqs;
    const long long fill = 4ll * 16 * (sm_count > 0 ? sm_count : 1);
    const long long per = tiles / fill;
    p.tiles_per_warp = static_cast<int>(per < 1 ? 1 : per > 8 ? 8 : per);
    auto score = [&]() -> cudaError_t {
#define X(D_, NT_) \
  if (p.head_dim == D_ && p.nq <= 8 * NT_) return launch_score_of<D_, NT_>(p, num_seqs, device, stream);
      X(64, 1) X(128, 1) X(192, 1) X(256, 1) X(64, 2) X(128, 2) X(192, 2) X(256, 2) X(64, 8) X(128, 8) X(192, 8) X(256, 8)
#undef X
      return cudaErrorInvalidValue;
    };
    const cudaError_t e = score();
    if (e != cudaSuccess) return e;
    p.after_scores = 1;
  }
  p.key_space = std::min(std::max(p.max_blocks, 1), kSelectMostKeys);
  return p.max_blocks <= 2048 ? launch_select_of<256>(p, num_seqs, device, stream)
                              : launch_select_of<1024>(p, num_seqs, device, stream);
}

}  // namespace pkv
