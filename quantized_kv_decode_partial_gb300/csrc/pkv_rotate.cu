// Norm and rotation of queries and keys in one pass, alone or with the write of keys and
// values into their pages. The row arithmetic lives in pkv_rotate.cuh.
//
// A step's projections are read once and written once, so HBM bounds the large calls and the
// launch with its chain of dependent loads the small ones. Warps take (token, share of its
// heads): a token's angles are computed once and turn every head of the share. Few tokens are
// spread over many warps, many tokens take all their heads in one warp each.
//
// Pages of bf16 rows get keys and values straight from registers; affine pages go row by row
// through the append's own quantiser (pkv_append.cuh), from shared memory. e4m3 pages have
// one scale per block, which needs the largest of the block's new values before the first code
// is written: there CTAs take (touched block, plane, a few KV heads), hold the rows in
// registers between the two uses and share the block's angles through shared memory.
#include <type_traits>

#include "pkv_append.cuh"
#include "pkv_e4m3.cuh"
#include "pkv_launch.h"
#include "pkv_rotate.cuh"

namespace pkv {

namespace {

constexpr int kPlain = 0;  // FMT of the kernel without the write

constexpr int kTokenBatch = 4;  // rows a lane has in flight
constexpr int kBlockHold = 8;   // row batches a lane of the block path keeps in registers
constexpr int kTableBytes = 40 << 10;  // of the 48 KB that a launch may have unasked

template <int FMT>
constexpr int kWarps = FMT == kFmtE4m3 ? 8 : 4;

// A new row's sequence and place.
struct TokenPlace {
  int seq, index;    // its sequence, and which of that one's new rows it is
  int count;         // new rows of the sequence
  bool in_sequence;  // false: a row of no sequence
};

__device__ __forceinline__ TokenPlace place_of(const RotateParams& p, int t) {
  TokenPlace at;
  if (p.tokens_per_seq > 0) {
    at.seq = t / p.tokens_per_seq;
    at.index = t - at.seq * p.tokens_per_seq;
    at.count = p.tokens_per_seq;
    at.in_sequence = true;
  } else {
    at.seq = find_last(p.num_seqs, t, [&](int b) { return p.query_starts[b]; });
    const int start = p.query_starts[at.seq], end = p.query_starts[at.seq + 1];
    at.index = t - start;
    at.count = end - start;
    at.in_sequence = start >= 0 && t >= start && t < end && end <= p.tokens;
  }
  return at;
}

__device__ __forceinline__ long long row_base(const HeadRows& r, const RotateParams& p, int t) {
  if (p.tokens_per_seq == 0) return t * r.token;
  const int b = t / p.tokens_per_seq;
  return b * r.seq + (t - b * p.tokens_per_seq) * r.token;
}

// A lane's eight norm weights (ones where the row has no norm).
__device__ __forceinline__ void lane_weights(const RotateParams& p, const void* weight, bool used, int off0, int off1,
                                             float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (weight && used) {
    load_weight4(weight, p.weight_f32, off0, p.weight_offset, w);
    load_weight4(weight, p.weight_f32, off1, p.weight_offset, w + 4);
  }
}

// cos and sin of a lane's four pairs at token t.
__device__ __forceinline__ void lane_angles(const RotateParams& p, int u, int t, int cache_place, float (&cs)[4],
                                            float (&sn)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = u * 4 + i;
    const int pos =
        p.positions ? p.positions[static_cast<long long>(axis_of(p.turn, f)) * p.tokens + t] : cache_place;
    turn_at(turn_step(p.inv_freq[f]), pos, p.turn.amplitude, cs[i], sn[i]);
  }
}

// One warp: share g of token t's rows. With pages, D and DV are theirs.
template <int D, int DV, int FMT>
__device__ __forceinline__ void token_rows(const RotateParams& p, int t, int g, __nv_bfloat16* stage) {
  using L = RowLanes<D>;
  const int lane = threadIdx.x & 31;
  const int sub = lane / L::kLanes, u = lane % L::kLanes;
  const bool used = u < L::kUsed;
  int off0, off1;
  run_offsets(p.turn, u, off0, off1);
  const int HQ = p.num_q_heads, HK = p.num_kv_heads;
  // keys that leave through registers join the queries' rows
  constexpr bool kKeysHere = FMT == kPlain || FMT == 16;
  const int rows = HQ + (kKeysHere ? HK : 0);
  const int slots = (rows + L::kRows - 1) / L::kRows;
  const __nv_bfloat16* q_src = p.q.data + row_base(p.q, p, t);
  const __nv_bfloat16* k_src = (FMT == kPlain && HK == 0) ? nullptr : p.k.data + row_base(p.k, p, t);

  uint2 a[kTokenBatch], b[kTokenBatch];
  auto load = [&](int s0) {
#pragma unroll
    for (int j = 0; j < kTokenBatch; ++j) {
      const int r = (s0 + j * p.groups) * L::kRows + sub;
      a[j] = b[j] = make_uint2(0u, 0u);
      if (used && r < rows) {
        const __nv_bfloat16* src = r < HQ ? q_src + r * p.q.head : k_src + (r - HQ) * p.k.head;
        a[j] = ld_nc_keep_v2(src + off0);
        b[j] = ld_nc_keep_v2(src + off1);
      }
    }
  };
  load(g);

  float wq[8], wk[8], cs[4], sn[4];
  lane_weights(p, p.q_weight, used, off0, off1, wq);
  lane_weights(p, p.k_weight, used, off0, off1, wk);

  // where the keys go
  TokenPlace at{};
  int phys = -1, offset = 0, cache_place = 0;
  if constexpr (FMT != kPlain) {
    at = place_of(p, t);
    if (!at.in_sequence) return;
    const int len = p.seq_lens[at.seq];
    cache_place = static_cast<int>(static_cast<unsigned>(len) + static_cast<unsigned>(at.index));
    if (FMT != kFmtE4m3) {
      const long long end = static_cast<long long>(len) + at.count;
      if (len < 0 || end > static_cast<long long>(p.max_blocks) * p.block_size) {
        if (lane == 0 && g == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadSeqLen);
      } else {
        const int blk = cache_place / p.block_size;
        offset = cache_place - blk * p.block_size;
        phys = p.block_tables[static_cast<size_t>(at.seq) * p.max_blocks + blk];
        if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
          if (lane == 0 && g == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
          phys = -1;
        }
      }
    }
  }
  const bool turned = u * 8 < p.turn.rot;
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = sn[i] = 0.f;
  if (turned) lane_angles(p, u, t, cache_place, cs, sn);

  const bool any_norm = p.q_weight || p.k_weight;
  const long long q_to = row_base(p.q_out, p, t);
  const long long k_to = FMT == kPlain && HK > 0 ? row_base(p.k_out, p, t) : 0;
  auto pool_row = [&](int h) { return (static_cast<size_t>(phys) * HK + h) * p.block_size + offset; };
  for (int s0 = g; s0 < slots; s0 += kTokenBatch * p.groups) {
    if (s0 != g) load(s0);
#pragma unroll
    for (int j = 0; j < kTokenBatch; ++j) {
      const int s = s0 + j * p.groups;
      if (s >= slots) break;
      const int r = s * L::kRows + sub;
      const bool key = r >= HQ;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = key ? wk[i] : wq[i];
      turn_row<D>(a[j], b[j], any_norm, (key ? p.k_weight : p.q_weight) != nullptr, w, p.eps, turned, p.turn.adjacent,
                  cs, sn);
      if (!used || r >= rows) continue;
      __nv_bfloat16* to;
      if (!key) {
        to = p.q_out.data + q_to + r * p.q_out.head;
      } else if constexpr (FMT == kPlain) {
        to = p.k_out.data + k_to + (r - HQ) * p.k_out.head;
      } else {
        if (phys < 0) continue;
        to = p.dst.k_pool_bf16 + pool_row(r - HQ) * D;
      }
      *reinterpret_cast<uint2*>(to + off0) = a[j];
      *reinterpret_cast<uint2*>(to + off1) = b[j];
    }
  }

  if constexpr (FMT == 16) {
    if (phys < 0) return;
    const __nv_bfloat16* v_src = p.v.data + row_base(p.v, p, t);
    constexpr int kChunks = DV / 8;
    for (int c = g * 32 + lane; c < HK * kChunks; c += p.groups * 32) {
      const int h = c / kChunks, at8 = (c % kChunks) * 8;
      *reinterpret_cast<uint4*>(p.dst.v_pool_bf16 + pool_row(h) * DV + at8) = ld_nc_keep_v4(v_src + h * p.v.head + at8);
    }
  }
  if constexpr (FMT == 4 || FMT == 8) {
    if (phys < 0) return;
    const __nv_bfloat16* v_src = p.v.data + row_base(p.v, p, t);
    for (int h0 = g * L::kRows; h0 < HK; h0 += p.groups * L::kRows) {
      const int h = h0 + sub;
      uint2 x = make_uint2(0u, 0u), y = x;
      if (used && h < HK) {
        x = ld_nc_keep_v2(k_src + h * p.k.head + off0);
        y = ld_nc_keep_v2(k_src + h * p.k.head + off1);
      }
      turn_row<D>(x, y, any_norm, p.k_weight != nullptr, wk, p.eps, turned, p.turn.adjacent, cs, sn);
      __syncwarp();  // the rows staged before have been read
      if (used) {
        *reinterpret_cast<uint2*>(stage + sub * D + off0) = x;
        *reinterpret_cast<uint2*>(stage + sub * D + off1) = y;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < L::kRows; ++i) {
        if (h0 + i >= HK) break;
        const size_t row = pool_row(h0 + i);
        append_plane<FMT, D>(stage + i * D, nullptr, p.dst.k_pool_words, p.dst.k_scales, p.dst.k_biases, row, lane);
        append_plane<FMT, DV>(v_src + (h0 + i) * p.v.head, nullptr, p.dst.v_pool_words, p.dst.v_scales, p.dst.v_biases,
                              row, lane);
      }
    }
  }
}

// One CTA: the new rows of one touched block, in one plane of the KV heads from h0 on. TURN: keys
// (normed and rotated), else values.
template <int D, bool TURN>
__device__ __forceinline__ void block_rows(const RotateParams& p, int slot, int h0, float2* table, uint32_t* red) {
  using L = RowLanes<D>;
  constexpr int kPlane = TURN ? 0 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = p.block_size;
  // Sequence b's blocks have the slots from floor(start_b / bs) + 2 b on: n rows touch at most
  // floor(n / bs) + 2 blocks, which is what its share holds.
  auto start_of = [&](int b) { return p.tokens_per_seq > 0 ? b * p.tokens_per_seq : p.query_starts[b]; };
  const int seq = find_last(p.num_seqs, slot, [&](int b) { return static_cast<long long>(start_of(b) / bs) + 2ll * b; });
  const int start = start_of(seq);
  const int n = p.tokens_per_seq > 0 ? p.tokens_per_seq : p.query_starts[seq + 1] - start;
  const long long t = slot - (static_cast<long long>(start / bs) + 2ll * seq);
  if (start < 0 || n <= 0 || t < 0 || static_cast<long long>(start) + n > p.tokens) {
    // starts that fall or leave the tokens: nothing is written
    if (threadIdx.x == 0 && p.error_flag && (n < 0 || start < 0 || static_cast<long long>(start) + n > p.tokens))
      atomicOr(p.error_flag, kDevErrBadSeqLen);
    return;
  }
  const int len = p.seq_lens[seq];
  const long long end = static_cast<long long>(len) + n;
  if (len < 0 || end > static_cast<long long>(p.max_blocks) * bs) {
    if (threadIdx.x == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadSeqLen);
    return;
  }
  const long long blk = len / bs + t;
  const long long first = blk * bs;  // the block's first position
  if (first >= end) return;
  const int r0 = first < len ? static_cast<int>(len - first) : 0;  // its first new row
  const int r1 = static_cast<int>(min(end - first, static_cast<long long>(bs)));
  const int j0 = static_cast<int>(first + r0 - len);  // which of the sequence's new rows that is
  const int phys = p.block_tables[static_cast<size_t>(seq) * p.max_blocks + blk];
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
    if (threadIdx.x == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
    return;
  }

  const int sub = lane / L::kLanes, u = lane % L::kLanes;
  const bool used = u < L::kUsed;
  int off0 = u * 8, off1 = u * 8 + 4;
  if (TURN) run_offsets(p.turn, u, off0, off1);
  const bool turned = TURN && u * 8 < p.turn.rot;
  const int per_head = p.head_warps;
  const int h = h0 + warp / per_head, part = warp % per_head;
  const bool live = h < p.num_kv_heads;
  const HeadRows& in = TURN ? p.k : p.v;
  const __nv_bfloat16* src = in.data +
                             (p.tokens_per_seq > 0 ? seq * in.seq + j0 * in.token : (static_cast<long long>(start) + j0) * in.token) +
                             static_cast<long long>(h) * in.head;
  const int row_step = per_head * L::kRows;
  const int row0 = r0 + part * L::kRows + sub;

  uint2 a[kBlockHold], b[kBlockHold];
#pragma unroll
  for (int k = 0; k < kBlockHold; ++k) {
    const int r = row0 + k * row_step;
    a[k] = b[k] = make_uint2(0u, 0u);
    if (live && used && r < r1) {
      const __nv_bfloat16* row = src + (r - r0) * in.token;
      a[k] = ld_nc_keep_v2(row + off0);
      b[k] = ld_nc_keep_v2(row + off1);
    }
  }
  float w[8];
  const int tabled = min(p.table_rows, r1 - r0), half = p.turn.rot / 2;
  if (TURN) {
    lane_weights(p, p.k_weight, used, off0, off1, w);
    for (int i = threadIdx.x; i < tabled * half; i += blockDim.x) {
      const int r = i / half, f = i - r * half;
      const int token = start + j0 + r;
      const int pos = p.positions ? p.positions[static_cast<long long>(axis_of(p.turn, f)) * p.tokens + token]
                                  : len + j0 + r;
      float c, s;
      turn_at(turn_step(p.inv_freq[f]), pos, p.turn.amplitude, c, s);
      table[i] = make_float2(c, s);
    }
    __syncthreads();
  }
  auto finish = [&](uint2& x, uint2& y, int r) {
    if constexpr (TURN) {
      float cs[4] = {0.f, 0.f, 0.f, 0.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
      if (turned && r < r1) {
        if (r - r0 < tabled) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = table[(r - r0) * half + u * 4 + i];
            cs[i] = v.x;
            sn[i] = v.y;
          }
        } else {
          lane_angles(p, u, start + j0 + r - r0, len + j0 + r - r0, cs, sn);
        }
      }
      turn_row<D>(x, y, p.k_weight != nullptr, p.k_weight != nullptr, w, p.eps, turned, p.turn.adjacent, cs, sn);
    }
  };
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < kBlockHold; ++k) {
    if (r0 + k * row_step >= r1) break;  // of every warp of the CTA
    finish(a[k], b[k], row0 + k * row_step);
    m = max_abs(m, make_uint4(a[k].x, a[k].y, b[k].x, b[k].y));
  }
  // rows beyond those that registers hold are computed twice
  auto later = [&](auto&& use) {
    for (int k = kBlockHold; r0 + k * row_step < r1; ++k) {
      const int r = row0 + k * row_step;
      uint2 x = make_uint2(0u, 0u), y = x;
      if (live && used && r < r1) {
        x = ld_nc_keep_v2(src + (r - r0) * in.token + off0);
        y = ld_nc_keep_v2(src + (r - r0) * in.token + off1);
      }
      finish(x, y, r);
      use(x, y, r);
    }
  };
  later([&](const uint2& x, const uint2& y, int) { m = max_abs(m, make_uint4(x.x, x.y, y.x, y.y)); });
  m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
  const size_t cell = static_cast<size_t>(phys) * p.num_kv_heads + h;
  const float old = live && r0 > 0 ? p.block_scales[kPlane][cell] : 0.f;
  if (lane == 0) red[warp] = m;
  __syncthreads();  // (and every warp has read the old scale)
  for (int i = 0; i < per_head; ++i) m = max(m, red[warp / per_head * per_head + i]);
  if (!live) return;
  const float need = pow2_scale(__uint_as_float(m << 16));
  const float s = fmaxf(old, need);
  uint8_t* block = p.block_pool[kPlane] + cell * bs * D;
  if (part == 0 && lane == 0) p.block_scales[kPlane][cell] = s;
  if (r0 > 0 && s > old) {  // the earlier rows' codes under the larger scale
    const float ratio = __fdiv_rn(old, s);
    uint2* words = reinterpret_cast<uint2*>(block);
    for (int i = part * 32 + lane; i < r0 * (D / 8); i += per_head * 32) {
      uint2 c = words[i];
      c.x = rescale4(c.x, ratio);
      c.y = rescale4(c.y, ratio);
      words[i] = c;
    }
  }
  const float inv = s > 0.f ? 1.f / s : 0.f;  // s = 0: every value is 0, and so is every code
  const float by = s > 0.f ? s : 1.f;
  auto write = [&](auto exact) {
    auto put = [&](const uint2& x, const uint2& y, int r) {
      const uint2 c = quantize8<decltype(exact)::value>(make_uint4(x.x, x.y, y.x, y.y), by, inv);
      if (used && r < r1) {
        *reinterpret_cast<uint32_t*>(block + static_cast<size_t>(r) * D + off0) = c.x;
        *reinterpret_cast<uint32_t*>(block + static_cast<size_t>(r) * D + off1) = c.y;
      }
    };
#pragma unroll
    for (int k = 0; k < kBlockHold; ++k) {
      if (r0 + k * row_step >= r1) break;
      put(a[k], b[k], row0 + k * row_step);
    }
    later(put);
  };
  if ((__float_as_uint(s) & 0x7FFFFFu) == 0u) {
    write(std::true_type{});
  } else {
    write(std::false_type{});
  }
}

template <int D, int DV, int FMT>
__global__ void __launch_bounds__(kWarps<FMT> * 32) pkv_rotate_kernel(const __grid_constant__ RotateParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint32_t red[kWarps<FMT>];
  wait_for_prerequisite_grids();
  if constexpr (FMT == kFmtE4m3) {
    if (blockIdx.x >= p.q_ctas) {
      const int heads = kWarps<FMT> / p.head_warps;
      const int head_groups = (p.num_kv_heads + heads - 1) / heads;
      const int unit = blockIdx.x - p.q_ctas;
      const int slot = unit / (2 * head_groups), rest = unit - slot * 2 * head_groups;
      float2* table = reinterpret_cast<float2*>(smem);
      if (rest & 1) {
        block_rows<DV, false>(p, slot, (rest >> 1) * heads, table, red);
      } else {
        block_rows<D, true>(p, slot, (rest >> 1) * heads, table, red);
      }
      return;
    }
  }
  const int warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps<FMT> + warp;
  const int t = static_cast<int>(unit / p.groups), g = static_cast<int>(unit - static_cast<long long>(t) * p.groups);
  if (t >= p.tokens) return;
  __nv_bfloat16* stage = reinterpret_cast<__nv_bfloat16*>(smem) + warp * RowLanes<D>::kRows * D;
  token_rows<D, DV, FMT>(p, t, g, stage);
}

// Warps per token: as many as fill the GPU, each with whole batches of rows where it has several.
int token_groups(long long tokens, int slots, int sm_count) {
  const long long want = 32ll * sm_count;
  long long groups = (want + tokens - 1) / tokens;
  groups = groups < 1 ? 1 : groups > slots ? slots : groups;
  int per = static_cast<int>((slots + groups - 1) / groups);
  if (per > kTokenBatch) per = (per + kTokenBatch - 1) / kTokenBatch * kTokenBatch;
  return (slots + per - 1) / per;
}

template <int D, int DV, int FMT>
cudaError_t launch_of(RotateParams p, int sm_count, cudaStream_t stream) {
  using L = RowLanes<D>;
  constexpr bool kKeysHere = FMT == kPlain || FMT == 16;
  const int rows = p.num_q_heads + (kKeysHere ? p.num_kv_heads : 0);
  p.groups = token_groups(p.tokens, (rows + L::kRows - 1) / L::kRows, sm_count);
  long long ctas = (static_cast<long long>(p.tokens) * p.groups + kWarps<FMT> - 1) / kWarps<FMT>;
  size_t smem = 0;
  if (FMT == 4 || FMT == 8) smem = kWarps<FMT> * L::kRows * D * 2;
  if (FMT == kFmtE4m3) {
    p.q_ctas = static_cast<int>(ctas);
    const int most = p.tokens_per_seq > 0 ? p.tokens_per_seq : p.tokens;
    const int held = most < p.block_size ? most : p.block_size;  // new rows of a block
    // Warps per KV head: enough that the block's rows stay in registers, and that few heads fill a CTA.
    const int batches = (held + L::kRows - 1) / L::kRows;
    p.head_warps = 1;
    while (p.head_warps < kWarps<FMT> &&
           (p.head_warps * kBlockHold < batches || 2 * p.head_warps * p.num_kv_heads <= kWarps<FMT>) &&
           p.head_warps < batches)
      p.head_warps *= 2;
    const int fit = kTableBytes / (p.turn.rot * 4);
    p.table_rows = held < fit ? held : fit;
    smem = static_cast<size_t>(p.table_rows) * p.turn.rot * 4;
    const int heads = kWarps<FMT> / p.head_warps;
    const long long head_groups = (p.num_kv_heads + heads - 1) / heads;
    ctas += (p.tokens / p.block_size + 2ll * p.num_seqs) * head_groups * 2;
  }
  if (ctas >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kWarps<FMT> * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits before it touches memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pkv_rotate_kernel<D, DV, FMT>, p);
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, int head_dim, int sm_count, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_of<64, 64, kPlain>(p, sm_count, stream);
    case 128: return launch_of<128, 128, kPlain>(p, sm_count, stream);
    case 192: return launch_of<192, 192, kPlain>(p, sm_count, stream);
    case 256: return launch_of<256, 256, kPlain>(p, sm_count, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_rotate_append(const RotateParams& p, int fmt, int head_dim, int v_head_dim, int sm_count,
                                 cudaStream_t stream) {
#define X(B_, DK_, DV_) \
  if (fmt == B_ && head_dim == DK_ && v_head_dim == DV_) return launch_of<DK_, DV_, B_>(p, sm_count, stream);
#define WIDE(B_) X(B_, 64, 64) X(B_, 128, 128) X(B_, 256, 256) X(B_, 192, 128) X(B_, 256, 128) X(B_, 128, 256)
#define AFFINE(B_) X(B_, 128, 128) X(B_, 256, 256) X(B_, 256, 128) X(B_, 128, 256)
  WIDE(16) WIDE(kFmtE4m3) AFFINE(4) AFFINE(8)
#undef AFFINE
#undef WIDE
#undef X
  return cudaErrorInvalidValue;
}

}  // namespace pkv
