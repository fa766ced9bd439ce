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
//
// Measured on a GB300, replayed graphs, against the bytes at the rate of a plain copy: 4 x 3001-5003 tokens, 28 + 4 heads
// of 128 dims, three axes: 50-52 us, 0.82-0.85 (with one unit of eight values per lane and trip instead of two: 56; the first form, a
// lane's values loaded when they were needed: 73). 2 x 4097-8191 tokens, 16 + 4 heads of 256 dims of which 64 turn: 55-57 us,
// 0.80-0.82. bf16 pages, 8 x 1025-4099 tokens: 96-97 us, 0.82; e4m3 pages, 8 x 2001-8192 tokens: 201-203 us, 0.71, with the
// queries' and the blocks' CTAs in one launch (in one each: 218). Affine pages, the prompts of the bf16 ones: 191 us with heads of
// 128 dims, 153 with half as many of 256, 0.36-0.48: rows go through the quantiser one after the other. One token: 2.9 us;
// one of each of 64 sequences with its write: 4.3, and 7.8 with cold caches, into affine pages 12.3.
#include <algorithm>
#include <type_traits>

#include "pkv_append.cuh"
#include "pkv_e4m3.cuh"
#include "pkv_launch.h"
#include "pkv_rotate.cuh"

namespace pkv {

namespace {

constexpr int kPlain = 0;  // FMT of the kernel without the write

constexpr int kRing = 4;        // slots (a warp's rows at once) in flight
constexpr int kSlotBytes = 1024;
constexpr int kWarpBytes = kRing * kSlotBytes + 128 * 8;  // ring and a token's angles
constexpr int kBlockHold = 8;   // row batches a lane of the block path keeps in registers
constexpr int kTableBytes = 36 << 10;  // of the 48 KB that a launch may have unasked

template <int FMT>
constexpr int kWarps = FMT == kFmtE4m3 ? 8 : 4;

// A new row's sequence and place.
struct TokenPlace {
  int seq, index;    // its sequence, and which of that one's new rows it is
  int count;         // new rows of the sequence
  int len;           // rows it held before
  bool in_sequence;  // false: a row of no sequence
};

constexpr int kPlaceRounds = 4;  // up to 32 * 4 sequences are looked through at once

// Starts and lengths of that many sequences, spread over a warp: one trip to memory instead of one after the other.
struct StartsAndLengths {
  int starts[kPlaceRounds], lens[kPlaceRounds], last;
  __device__ __forceinline__ explicit StartsAndLengths(const RotateParams& p) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kPlaceRounds; ++i) {
      const int b = i * 32 + lane;
      starts[i] = b < p.num_seqs ? p.query_starts[b] : 0;
      lens[i] = b < p.num_seqs ? p.seq_lens[b] : 0;
    }
    last = p.query_starts[p.num_seqs];
  }
  // Of sequence b: where it begins and ends, and its length.
  __device__ __forceinline__ void of(const RotateParams& p, int b, int& start, int& end, int& len) const {
    start = len = end = 0;
#pragma unroll
    for (int i = 0; i < kPlaceRounds; ++i) {
      const int s = __shfl_sync(0xffffffffu, starts[i], b & 31), l = __shfl_sync(0xffffffffu, lens[i], b & 31);
      const int e = __shfl_sync(0xffffffffu, starts[i], (b + 1) & 31);
      if (i == b / 32) {
        start = s;
        len = l;
      }
      if (i == (b + 1) / 32) end = e;
    }
    if (b + 1 == p.num_seqs) end = last;
  }
};

__device__ __forceinline__ TokenPlace place_of(const RotateParams& p, int t) {
  TokenPlace at;
  if (p.tokens_per_seq > 0) {
    at.seq = t / p.tokens_per_seq;
    at.index = t - at.seq * p.tokens_per_seq;
    at.count = p.tokens_per_seq;
    at.len = p.seq_lens[at.seq];
    at.in_sequence = true;
    return at;
  }
  int start, end;
  if (p.num_seqs <= 32 * kPlaceRounds) {
    const StartsAndLengths all(p);
    int count = 0;  // sequences that begin at or before t
#pragma unroll
    for (int i = 0; i < kPlaceRounds; ++i)
      count += __popc(__ballot_sync(0xffffffffu, i * 32 + (threadIdx.x & 31) < p.num_seqs && all.starts[i] <= t));
    at.seq = max(count - 1, 0);
    all.of(p, at.seq, start, end, at.len);
  } else {
    at.seq = find_last(p.num_seqs, t, [&](int b) { return p.query_starts[b]; });
    start = p.query_starts[at.seq];
    end = p.query_starts[at.seq + 1];
    at.len = p.seq_lens[at.seq];
  }
  at.index = t - start;
  at.count = end - start;
  at.in_sequence = start >= 0 && t >= start && t < end && end <= p.tokens;
  return at;
}

// A token's sequence and place where the rows are not packed: (0, t) else.
struct RowAt {
  int seq, token;
};
__device__ __forceinline__ RowAt row_at(const RotateParams& p, int t) {
  if (p.tokens_per_seq == 0 || p.num_seqs == 1) return {0, t};
  const int b = t / p.tokens_per_seq;
  return {b, t - b * p.tokens_per_seq};
}
__device__ __forceinline__ __nv_bfloat16* rows_of(const HeadRows& r, const RowAt& at) {
  return r.data + at.seq * r.seq + at.token * r.token;
}

// A lane's eight norm weights.
template <int D>
__device__ __forceinline__ void lane_weights(const RotateTables<D>& tab, bool key, bool used, int off0, int off1, float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (used) {
    const float4 a = *reinterpret_cast<const float4*>(&tab.weight[key][off0]);
    const float4 b = *reinterpret_cast<const float4*>(&tab.weight[key][off1]);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// cos and sin of a lane's four pairs at token t.
template <int D>
__device__ __forceinline__ void lane_angles(const RotateParams& p, const RotateTables<D>& tab, int u, int t, int cache_place,
                                            float (&cs)[4], float (&sn)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = u * 4 + i;
    const int pos = p.positions ? p.positions[static_cast<long long>(tab.axis[f]) * p.tokens + t] : cache_place;
    turn_at(tab.step[f], pos, p.turn.amplitude, cs[i], sn[i]);
  }
}

// One warp: cos and sin of every pair at token t, in shared memory.
template <int D>
__device__ __forceinline__ void token_angles(const RotateParams& p, const RotateTables<D>& tab, int t, int cache_place,
                                             float2* angles) {
  const int half = p.turn.rot / 2;
  for (int f = threadIdx.x & 31; f < half; f += 32) {
    const int pos = p.positions ? p.positions[static_cast<long long>(tab.axis[f]) * p.tokens + t] : cache_place;
    float2 v;
    turn_at(tab.step[f], pos, p.turn.amplitude, v.x, v.y);
    angles[f] = v;
  }
  __syncwarp();
}

// One warp: share g of token t's rows. With pages, D and DV are theirs. prepare(): called once the first rows are asked for.
template <int D, int DV, int FMT, bool SIMPLE, typename Prepare>
__device__ __forceinline__ void token_rows(const RotateParams& p, const RotateTables<D>& tab, int t, int g,
                                           unsigned char* ring_smem, float2* angles, __nv_bfloat16* stage, const Prepare& prepare) {
  using L = RowLanes<D>;
  constexpr int kRows = L::kRows2;
  const int lane = threadIdx.x & 31;
  const int sub = lane / L::kHalf, u = lane % L::kHalf;
  // the lane's units u and u + kHalf: whether they hold values, and where their runs are
  const bool used[2] = {true, L::kUsed == L::kLanes || u + L::kHalf < L::kUsed};
  int off0[2], off1[2];
  run_offsets(p.turn, u, off0[0], off1[0]);
  run_offsets(p.turn, u + L::kHalf, off0[1], off1[1]);
  const int HQ = p.num_q_heads, HK = p.num_kv_heads;
  // Keys that leave through registers follow the queries: slots of kRows rows, this share's every groups-th.
  constexpr bool kKeysHere = FMT == kPlain || FMT == 16;
  const int q_slots = (HQ + kRows - 1) / kRows, k_slots = kKeysHere ? (HK + kRows - 1) / kRows : 0;
  const int slots = q_slots + k_slots, G = p.groups;
  const RowAt row = row_at(p, t);
  const __nv_bfloat16* k_src = (FMT == kPlain && HK == 0) ? nullptr : rows_of(p.k, row);

  // Rows come through a ring in shared memory, kRing slots ahead: loads in flight without registers. Rows that do not
  // exist are asked for with no bytes, which leaves zeros.
  const uint32_t ring = smem_addr(ring_smem) + sub * (L::kLanes * 16);
  auto key_row = [&](const __nv_bfloat16* base, long long head, int s) { return base + ((s - q_slots) * kRows + sub) * head; };
  int ask_s = g;
  const __nv_bfloat16* ask_at =
      (g < q_slots ? rows_of(p.q, row) + (g * kRows + sub) * p.q.head : key_row(k_src, p.k.head, g)) + u * 8;
  long long ask_step = (g < q_slots ? p.q.head : p.k.head) * (G * kRows);
  int ask_left = (g < q_slots ? HQ : q_slots * kRows + HK) - (g * kRows + sub);
  auto ask = [&](uint32_t place) {
    if (ask_s >= slots) {
      cp_async_commit();
      return;
    }
    const bool there = ask_left > 0;
    const uint32_t to = ring + place + u * 16;
    cp_async_16_or_zeros(to, there ? ask_at : p.q.data, there);
    cp_async_16_or_zeros(to + L::kHalf * 16, there && used[1] ? ask_at + L::kHalf * 8 : p.q.data, there && used[1]);
    cp_async_commit();
    const bool was_query = ask_s < q_slots;
    ask_s += G;
    ask_left -= G * kRows;
    ask_at += ask_step;
    if (kKeysHere && was_query && ask_s >= q_slots) {
      ask_at = key_row(k_src, p.k.head, ask_s) + u * 8;
      ask_step = p.k.head * (G * kRows);
      ask_left = HK - ((ask_s - q_slots) * kRows + sub);
    }
  };
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) ask(i * kSlotBytes);
  prepare();

  // where the keys go
  TokenPlace at{};
  int phys = -1, offset = 0, cache_place = 0;
  if constexpr (FMT != kPlain) {
    at = place_of(p, t);
    if (!at.in_sequence) {
      cp_async_wait<0>();
      return;
    }
    const int len = at.len;
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
  const bool adjacent = p.turn.adjacent != 0;
  const bool turned[2] = {SIMPLE || u * 8 < p.turn.rot, SIMPLE || (u + L::kHalf) * 8 < p.turn.rot};
  token_angles(p, tab, t, cache_place, angles);
  bool key = g >= q_slots;
  LaneTurn turn[2];
  auto make_turns = [&] {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[8], cs[4] = {0.f, 0.f, 0.f, 0.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
      lane_weights(tab, key, used[i], off0[i], off1[i], w);
      if (turned[i] && used[i]) {
        const float4* at4 = reinterpret_cast<const float4*>(angles + (u + i * L::kHalf) * 4);
        const float4 x = at4[0], y = at4[1];
        cs[0] = x.x, sn[0] = x.y, cs[1] = x.z, sn[1] = x.w;
        cs[2] = y.x, sn[2] = y.y, cs[3] = y.z, sn[3] = y.w;
      }
      turn[i] = make_turn<SIMPLE>(w, cs, sn, turned[i], adjacent);
    }
  };
  make_turns();

  auto pool_row = [&](int h) { return (static_cast<size_t>(phys) * HK + h) * p.block_size + offset; };
  __nv_bfloat16* k_to = nullptr;
  long long k_head = 0;
  if constexpr (FMT == kPlain) {
    if (HK > 0) k_to = rows_of(p.k_out, row);
    k_head = p.k_out.head;
  } else if constexpr (FMT == 16) {
    if (phys >= 0) k_to = p.dst.k_pool_bf16 + pool_row(0) * D;
    k_head = static_cast<long long>(p.block_size) * D;
  }
  __nv_bfloat16* to = key ? (k_to ? k_to + ((g - q_slots) * kRows + sub) * k_head : nullptr)
                          : rows_of(p.q_out, row) + (g * kRows + sub) * p.q_out.head;
  long long to_step = (key ? k_head : p.q_out.head) * (G * kRows);
  int left = (key ? q_slots * kRows + HK : HQ) - (g * kRows + sub);  // rows of this kind from the lane's on
  bool normed = (key ? p.k_weight : p.q_weight) != nullptr;
  uint32_t place = 0;
  const int end = k_to ? slots : q_slots;  // keys without a place go nowhere
#pragma unroll 1
  for (int s = g; s < end; s += G) {
    if (kKeysHere && !key && s >= q_slots) {  // from here on keys
      key = true;
      make_turns();
      to = k_to + ((s - q_slots) * kRows + sub) * k_head;
      to_step = k_head * (G * kRows);
      left = HK - ((s - q_slots) * kRows + sub);
      normed = p.k_weight != nullptr;
    }
    cp_async_wait<kRing - 1>();
    __syncwarp();  // every lane's part of the slot is there
    uint2 a[2], b[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[i] = ld_shared_v2(ring + place + off0[i] * 2);
      b[i] = ld_shared_v2(ring + place + off1[i] * 2);
      if (!used[i]) a[i] = b[i] = make_uint2(0u, 0u);
    }
    __syncwarp();  // every lane has read the slot
    ask(place);
    place = (place + kSlotBytes) & (kRing * kSlotBytes - 1);
    turn_row2<D, SIMPLE>(a, b, normed, p.eps, turned, adjacent, turn);
    if (left > 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!used[i]) continue;
        *reinterpret_cast<uint2*>(to + off0[i]) = a[i];
        *reinterpret_cast<uint2*>(to + off1[i]) = b[i];
      }
    }
    to += to_step;
    left -= G * kRows;
  }
  cp_async_wait<0>();
  __syncwarp();  // the angles are the next token's

  if constexpr (FMT == 16) {
    if (phys < 0) return;
    const __nv_bfloat16* v_src = rows_of(p.v, row);
    constexpr int kChunks = DV / 8;
    for (int c = g * 32 + lane; c < HK * kChunks; c += G * 32) {
      const int h = c / kChunks, at8 = (c % kChunks) * 8;
      *reinterpret_cast<uint4*>(p.dst.v_pool_bf16 + pool_row(h) * DV + at8) = ld_keep_v4(v_src + h * p.v.head + at8);
    }
  }
  if constexpr (FMT == 4 || FMT == 8) {
    if (phys < 0) return;
    const __nv_bfloat16* v_src = rows_of(p.v, row);
    key = true;
    make_turns();
    for (int h0 = g * kRows; h0 < HK; h0 += G * kRows) {
      const int h = h0 + sub;
      uint2 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = b[i] = make_uint2(0u, 0u);
        if (used[i] && h < HK) {
          a[i] = ld_keep_v2(k_src + h * p.k.head + off0[i]);
          b[i] = ld_keep_v2(k_src + h * p.k.head + off1[i]);
        }
      }
      turn_row2<D, SIMPLE>(a, b, p.k_weight != nullptr, p.eps, turned, adjacent, turn);
      __syncwarp();  // the rows staged before have been read
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!used[i]) continue;
        *reinterpret_cast<uint2*>(stage + sub * D + off0[i]) = a[i];
        *reinterpret_cast<uint2*>(stage + sub * D + off1[i]) = b[i];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (h0 + i >= HK) break;
        const size_t to_row = pool_row(h0 + i);
        append_plane<FMT, D>(stage + i * D, nullptr, p.dst.k_pool_words, p.dst.k_scales, p.dst.k_biases, to_row, lane);
        append_plane<FMT, DV>(v_src + (h0 + i) * p.v.head, nullptr, p.dst.v_pool_words, p.dst.v_scales, p.dst.v_biases,
                              to_row, lane);
      }
    }
    __syncwarp();  // the stage is the next token's ring, the angles its angles
  }
}

// One CTA: the new rows of one touched block, in one plane of the KV heads from h0 on. TURN: keys
// (normed and rotated), else values.
template <int D, bool TURN, bool SIMPLE, typename Tables>
__device__ __forceinline__ void block_rows(const RotateParams& p, Tables& tab, int slot, int h0, float2* table, uint32_t* red) {
  using L = RowLanes<D>;
  constexpr int kPlane = TURN ? 0 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = p.block_size;
  // Sequence b's blocks have the slots from floor(start_b / bs) + 2 b on: n rows touch at most
  // floor(n / bs) + 2 blocks, which is what its share holds.
  TablesAhead<D> ahead;
  if constexpr (TURN) ahead.load(p);  // on their way while the block is found
  int seq, start, n, len;
  if (p.tokens_per_seq > 0 || p.num_seqs > 32 * kPlaceRounds) {
    auto start_of = [&](int b) { return p.tokens_per_seq > 0 ? b * p.tokens_per_seq : p.query_starts[b]; };
    seq = find_last(p.num_seqs, slot, [&](int b) { return static_cast<long long>(start_of(b) / bs) + 2ll * b; });
    start = start_of(seq);
    n = p.tokens_per_seq > 0 ? p.tokens_per_seq : p.query_starts[seq + 1] - start;
    len = p.seq_lens[seq];
  } else {
    const StartsAndLengths all(p);
    int count = 0;
#pragma unroll
    for (int i = 0; i < kPlaceRounds; ++i) {
      const int b = i * 32 + lane;
      count += __popc(__ballot_sync(0xffffffffu, b < p.num_seqs && static_cast<long long>(all.starts[i] / bs) + 2ll * b <= slot));
    }
    seq = max(count - 1, 0);
    int end;
    all.of(p, seq, start, end, len);
    n = end - start;
  }
  const long long t = slot - (static_cast<long long>(start / bs) + 2ll * seq);
  if (start < 0 || n <= 0 || t < 0 || static_cast<long long>(start) + n > p.tokens) {
    return;  // (starts that fall or leave the tokens are flagged elsewhere)
  }
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

  const int sub = lane / L::kLanes, u = lane % L::kLanes;
  const bool used = u < L::kUsed;
  int off0 = u * 8, off1 = u * 8 + 4;
  if (TURN) run_offsets(p.turn, u, off0, off1);
  const bool turned = TURN && (SIMPLE || u * 8 < p.turn.rot) && used;
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
      a[k] = ld_keep_v2(row + off0);
      b[k] = ld_keep_v2(row + off1);
    }
  }
  // the rows are in flight while the table's answer arrives
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
    if (threadIdx.x == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
    return;
  }
  const size_t cell = static_cast<size_t>(phys) * p.num_kv_heads + h;
  const float old = live && r0 > 0 ? p.block_scales[kPlane][cell] : 0.f;
  float w[8];
  const int tabled = min(p.table_rows, r1 - r0), half = p.turn.rot / 2;
  if constexpr (TURN) {
    ahead.store(tab, p);
    __syncthreads();
    lane_weights(tab, true, used, off0, off1, w);
    for (int i = threadIdx.x; i < tabled * half; i += blockDim.x) {
      const int r = i / half, f = i - r * half;
      const int token = start + j0 + r;
      const int pos =
          p.positions ? p.positions[static_cast<long long>(tab.axis[f]) * p.tokens + token] : len + j0 + r;
      float c, s;
      turn_at(tab.step[f], pos, p.turn.amplitude, c, s);
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
          lane_angles(p, tab, u, start + j0 + r - r0, len + j0 + r - r0, cs, sn);
        }
      }
      turn_row<D, SIMPLE>(x, y, p.k_weight != nullptr, p.eps, turned, p.turn.adjacent,
                          make_turn<SIMPLE>(w, cs, sn, turned, p.turn.adjacent));
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
        x = ld_keep_v2(src + (r - r0) * in.token + off0);
        y = ld_keep_v2(src + (r - r0) * in.token + off1);
      }
      finish(x, y, r);
      use(x, y, r);
    }
  };
  later([&](const uint2& x, const uint2& y, int) { m = max_abs(m, make_uint4(x.x, x.y, y.x, y.y)); });
  m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
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

template <int D, int DV, int FMT, bool SIMPLE>
__global__ void __launch_bounds__(kWarps<FMT> * 32, FMT == kFmtE4m3 ? 3 : 5) pkv_rotate_kernel(const __grid_constant__ RotateParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ RotateTables<D> tab;
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
        block_rows<DV, false, SIMPLE>(p, tab, slot, (rest >> 1) * heads, table, red);
      } else {
        block_rows<D, true, SIMPLE>(p, tab, slot, (rest >> 1) * heads, table, red);
      }
      return;
    }
  }
  const int warp = threadIdx.x >> 5;
  bool ready = false;
  TablesAhead<D> ahead;
  ahead.load(p);
  auto prepare = [&] {  // the tables, beside the first rows' way here
    if (ready) return;
    ahead.store(tab, p);
    __syncthreads();
    ready = true;
  };
  unsigned char* mine = smem + warp * kWarpBytes;  // staged rows of the affine write take the ring's place
  float2* angles = reinterpret_cast<float2*>(mine + kRing * kSlotBytes);
  const long long units = static_cast<long long>(p.tokens) * p.groups, step = static_cast<long long>(p.q_ctas) * kWarps<FMT>;
  for (long long unit = static_cast<long long>(blockIdx.x) * kWarps<FMT> + warp; unit < units; unit += step) {
    const int t = p.groups == 1 ? static_cast<int>(unit) : static_cast<int>(unit / p.groups);
    const int g = static_cast<int>(unit - static_cast<long long>(t) * p.groups);
    token_rows<D, DV, FMT, SIMPLE>(p, tab, t, g, mine, angles, reinterpret_cast<__nv_bfloat16*>(mine), prepare);
  }
  prepare();  // a warp without a token
  if (FMT != kPlain && p.tokens_per_seq == 0 && blockIdx.x == 0 && warp == 0)
    check_starts(p.query_starts, p.num_seqs, p.tokens, p.error_flag);
}

// Warps per token: as many as fill the GPU.
int token_groups(long long tokens, int slots, int sm_count) {
  const long long want = 32ll * sm_count;
  long long groups = (want + tokens - 1) / tokens;
  groups = groups < 1 ? 1 : groups > slots ? slots : groups;
  const int per = static_cast<int>((slots + groups - 1) / groups);
  return (slots + per - 1) / per;
}

template <int D, int DV, int FMT>
cudaError_t launch_of(RotateParams p, int sm_count, cudaStream_t stream) {
  using L = RowLanes<D>;
  constexpr bool kKeysHere = FMT == kPlain || FMT == 16;
  const int slots = (p.num_q_heads + L::kRows2 - 1) / L::kRows2 + (kKeysHere ? (p.num_kv_heads + L::kRows2 - 1) / L::kRows2 : 0);
  p.groups = token_groups(p.tokens, slots, sm_count);
  // One wave of CTAs, each of which fills its tables once and takes many tokens.
  const long long most_ctas = (FMT == kFmtE4m3 ? 3ll : 5ll) * sm_count;
  long long ctas = (static_cast<long long>(p.tokens) * p.groups + kWarps<FMT> - 1) / kWarps<FMT>;
  ctas = std::min(ctas, most_ctas);
  p.q_ctas = static_cast<int>(ctas);
  size_t smem = kWarps<FMT> * kWarpBytes;
  if (FMT == kFmtE4m3) {
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
    smem = std::max(smem, static_cast<size_t>(p.table_rows) * p.turn.rot * 4);
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
  return p.turn.rot == D && !p.turn.adjacent ? cudaLaunchKernelEx(&cfg, pkv_rotate_kernel<D, DV, FMT, true>, p)
                                             : cudaLaunchKernelEx(&cfg, pkv_rotate_kernel<D, DV, FMT, false>, p);
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
