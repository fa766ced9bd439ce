// Attention of many new tokens of each sequence over its paged cache: tcgen05 products with
// scores, weights and outputs in tensor memory.
//
// A CTA takes one KV head and up to NQ tiles of 128 query rows; a tile's rows are
// floor(128 / REP) consecutive tokens times the KV head's REP query heads, so that short
// chunks fill tiles and every key tile serves all of them. Keys pass in tiles of KT rows.
// One warp copies K and V tiles (TMA, one box per run of rows that lie in one block and 64
// dims), one warp issues the products, and a warpgroup per query tile (thread = query row) turns
// scores into weights:
//     S = Q K^T (tensor memory) -> p = 2^(c s - c m), written over S as bf16 -> O += P V
// with P read by the product from tensor memory and O never leaving it. The maximum m follows
// the scores only when they exceed it by more than 2^8 in weight, so O is rescaled rarely; f32
// sums and bf16 weights lose nothing by the factor. With two query tiles one tile's softmax runs
// beside the other's products; with one (dims of 256), its next scores are computed meanwhile.
//
// Few query rows over long caches: the key tiles of each CTA's rows are split over `splits`
// CTAs whose f32 states (O, m, l) are joined by a second kernel.
//
// Measured on a GB300: 8 prompts of 1025-8192 tokens, 8 KV heads of 4, 128 dims: 1.42-1.48 ms, 1255-1305 TFLOP/s of
// products, 0.66-0.69 of what a large library matrix product reaches alone; 2 chunks of 500-1024 tokens over 30011-60000 rows:
// 1310-1394 TFLOP/s. The prompts with heads of 64 dims, whose softmax is the same beside half the products: 720-726 TFLOP/s;
// 192 for keys, 128 for values: 954-989; 4 KV heads of 256: 1106-1116, 256 and 128: 1131-1146, 128 and 256: 897. e4m3 codes
// read directly, 16 x 1-16 tokens over 700-16000 rows: 500 us, 12 times the bytes' floor; a tile of keys takes a CTA 4 us. The
// step is bound by hand-overs between products and softmax (without any exponential, sum or maximum it takes 0.91 of its time)
// and by the power limit, under which the SM clock settles near 1.5 of 2.07 GHz. Two threads per row with a barrier
// between them took 1.14 times as long, weights handed over by halves 1.19 times. 37 tokens alone: 8.4 us.
#pragma once

#include "pkv_codes.cuh"
#include "pkv_rotate.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kPrefillRoom = 225 * 1024;  // for tiles: 227 KB less barriers and the alignment of the first tile

// Tiles of one instantiation. FMT: 16 (rows of 16-bit values) or kFmtE4m3.
template <int D, int DV, int FMT>
struct PrefillShape {
  static constexpr bool kCodes = FMT != 16;
  // Query tiles per CTA: two where tensor and shared memory hold both.
  static constexpr int kQ = DV == 256 || (kCodes && D == 256) ? 1 : 2;
  static constexpr int KT = D <= 128 && DV <= 128 ? 128 : 64;  // key rows per tile
  static constexpr int kQBytes = 128 * D * 2, kKBytes = KT * D * 2, kVBytes = KT * DV * 2;
  // e4m3 codes come in through a ring of quarter tiles, which six warps, in pairs, turn into bf16.
  static constexpr int kPairs = 3;
  static constexpr int kRawBytes = KT / 4 * (D > DV ? D : DV);
  // As many as fit beside two stages of K and V (up to 9), and of each of the three pairs as many as of the others: a slot is one
  // pair's alone. A pair that came upon another's slot could be two phases ahead of its barrier, whose parity then passes
  // although the codes are still on their way. (Eight slots and one more wait, for the release of the codes before: the same time.)
  static constexpr int kRawFit = (kPrefillRoom - kQ * kQBytes - 2 * (kKBytes + kVBytes)) / kRawBytes;
  static constexpr int kRawSlots = !kCodes ? 0 : (kRawFit > 9 ? 9 : kRawFit) / kPairs * kPairs;
  static constexpr int kThreads = kCodes ? 512 : 384;
  // Stages of K and of V: as many as fit (up to 4), K first. A K tile is asked for when the last product that
  // read its stage is done; with two stages that is five products ahead, a copy's latency at best.
  static constexpr int kRoom = kPrefillRoom - kQ * kQBytes - kRawSlots * kRawBytes;
  static constexpr int kVS = kRoom / (kKBytes + kVBytes) > 4 ? 4 : kRoom / (kKBytes + kVBytes);
  static constexpr int kKS = (kRoom - kVS * kVBytes) / kKBytes > 4 ? 4 : (kRoom - kVS * kVBytes) / kKBytes;
  static constexpr int kSmem = kQ * kQBytes + kKS * kKBytes + kVS * kVBytes + kRawSlots * kRawBytes + 1024;
  static constexpr int kTmemO = 2 * KT;  // columns: two score tiles, then the outputs
  static_assert(kTmemO + kQ * DV <= 512, "tensor memory");
  static_assert(kVS >= 2 && kKS >= 2 && (!kCodes || (kRawSlots >= 2 * kPairs && kRawSlots % kPairs == 0)) &&
                    kSmem <= kPrefillRoom + 1024 && kRawBytes % 128 == 0,
                "shared memory");
};

// Registers: softmax threads hold a row's scores. With 384 threads (two softmax warpgroups, one with the product
// and copy warps) 2 * 128 * 208 + 128 * 88 is what the block was launched with, 384 * 168; with 512 (a fourth of
// warps that convert codes) 2 * 128 * 192 + 2 * 128 * 64 = 512 * 128. The change stands inside the branches: before
// them it bounds both sides' registers.
template <bool CODES>
__device__ __forceinline__ void more_registers() {
  if constexpr (CODES) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  }
}
template <bool CODES>
__device__ __forceinline__ void fewer_registers() {
  if constexpr (CODES) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  }
}
constexpr int kPrefillStates = 512;   // tensor memory columns

// A work unit's place: computed by every warp from the same words.
struct PrefillUnit {
  int seq, head, split;
  int first;           // first token of the unit (packed), and its tokens
  int tokens;
  int position;        // cache place of the first token
  const int32_t* table;
  int dense;           // with values written beforehand: key t lies in block dense + t / 128
  bool live, valid;    // live: has tokens; valid: its sequence's lengths are
};

__device__ __forceinline__ PrefillUnit prefill_unit(const PrefillParams& p, int unit_tokens) {
  PrefillUnit u;
  int x = blockIdx.x;
  u.split = x % p.splits;
  x /= p.splits;
  u.head = x % p.num_kv_heads;
  // Later tiles of a sequence see more keys: they start first.
  const int slots = gridDim.x / (p.splits * p.num_kv_heads);
  const int slot = slots - 1 - x / p.num_kv_heads;
  // Sequence b's units have the slots from floor(start_b / unit) + b on, as many as it can need.
  const int b = find_last(p.num_seqs, slot,
                          [&](int i) { return static_cast<long long>(p.query_starts[i] / unit_tokens) + i; });
  const int start = p.query_starts[b];
  const long long n = static_cast<long long>(p.query_starts[b + 1]) - start;
  const long long first = (slot - (static_cast<long long>(start / unit_tokens) + b)) * unit_tokens;
  const int len = p.seq_lens[b];
  const bool starts_ok = start >= 0 && n >= 0 && start + n <= p.tokens;
  u.seq = b;
  u.live = starts_ok && first >= 0 && first < n;
  u.valid = u.live && len >= n && len <= static_cast<long long>(p.max_blocks) * p.block_size;
  u.first = u.live ? static_cast<int>(start + first) : 0;
  u.tokens = u.live ? static_cast<int>(min(n - first, static_cast<long long>(unit_tokens))) : 0;
  u.position = u.valid ? static_cast<int>(len - n + first) : 0;
  u.table = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  u.dense = u.valid ? p.values.base(b, start) - p.values.first_row(len, static_cast<int>(n), p.window) / kValueRows : 0;
  if (u.live && !u.valid && threadIdx.x == 0 && p.error_flag)
    atomicOr(p.error_flag, kDevErrBadSeqLen);
  return u;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// A row's KT scores.
template <int KT>
__device__ __forceinline__ void tmem_ld_tile(uint32_t addr, float (&s)[KT]) {
  uint32_t v[KT / 32][32];
#pragma unroll
  for (int h = 0; h < KT / 32; ++h) tmem_ld_32(addr + 32 * h, v[h]);
#pragma unroll
  for (int h = 0; h < KT / 32; ++h) {
    tmem_wait_ld(v[h]);
#pragma unroll
    for (int e = 0; e < 32; ++e) s[32 * h + e] = __uint_as_float(v[h][e]);
  }
}

template <int KT>
__device__ __forceinline__ float row_max(const float (&s)[KT]) {
  float top[8];
#pragma unroll
  for (int n = 0; n < 8; ++n) top[n] = fmaxf(s[n], s[8 + n]);
#pragma unroll
  for (int e = 16; e < KT; e += 16)
#pragma unroll
    for (int n = 0; n < 8; ++n) top[n] = max3(top[n], s[e + n], s[e + 8 + n]);
  return max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], top[5]), fmaxf(top[6], top[7]));
}

// s - m, where there is an m.
template <int KT>
__device__ __forceinline__ void subtract(float (&s)[KT], float m) {
  if (m == -INFINITY) return;
#pragma unroll
  for (int e = 0; e < KT; ++e) s[e] -= m;
}

// A row's weights 2^(c s - c m) as pairs of bf16 (or fp16), their f32 sums added to `sums`; returns the largest score.
// fp16 ends at 2^-24 (what is at most half of it is lost) and its steps are even below 2^-14, where a few keys can stand
// against a million small ones. There all weights, and so their sums, are 2^7 times as large: at most 2^15 with what
// the maximum may lag behind, and lost only below 2^-32 of the maximum's.
template <int KT, bool HALF>
__device__ __forceinline__ float weights(const float (&s)[KT], float c, float m, uint64_t (&sums)[2], uint32_t (&w)[KT / 2]) {
  constexpr float kUp = HALF ? 7.f : 0.f;
  const float mc = fabsf(m) < INFINITY ? m * c : 0.f;
  const uint64_t cc = pair(c, c), mm = pair(kUp - mc, kUp - mc);
#pragma unroll
  for (int e = 0; e < KT / 2; ++e) {
    float x, y;
    unpair(fma2(pair(s[2 * e], s[2 * e + 1]), cc, mm), x, y);
    x = fast_exp2(x);
    y = fast_exp2(y);
    sums[e & 1] = add2(sums[e & 1], pair(x, y));
    w[e] = HALF ? pack_f16x2(x, y) : pack_bf16x2(x, y);
  }
  return row_max<KT>(s);
}

// Half of a quarter tile of codes (a warp's part of two): rows [first, first + KT/4) of the tile, 16 values a lane
// at a time. Rows that nobody sees and those of pieces without their bit become zeros.
template <int D, int FMT, int KT>
__device__ __forceinline__ void convert_quarter(uint32_t to, uint32_t from, int part, int first, int seen_lo, int seen_hi,
                                                uint32_t bits, uint32_t scales, int piece_log2) {
  constexpr int kPerRow = D / 16, kChunks = KT / 4 * kPerRow;
  const int lane = threadIdx.x & 31;
  const bool whole = seen_lo <= first && seen_hi >= first + KT / 4 && bits == (1u << ((KT / 4) >> piece_log2)) - 1u;
  constexpr int kRounds = (kChunks + 63) / 64;
  uint4 v[kRounds];  // all loads first: one round's latency instead of every round's
  float scale[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int c = i * 64 + part * 32 + lane;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = 0.f;
    if (kChunks % 64 && c >= kChunks) break;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                 : "r"(from + c * 16)
                 : "memory");
    scale[i] = ld_shared_f32(scales + 4 * (c / kPerRow >> piece_log2));
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int c = i * 64 + part * 32 + lane;
    if (kChunks % 64 && c >= kChunks) break;
    const int r = c / kPerRow, col = c % kPerRow;
    uint32_t w[8];
    codes_to_values<FMT>(v[i], scale[i], 0.f, w);
    if (!whole && !(first + r >= seen_lo && first + r < seen_hi && (bits >> (r >> piece_log2) & 1))) {
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 0u;
    }
    // 16-byte places of the swizzled row; odd runs of 64 dims write their second one first, so that eight
    // lanes meet eight different groups of banks
    const int row = first + r;
    const uint32_t at = to + col / 4 * (KT * 128) + row * 128;
    const int k0 = col % 4 * 2, odd = col / 4 & 1;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int y = x ^ odd;
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((k0 + y) ^ (row & 7)) << 4)),
                   "r"(y ? w[4] : w[0]), "r"(y ? w[5] : w[1]), "r"(y ? w[6] : w[2]), "r"(y ? w[7] : w[3])
                   : "memory");
    }
  }
}

// A query row's results: bf16 outputs, or with splits its f32 state.
struct PrefillRow {
  bool live;
  size_t row;  // token * HQ + head
};

// tq, tk, tv: TMA descriptors of the queries ([64 dims][head][token][run of dims]) and of the pools'
// planes ([64 dims][row][run of dims]).
// HALF: K and V are fp16 values (PrefillParams.factors); queries become fp16 in shared memory, each row under a power of
// two of its own, and weights are fp16.
template <int D, int DV, int FMT, bool HALF>
__global__ void __launch_bounds__(PrefillShape<D, DV, FMT>::kThreads, 1)
    pkv_prefill_kernel(const __grid_constant__ PrefillParams p, const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using T = PrefillShape<D, DV, FMT>;
  constexpr int KT = T::KT, KS = T::kKS, VS = T::kVS, RS = T::kCodes ? T::kRawSlots : 1;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * (KS + VS + RS) + 9];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ uint32_t piece_bits[VS];
  __shared__ uint32_t unit_bits[RS];  // codes: a quarter tile's pieces, and their scales
  __shared__ float unit_scales[RS][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  wait_for_prerequisite_grids();
  if (blockIdx.x == 0 && warp == 0) check_starts(p.query_starts, p.num_seqs, p.tokens, p.error_flag);
  const int unit_tokens = T::kQ * p.tile_tokens;
  const PrefillUnit u = prefill_unit(p, unit_tokens);
  if (!u.live) return;
  const size_t all_rows = static_cast<size_t>(p.tokens) * p.num_q_heads;
  // The unit's row i: token i / rep, query head i % rep of the KV head.
  auto row_of = [&](int tile, int r) {
    const int token = r / p.rep, t = tile * p.tile_tokens + token;
    PrefillRow q;
    q.live = token < p.tile_tokens && t < u.tokens;
    q.row = (static_cast<size_t>(u.first) + t) * p.num_q_heads + u.head * p.rep + (r - token * p.rep);
    return q;
  };
  const int tiles_q = (u.tokens + p.tile_tokens - 1) / p.tile_tokens;  // 1 .. kQ
  // Keys that any row of the unit sees: [lo, hi).
  const int hi = u.position + u.tokens;
  const int lo = p.window > 0 ? max(0, u.position - p.window + 1) : 0;
  const int tile_lo = lo / KT, tile_n = (hi - 1) / KT + 1 - tile_lo;
  const int t0 = tile_lo + static_cast<int>(static_cast<long long>(tile_n) * u.split / p.splits);
  const int nt = u.valid ? tile_lo + static_cast<int>(static_cast<long long>(tile_n) * (u.split + 1) / p.splits) - t0 : 0;

  if (nt == 0) {  // nothing to see, or a bad length: zeros
    for (int i = threadIdx.x; i < tiles_q * 128; i += blockDim.x) {
      const PrefillRow q = row_of(i >> 7, i & 127);
      if (!q.live) continue;
      if (p.splits > 1) {
        float* ml = p.ws_ml + (u.split * all_rows + q.row) * 2;
        ml[0] = -INFINITY;
        ml[1] = 0.f;
      } else {
        uint4* o = reinterpret_cast<uint4*>(p.out + q.row * DV);
        for (int d = 0; d < DV / 8; ++d) o[d] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    return;
  }

  const uint32_t smem = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t smem_k = smem + T::kQ * T::kQBytes, smem_v = smem_k + KS * T::kKBytes;
  const uint32_t smem_raw_codes = smem_v + VS * T::kVBytes;
  const uint32_t bar0 = smem_addr(bars);
  auto k_full = [&](int s) { return bar0 + 8 * s; };
  auto k_empty = [&](int s) { return bar0 + 8 * (KS + s); };
  auto v_full = [&](int s) { return bar0 + 8 * (2 * KS + s); };
  auto v_empty = [&](int s) { return bar0 + 8 * (2 * KS + VS + s); };
  auto raw_full = [&](int s) { return bar0 + 8 * (2 * KS + 2 * VS + s); };
  auto raw_empty = [&](int s) { return bar0 + 8 * (2 * KS + 2 * VS + RS + s); };
  constexpr int kRest = 2 * (KS + VS + RS);
  auto s_full = [&](int s) { return bar0 + 8 * (kRest + s); };
  auto p_full = [&](int s) { return bar0 + 8 * (kRest + 2 + s); };
  auto o_done = [&](int s) { return bar0 + 8 * (kRest + 4 + s); };
  const uint32_t q_full = bar0 + 8 * (kRest + 6), drained = bar0 + 8 * (kRest + 7), q_half = bar0 + 8 * (kRest + 8);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRest + 9; ++i) {
      int arrivals = 1;
      if (i == kRest + 2 || i == kRest + 3) arrivals = 4;  // p_full: the four warps of a query tile
      if (i == kRest + 8) arrivals = 4 * tiles_q;           // q_half
      if (T::kCodes) {                                     // two warps for each quarter of a tile
        if (i < KS || (i >= 2 * KS && i < 2 * KS + VS)) arrivals = 8;
        if (i >= 2 * (KS + VS) + RS && i < kRest) arrivals = 2;
      }
      mbar_init(bar0 + 8 * i, arrivals);
    }
    fence_barrier_init();
    abort_flag = 0;
  }
  if (warp == 8) tmem_alloc(smem_addr(&tmem_slot), kPrefillStates);
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const int piece = 1 << p.piece_log2, pieces = KT >> p.piece_log2;
  const int items = nt * tiles_q;  // item i: query tile i % tiles_q, key tile t0 + i / tiles_q, score tile i & 1
  // The pieces of key tile t that are copied, and (lane l) the row of piece l in the pool or among the values.
  auto tile_pieces = [&](int t, int& row) {
    const int key = t * KT + lane * piece;
    bool ok = lane < pieces && key < hi && key + piece > lo;
    row = 0;
    if (ok && p.values.used) {
      row = ((u.dense + key / kValueRows) * p.num_kv_heads + u.head) * kValueRows + key % kValueRows;
    } else if (ok) {
      const int blk = key / p.block_size;
      const int phys = static_cast<int>(ld_keep_u32(u.table + blk));
      ok = static_cast<unsigned>(phys) < static_cast<unsigned>(p.num_blocks);
      row = ok ? (phys * p.num_kv_heads + u.head) * p.block_size + (key - blk * p.block_size) : 0;
    }
    return __ballot_sync(0xffffffffu, ok);
  };
  // Of 32 keys from `key` on, those whose block is in the pool (asked where some block is not).
  auto good_keys = [&](int key) {
    const int blk = min(key + lane, hi - 1) / p.block_size;
    const bool ok = static_cast<unsigned>(u.table[blk]) < static_cast<unsigned>(p.num_blocks);
    return __ballot_sync(0xffffffffu, ok);
  };

  // Asks for the query tiles (one lane).
  auto ask_queries = [&] {
    mbar_arrive_expect_tx(q_full, tiles_q * (D / 64) * p.tile_tokens * p.rep * 128);
    for (int t = 0; t < tiles_q; ++t)
      for (int c = 0; c < D / 64; ++c)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem + t * T::kQBytes + c * 128 * 128),
            "l"(reinterpret_cast<uint64_t>(&tq)), "r"(0), "r"(u.head * p.rep), "r"(u.first + t * p.tile_tokens), "r"(c),
            "r"(q_full)
            : "memory");
  };
  if (!T::kCodes && (warp == 9 || warp == 10)) {
    // ------------------------------------------------------------------ copies: Q and K, and V
    fewer_registers<T::kCodes>();
    const bool is_k = warp == 9;
    if (is_k && lane == 0) ask_queries();
    const int stages = is_k ? KS : VS, runs = is_k ? D / 64 : DV / 64, bytes = is_k ? T::kKBytes : T::kVBytes;
    const uint32_t base = is_k ? smem_k : smem_v, full0 = is_k ? k_full(0) : v_full(0), empty0 = is_k ? k_empty(0) : v_empty(0);
    const uint64_t map = reinterpret_cast<uint64_t>(is_k ? &tk : &tv);
    int row, asked = 0;
    uint32_t bits = tile_pieces(t0, row);
    for (int j = 0; j < nt; ++j) {
      const int s = j % stages;
      int next_row = 0;
      uint32_t next_bits = 0;
      if (j + 1 < nt) next_bits = tile_pieces(t0 + j + 1, next_row);  // before the wait: its table words take a while
      if (j >= stages && !mbar_wait_close(empty0 + 8 * s, (j / stages - 1) & 1, &abort_flag, p.error_flag, p.wait_limit_ns))
        break;
      if (lane == 0) {
        if (!is_k) piece_bits[s] = bits;
        mbar_arrive_expect_tx(full0 + 8 * s, __popc(bits) * runs * piece * 128);
      }
      __syncwarp();
      for (int i0 = 0; i0 < pieces * runs; i0 += 32) {
        const int i = i0 + lane;
        const int pc = i % pieces, c = i / pieces;
        const int y = __shfl_sync(0xffffffffu, row, pc);
        if (i < pieces * runs && (bits >> pc & 1))
          asm volatile(
              "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
              "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(base + s * bytes + c * (KT * 128) + pc * piece * 128),
              "l"(map), "r"(0), "r"(y), "r"(c), "r"(full0 + 8 * s)
              : "memory");
      }
      __syncwarp();
      ++asked;
      row = next_row;
      bits = next_bits;
    }
    // Every copy lands before the CTA ends, whatever the other warps did.
    int none = 0;
    if (is_k) mbar_wait_close(q_full, 0, &none, p.error_flag, kWaitLimitNs);
    for (int i = max(0, asked - stages); i < asked; ++i)
      mbar_wait_close(full0 + 8 * (i % stages), (i / stages) & 1, &none, p.error_flag, kWaitLimitNs);
  } else if (T::kCodes && warp >= 9) {
    // ------------------------------------------------------------------ e4m3 codes, to bf16 tiles
    // Quarter tiles in the order K(0), K(1), V(0), K(2), V(1), ...: unit n is quarter n & 3 of plane tile n / 4. Warp 9
    // copies their codes, RS units ahead; pairs of warps turn them into bf16 in turn.
    fewer_registers<T::kCodes>();
    if constexpr (T::kCodes) {
      constexpr int kQuarter = KT / 4;
      auto plane_tile = [&](int x, bool& is_k, int& j) {
        if (nt == 1) {
          is_k = x == 0;
          j = 0;
        } else if (x <= 1) {
          is_k = true;
          j = x;
        } else {
          is_k = (x & 1) && (x + 1) / 2 < nt;
          j = is_k ? (x + 1) / 2 : (x & 1) ? nt - 1 : x / 2 - 1;
        }
      };
      if (warp == 9) {
        if (lane == 0) ask_queries();
        const int per = kQuarter >> p.piece_log2;  // pieces of a quarter
        bool is_k, ok = true;
        int j, row, asked = 0;
        plane_tile(0, is_k, j);
        uint32_t bits = tile_pieces(t0 + j, row);
        for (int x = 0; ok && x < 2 * nt; ++x) {
          float scale = 0.f;
          if (bits >> lane & 1) scale = (is_k ? p.k_scales : p.v_scales)[row / p.block_size];
          bool next_k = false;
          int next_j = 0, next_row = 0;
          uint32_t next_bits = 0;
          if (x + 1 < 2 * nt) {  // its table words arrive before this one's copies wait
            plane_tile(x + 1, next_k, next_j);
            next_bits = tile_pieces(t0 + next_j, next_row);
          }
          const int row_bytes = is_k ? D : DV;
          for (int h = 0; h < 4; ++h) {
            const int n = 4 * x + h, s = n % RS, first = h * per;
            if (n >= RS) ok = mbar_wait_close(raw_empty(s), (n / RS - 1) & 1, &abort_flag, p.error_flag, p.wait_limit_ns);
            if (!ok) break;
            const uint32_t mine = bits >> first & ((1u << per) - 1u);
            const bool copies = lane >= first && lane < first + per;
            if (copies) unit_scales[s][lane - first] = scale;
            __syncwarp();
            if (lane == 0) {
              unit_bits[s] = mine;
              mbar_arrive_expect_tx(raw_full(s), __popc(mine) * piece * row_bytes);
            }
            __syncwarp();
            if (copies && (bits >> lane & 1))
              asm volatile(
                  "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                  "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_raw_codes + s * T::kRawBytes + (lane - first) * piece * row_bytes),
                  "l"(reinterpret_cast<uint64_t>(is_k ? &tk : &tv)), "r"(0), "r"(row), "r"(raw_full(s))
                  : "memory");
            __syncwarp();
            ++asked;
          }
          is_k = next_k;
          j = next_j;
          row = next_row;
          bits = next_bits;
        }
        int none = 0;  // every copy lands before the CTA ends
        mbar_wait_close(q_full, 0, &none, p.error_flag, kWaitLimitNs);
        for (int n = max(0, asked - RS); n < asked; ++n)
          mbar_wait_close(raw_full(n % RS), (n / RS) & 1, &none, p.error_flag, kWaitLimitNs);
      } else {
        const int group = (warp - 10) >> 1, part = (warp - 10) & 1;
        for (int n = group; n < 8 * nt; n += T::kPairs) {
          bool is_k;
          int j;
          plane_tile(n >> 2, is_k, j);
          const int s = n % RS, stage = is_k ? j % KS : j % VS, round = is_k ? j / KS : j / VS;
          if (round > 0 && !mbar_wait_close(is_k ? k_empty(stage) : v_empty(stage), (round - 1) & 1, &abort_flag, p.error_flag,
                                           p.wait_limit_ns))
            break;
          if (!mbar_wait_close(raw_full(s), (n / RS) & 1, &abort_flag, p.error_flag, p.wait_limit_ns)) break;
          const uint32_t from = smem_raw_codes + s * T::kRawBytes, scales = smem_addr(unit_scales[s]);
          const int key = (t0 + j) * KT, first = (n & 3) * kQuarter;
          if (is_k) {
            convert_quarter<D, FMT, KT>(smem_k + stage * T::kKBytes, from, part, first, lo - key, hi - key, unit_bits[s], scales,
                                        p.piece_log2);
          } else {
            convert_quarter<DV, FMT, KT>(smem_v + stage * T::kVBytes, from, part, first, lo - key, hi - key, unit_bits[s], scales,
                                         p.piece_log2);
          }
          fence_proxy_async_smem();  // the tile's rows are there for the products
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(is_k ? k_full(stage) : v_full(stage));
            mbar_arrive(raw_empty(s));
          }
        }
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ products
    fewer_registers<T::kCodes>();
    const uint32_t leader = elect_lane(), base = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t instr_s = umma_instr(KT, false, p.negate != 0, HALF), instr_o = umma_instr(DV, true, false, HALF);
    bool ok = mbar_wait_close(HALF ? q_half : q_full, 0, &abort_flag, p.error_flag, p.wait_limit_ns);
    // Item i's query tile and key tile are counted along; a stage's index and parity follow its ring.
    struct Place {
      int q, tile, stage, parity;
    } sp{0, 0, 0, 0}, op{0, 0, 0, 0};  // of the scores and of the outputs that come next
    auto next = [&](Place& x, int stages) {
      if (++x.q < tiles_q) return;
      x.q = 0;
      ++x.tile;
      if (++x.stage == stages) {
        x.stage = 0;
        x.parity ^= 1;
      }
    };
    auto scores = [&](int slot) {
      const int s = sp.stage;
      if (sp.q == 0) ok = mbar_wait_close(k_full(s), sp.parity, &abort_flag, p.error_flag, p.wait_limit_ns);
      if (!ok) return;
      tmem_fence_after_sync();
      const uint64_t a0 = umma_desc(smem + sp.q * T::kQBytes, 0), b0 = umma_desc(smem_k + s * T::kKBytes, 0);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        umma_ss(leader, base + slot * KT, a0 + ((k / 4) * (128 * 128) + (k % 4) * 32) / 16,
                b0 + ((k / 4) * (KT * 128) + (k % 4) * 32) / 16, instr_s, k > 0);
      umma_commit(leader, s_full(slot));
      if (sp.q == tiles_q - 1) umma_commit(leader, k_empty(s));
      next(sp, KS);
    };
    if (ok) scores(0);
    if (ok && items > 1) scores(1);
    for (int i = 0; ok && i < items; ++i) {
      const int s = op.stage, slot = i & 1;
      if (op.q == 0) {
        ok = mbar_wait_close(v_full(s), op.parity, &abort_flag, p.error_flag, p.wait_limit_ns);
        // Rows that nobody sees have weight zero, which must meet zeros, whatever is there.
        const int key = (t0 + op.tile) * KT;
        const uint32_t bits = piece_bits[s];
        if (!T::kCodes && ok && (key < lo || key + KT > hi || bits != (1u << pieces) - 1u)) {
          for (int r = lane; r < KT; r += 32) {
            if (key + r >= lo && key + r < hi && (bits >> (r >> p.piece_log2) & 1)) continue;
            for (int c = 0; c < DV / 64; ++c)
              for (int w = 0; w < 8; ++w)
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(smem_v + s * T::kVBytes + c * (KT * 128) +
                                                                             r * 128 + w * 16),
                             "r"(0u)
                             : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
      }
      ok = ok && mbar_wait_close(p_full(slot), (i >> 1) & 1, &abort_flag, p.error_flag, p.wait_limit_ns);
      if (!ok) break;
      tmem_fence_after_sync();
      const uint64_t b0 = umma_desc(smem_v + s * T::kVBytes, KT * 128);
      const uint32_t o = base + T::kTmemO + op.q * DV, w = base + slot * KT;
#pragma unroll
      for (int k = 0; k < KT / 16; ++k) umma_ts(leader, o, w + k * 8, b0 + k * 2048 / 16, instr_o, op.tile > 0 || k > 0);
      umma_commit(leader, o_done(op.q));
      if (op.q == tiles_q - 1) umma_commit(leader, v_empty(s));
      next(op, VS);
      // Into the weights' columns, which the product before reads: one thread's products run in order.
      if (i + 2 < items) scores(slot);
    }
  } else if (warp < 8 && (warp >> 2) < tiles_q) {
    // ------------------------------------------------------------------ softmax of one query tile
    more_registers<T::kCodes>();
    const int q = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's 32 lanes
    const PrefillRow out = row_of(q, r);
    const int first = q * p.tile_tokens;  // the tile's first token, and its last
    const int last = min(first + p.tile_tokens, u.tokens) - 1;
    const int pos = u.position + min(first + r / p.rep, last);  // rows without a token go along with the last one
    const int below = p.window > 0 ? pos - p.window : -1;       // keys at or below it are out of the window
    float c = p.score_scale;
    float out_factor = 1.f;
    float m = -INFINITY;          // running maximum of the unscaled scores
    // c s - c m is rounded once, but c m before it: where that could be off by more than 2^-4 in a row of the warp,
    // s - m comes first. Only rows of the unit's tokens have a say in what their warp does: the others hold the next sequence's
    // queries, or whatever was in shared memory, and no output may depend on them.
    bool far = false;
    uint64_t l[2] = {0ull, 0ull};  // sums of weights, two pairs
    const uint32_t o_at = tmem + lanes + T::kTmemO + q * DV;
    // Are all blocks of this CTA's keys in the pool? Almost always; then no tile asks again.
    bool any_bad = false;
    {
      const int b0 = max(lo, t0 * KT) / p.block_size, b1 = (min(hi, (t0 + nt) * KT) - 1) / p.block_size;
      for (int i = b0 + r; i <= b1; i += 128)
        if (static_cast<unsigned>(u.table[i]) >= static_cast<unsigned>(p.num_blocks)) any_bad = true;
      if (any_bad && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
      any_bad = group_barrier_any(1 + q, 128, any_bad);
    }
    bool ok = true;
    if constexpr (HALF) {
      // This thread's query row to fp16, its largest value brought to [2^13, 2^14): what is below 2^-39 of that is lost.
      ok = mbar_wait_close(q_full, 0, &abort_flag, p.error_flag, p.wait_limit_ns);
      const uint32_t row = smem + q * T::kQBytes + r * 128;
      auto at = [&](int i) { return row + i / 8 * (128 * 128) + ((i % 8 ^ (r & 7)) << 4); };
      uint32_t most = 0u;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint32_t x[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at(i)) : "memory");
#pragma unroll
        for (int k = 0; k < 4; ++k) most = max(most, max(x[k] & 0x7FFFu, x[k] >> 16 & 0x7FFFu));
      }
      // 2^e with e = 13 - exponent; zeros and values that are not finite stay as they are
      const int e = most == 0u || most >= 0x7F80u ? 0 : min(13 - (static_cast<int>(most >> 7) - 127), 120);
      const float by = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint32_t x[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at(i)) : "memory");
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = pack_f16x2(__uint_as_float(x[k] << 16) * by, __uint_as_float(x[k] & 0xFFFF0000u) * by);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at(i)), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]) : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(q_half);
      const float* factors = p.factors + static_cast<size_t>(u.seq) * p.num_kv_heads + u.head;
      c = fmaxf(c / by / factors[0], 1e-37f);  // not zero, as ever
      out_factor = 1.f / factors[static_cast<size_t>(p.num_seqs) * p.num_kv_heads];
    }
    const int tiles = HALF && !ok ? 0 : nt;
    for (int j = 0; j < tiles; ++j) {
      const int i = j * tiles_q + q;
      const int key = (t0 + j) * KT;
      ok = mbar_wait_close(s_full(i & 1), (i >> 1) & 1, &abort_flag, p.error_flag, p.wait_limit_ns);
      if (!ok) break;
      tmem_fence_after_sync();
      const uint32_t s_at = tmem + lanes + (i & 1) * KT;
      // Which of the tile's keys this row sees: [v0, v1), less the pieces that were not copied.
      const bool masked = any_bad || key + KT > u.position + first + 1 ||
                          (p.window > 0 && key <= u.position + last - p.window);
      // Weights by the maximum so far, while the tile's own is found beside them. Where that one is more than
      // 2^8 above, the outputs are rescaled and the weights computed again, from scores that are still there.
      // The first tile waits for its maximum.
      uint32_t w[KT / 2];
#pragma unroll 1
      for (bool again = false;; again = true) {
        float s[KT];
        tmem_ld_tile<KT>(s_at, s);
        if (masked) {
          const int v0 = below + 1 - key, v1 = pos + 1 - key;
#pragma unroll
          for (int h = 0; h < KT / 32; ++h) {
            uint32_t seen = low_bits(v1 - 32 * h) & ~low_bits(v0 - 32 * h);
            if (any_bad) seen &= good_keys(key + 32 * h);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[32 * h + e] = (seen >> e & 1) ? s[32 * h + e] : -INFINITY;
          }
        }
        if (j == 0) m = row_max<KT>(s);
        uint64_t sums[2] = {l[0], l[1]};
        if (j == 0) far = __any_sync(0xffffffffu, out.live && fabsf(m) * c > 0x1p20f && fabsf(m) < INFINITY);
        if (far) subtract<KT>(s, m);
        const float up = fmaxf(m, weights<KT, HALF>(s, c, far ? 0.f : m, sums, w) + (far && m > -INFINITY ? m : 0.f));
        if (again || j == 0 ||
            !__any_sync(0xffffffffu, out.live && ((up - m) * c > 8.f || (m == -INFINITY && up > m)))) {
          l[0] = sums[0];
          l[1] = sums[1];
          break;
        }
        const float by = m == -INFINITY ? 0.f : fast_exp2((m - up) * c);
        m = up;
        far = __any_sync(0xffffffffu, out.live && fabsf(m) * c > 0x1p20f && fabsf(m) < INFINITY);
#pragma unroll
        for (int n = 0; n < 2; ++n) l[n] = mul2(l[n], pair(by, by));
        ok = mbar_wait_close(o_done(q), (j - 1) & 1, &abort_flag, p.error_flag, p.wait_limit_ns);
        if (!ok) break;
        tmem_fence_after_sync();
#pragma unroll 1
        for (int d = 0; d < DV; d += 32) {
          uint32_t o[32];
          tmem_ld_32(o_at + d, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
          tmem_st_32(o_at + d, o);
        }
      }
      if (!ok) break;
#pragma unroll
      for (int h = 0; h < KT / 64; ++h) tmem_st_32(s_at + h * 32, *reinterpret_cast<uint32_t(*)[32]>(w + 32 * h));  // over the scores
      tmem_wait_st();
      // Every phase of o_done is over before the next one's product can be issued, so that a parity
      // stands for one phase. With two query tiles this tile's scores came after that product.
      if (j > 0 && tiles_q == 1) ok = mbar_wait_close(o_done(q), (j - 1) & 1, &abort_flag, p.error_flag, p.wait_limit_ns);
      if (!ok) break;
      tmem_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(i & 1));
    }
    if (ok) ok = mbar_wait_close(o_done(q), (nt - 1) & 1, &abort_flag, p.error_flag, p.wait_limit_ns);
    if (ok) {
      tmem_fence_after_sync();
      const bool split = p.splits > 1;
      float l0, l1, l2, l3;
      unpair(l[0], l0, l1);
      unpair(l[1], l2, l3);
      const float sum = (l0 + l1) + (l2 + l3);
      const float inv = (sum != 0.f ? 1.f / sum : 0.f) * out_factor;
      if (split && out.live) {
        float* ml = p.ws_ml + (u.split * all_rows + out.row) * 2;
        ml[0] = m * (c / p.score_scale);  // unscaled (the factor is a power of two), so that the join can take differences first
        ml[1] = sum;
      }
#pragma unroll 1
      for (int d = 0; d < DV; d += 32) {
        uint32_t o[32];
        tmem_ld_32(o_at + d, o);
        tmem_wait_ld(o);
        if (out.live && split) {
          float4* to = reinterpret_cast<float4*>(p.ws_o + (u.split * all_rows + out.row) * DV + d);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            to[e] = make_float4(__uint_as_float(o[4 * e]) * out_factor, __uint_as_float(o[4 * e + 1]) * out_factor,
                                __uint_as_float(o[4 * e + 2]) * out_factor, __uint_as_float(o[4 * e + 3]) * out_factor);
        } else if (out.live) {
          uint4* to = reinterpret_cast<uint4*>(p.out + out.row * DV + d);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * inv, __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
            to[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
      }
    }
  } else if (warp >= 8) {
    fewer_registers<T::kCodes>();  // the rest of that warpgroup
  }

  __syncwarp();
  tmem_fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tmem_fence_after_sync();
    if (abort_flag) {  // a wait gave up: products may still run, and tensor memory is theirs until they are done
      int none = 0;
      umma_commit(elect_lane(), drained);  // the lane that issued the products
      mbar_wait_close(drained, 0, &none, p.error_flag, kWaitLimitNs);
    }
    tmem_free(tmem, kPrefillStates);
  }
}

}  // namespace pkv
