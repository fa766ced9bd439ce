// Prompt attention over bf16 pages, and the join of split key ranges.
#include "pkv_prefill_instances.cuh"

namespace pkv {

namespace {

struct PrefillJoinParams {
  const float* ws_o;
  const float* ws_ml;
  const int32_t* query_starts;
  __nv_bfloat16* out;
  int num_seqs, tokens, num_q_heads, splits;
  float score_scale;
};

// One warp per output row: the states of its splits, weighted by 2^(c (m - max m)). Differences of maxima come before
// the scale: rounded products c m would lose them far from zero.
template <int DV>
__global__ void __launch_bounds__(128) pkv_prefill_join_kernel(const __grid_constant__ PrefillJoinParams p) {
  wait_for_prerequisite_grids();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const long long rows = static_cast<long long>(p.tokens) * p.num_q_heads;
  if (row >= rows) return;
  const int t = static_cast<int>(row / p.num_q_heads);
  const int b = find_last(p.num_seqs, t, [&](int i) { return p.query_starts[i]; });
  if (p.query_starts[b] > t || p.query_starts[b + 1] <= t) return;  // a row of no sequence stays as it was
  constexpr int V = DV / 32 >= 4 ? 4 : 2;  // values a lane takes at once
  constexpr int N = DV / (32 * V);
  float acc[N][V] = {}, total = 0.f, top = -INFINITY;
  for (int s0 = 0; s0 < p.splits; s0 += 32) {
    const float* ml = p.ws_ml + (static_cast<size_t>(s0 + lane) * rows + row) * 2;
    const bool have = s0 + lane < p.splits;
    const float m = have ? ml[0] : -INFINITY, l = have ? ml[1] : 0.f;
    float mx = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float up = fmaxf(top, mx);
    if (up == -INFINITY) continue;
    const float by = top == -INFINITY ? 0.f : fast_exp2((top - up) * p.score_scale);
    top = up;
    total *= by;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[n][v] *= by;
    const float w = l != 0.f ? fast_exp2((m - up) * p.score_scale) : 0.f;  // a split without keys has no outputs
    float sum = w * l;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    total += sum;
    for (int s = 0; s < min(32, p.splits - s0); ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s);
      if (__shfl_sync(0xffffffffu, l, s) == 0.f) continue;
      const float* o = p.ws_o + (static_cast<size_t>(s0 + s) * rows + row) * DV + lane * V;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(o + n * 32 * V);
          acc[n][0] = fmaf(ws, x.x, acc[n][0]);
          acc[n][1] = fmaf(ws, x.y, acc[n][1]);
          acc[n][2] = fmaf(ws, x.z, acc[n][2]);
          acc[n][3] = fmaf(ws, x.w, acc[n][3]);
        } else {
          const float2 x = *reinterpret_cast<const float2*>(o + n * 32 * V);
          acc[n][0] = fmaf(ws, x.x, acc[n][0]);
          acc[n][1] = fmaf(ws, x.y, acc[n][1]);
        }
      }
    }
  }
  const float inv = total != 0.f ? 1.f / total : 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    __nv_bfloat16* to = p.out + row * DV + n * 32 * V + lane * V;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      *reinterpret_cast<uint32_t*>(to + v) = pack_bf16x2(acc[n][v] * inv, acc[n][v + 1] * inv);
  }
}

}  // namespace

PKV_PREFILL_FORMAT(bf16, 16, false, PKV_PREFILL_WIDE)

cudaError_t launch_prefill_join(const PrefillParams& p, int dv, cudaStream_t stream) {
  PrefillJoinParams j{p.ws_o, p.ws_ml, p.query_starts, p.out, p.num_seqs, p.tokens, p.num_q_heads, p.splits, p.score_scale};
  const long long rows = static_cast<long long>(p.tokens) * p.num_q_heads;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
  if (dv == 64) return launch_dependent(pkv_prefill_join_kernel<64>, grid, 128, 0, stream, j);
  if (dv == 128) return launch_dependent(pkv_prefill_join_kernel<128>, grid, 128, 0, stream, j);
  return launch_dependent(pkv_prefill_join_kernel<256>, grid, 128, 0, stream, j);
}

}  // namespace pkv
