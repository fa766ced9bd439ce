// Values of the cached rows that a prompt attention call sees, from pages of codes: written once, where several query
// tiles would otherwise turn the same codes each for itself.
//
// e4m3 codes become bf16, which holds a code times a power of two exactly. Affine values need more bits than bf16 has:
// rounded to it, keys and values together cost the output as much again as its own rounding and that of bf16 weights
// do (root mean square 2.5e-3 of the output against 1.7e-3). They become fp16, each (sequence, KV head) and plane
// brought into fp16's range by a power of two that a pass over the scales and biases alone finds first; what is below
// 2^-39 of the largest is lost. Weights and queries are fp16 then as well.
//
// One CTA per (32 rows, KV head, plane): 16 codes a thread at a time, every load ahead of the first conversion. Bound by
// HBM: it reads the codes and writes twice (8-bit) or four times (4-bit) their bytes.
#include "pkv_codes.cuh"
#include "pkv_launch.h"
#include "pkv_rotate.cuh"

namespace pkv {

namespace {

constexpr int kRows = 32;
constexpr int kThreads = 128;

// Rows below `lowest` are nobody's: their blocks may have been given to others, so nothing of them is read.
template <int D, int FMT>
__device__ __forceinline__ void plane_values(const PrefillValuesParams& p, int plane, const int32_t* table, int first_row,
                                             int lowest, int len, uint16_t* out, int head, float factor) {
  constexpr int kPerRow = D / 16, kRounds = kRows * kPerRow / kThreads;
  uint4 v[kRounds];
  float scale[kRounds], bias[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int c = i * kThreads + threadIdx.x, r = c / kPerRow, col = c % kPerRow, t = first_row + r;
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    scale[i] = bias[i] = 0.f;
    if (t < lowest || t >= len) continue;
    const int blk = t / p.block_size;
    const int phys = table[blk];
    if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) continue;  // flagged by the attention
    const size_t cell = static_cast<size_t>(phys) * p.num_kv_heads + head;
    const size_t row = cell * p.block_size + (t - blk * p.block_size);
    if constexpr (FMT == 4) {
      const uint2 w = ld_keep_v2(p.pool[plane] + row * (D / 2) + col * 8);
      v[i].x = w.x;
      v[i].y = w.y;
    } else {
      v[i] = ld_keep_v4(p.pool[plane] + row * D + col * 16);
    }
    if constexpr (FMT == kFmtE4m3) {
      scale[i] = p.planes[plane].block_scales[cell];
    } else {
      scale[i] = __bfloat162float(p.planes[plane].scales[row * (D / 64) + col / 4]) * factor;
      bias[i] = __bfloat162float(p.planes[plane].biases[row * (D / 64) + col / 4]) * factor;
    }
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int c = i * kThreads + threadIdx.x, r = c / kPerRow;
    if (first_row + r < lowest || first_row + r >= len) continue;  // nobody's rows are left as they are
    uint32_t w[8];
    codes_to_values<FMT>(v[i], scale[i], bias[i], w);
    uint4* to = reinterpret_cast<uint4*>(out) + 2 * c;
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D, int DV, int FMT>
__global__ void __launch_bounds__(kThreads) pkv_prefill_values_kernel(const __grid_constant__ PrefillValuesParams p) {
  wait_for_prerequisite_grids();
  constexpr int kPer = kValueRows / kRows;
  const int block = blockIdx.x / kPer, head = blockIdx.y, plane = blockIdx.z, row0 = blockIdx.x % kPer * kRows;
  const int b = find_last(p.num_seqs, block, [&](int i) { return p.values.base(i, p.query_starts[i]); });
  const int start = p.query_starts[b], len = p.seq_lens[b];
  const long long n = static_cast<long long>(p.query_starts[b + 1]) - start;
  // bad starts and lengths are the attention's to flag
  if (start < 0 || n <= 0 || start + n > p.tokens || len < n || len > static_cast<long long>(p.max_blocks) * p.block_size)
    return;
  const long long row = static_cast<long long>(block - p.values.base(b, start)) * kValueRows +
                        p.values.first_row(len, static_cast<int>(n), p.window) + row0;
  if (block < p.values.base(b, start) || row >= len) return;
  const int lowest = p.values.lowest(len, static_cast<int>(n), p.window);
  const int32_t* table = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  const size_t to = (static_cast<size_t>(block) * p.num_kv_heads + head) * kValueRows + row0;
  uint16_t* out = static_cast<uint16_t*>(p.out[plane]);
  const float factor = FMT == kFmtE4m3 ? 1.f : p.factors[(plane * p.num_seqs + b) * p.num_kv_heads + head];
  if (plane == 0) {
    plane_values<D, FMT>(p, 0, table, static_cast<int>(row), lowest, len, out + to * D, head, factor);
  } else {
    plane_values<DV, FMT>(p, 1, table, static_cast<int>(row), lowest, len, out + to * DV, head, factor);
  }
}

// One CTA per (KV head, sequence, plane): the largest |scale * code + bias| that any code could have in the rows that
// are seen, and the power of two that brings it to [2^13, 2^14).
template <int FMT>
__global__ void __launch_bounds__(1024) pkv_prefill_range_kernel(const __grid_constant__ PrefillValuesParams p) {
  __shared__ float most[32];
  wait_for_prerequisite_grids();
  const int head = blockIdx.x, b = blockIdx.y, plane = blockIdx.z;
  const int start = p.query_starts[b], len = p.seq_lens[b];
  const long long n = static_cast<long long>(p.query_starts[b + 1]) - start;
  const bool seen = start >= 0 && n > 0 && start + n <= p.tokens && len >= n &&
                    len <= static_cast<long long>(p.max_blocks) * p.block_size;
  const int32_t* table = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  const int pairs = p.dim[plane] / 128;  // of groups in a row, one 32-bit word of scales each
  constexpr float kLevels = static_cast<float>((1 << FMT) - 1);
  float m = 0.f;
  if (seen) {
#pragma unroll 4
    for (int t = p.values.lowest(len, static_cast<int>(n), p.window) + threadIdx.x; t < len; t += 1024) {
      const int blk = t / p.block_size;
      const int phys = table[blk];
      if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) continue;
      const size_t row = (static_cast<size_t>(phys) * p.num_kv_heads + head) * p.block_size + (t - blk * p.block_size);
      for (int i = 0; i < pairs; ++i) {
        const __nv_bfloat162 s2 = reinterpret_cast<const __nv_bfloat162*>(p.planes[plane].scales)[row * pairs + i];
        const __nv_bfloat162 b2 = reinterpret_cast<const __nv_bfloat162*>(p.planes[plane].biases)[row * pairs + i];
        const float2 sc = __bfloat1622float2(s2), bi = __bfloat1622float2(b2);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(bi.x), fabsf(fmaf(sc.x, kLevels, bi.x))),
                           fmaxf(fabsf(bi.y), fabsf(fmaf(sc.y, kLevels, bi.y)))));
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 32; ++i) m = fmaxf(m, most[i]);
    // 2^(13 - exponent of m), within what f32 and its reciprocal hold
    const int e = 13 - (static_cast<int>(__float_as_uint(m) >> 23) - 127);
    p.factors[(plane * p.num_seqs + b) * p.num_kv_heads + head] =
        m > 0.f && m < INFINITY ? __uint_as_float(static_cast<uint32_t>(min(max(e, -120), 120) + 127) << 23) : 1.f;
  }
}

template <typename Kernel>
cudaError_t launch(Kernel kernel, dim3 grid, int threads, const PrefillValuesParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernels wait before they touch memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int DV, int FMT>
cudaError_t launch_of(const PrefillValuesParams& p, cudaStream_t stream) {
  if constexpr (FMT != kFmtE4m3) {
    const cudaError_t e = launch(pkv_prefill_range_kernel<FMT>, dim3(p.num_kv_heads, p.num_seqs, 2), 1024, p, stream);
    if (e != cudaSuccess) return e;
  }
  return launch(pkv_prefill_values_kernel<D, DV, FMT>, dim3(p.blocks * (kValueRows / kRows), p.num_kv_heads, 2), kThreads, p,
                stream);
}

}  // namespace

cudaError_t launch_prefill_values(const PrefillValuesParams& p, int fmt, cudaStream_t stream) {
#define X(B_, DK_, DV_) \
  if (fmt == B_ && p.dim[0] == DK_ && p.dim[1] == DV_) return launch_of<DK_, DV_, B_>(p, stream);
#define AFFINE(B_) X(B_, 128, 128) X(B_, 256, 256) X(B_, 256, 128) X(B_, 128, 256)
  AFFINE(kFmtE4m3) X(kFmtE4m3, 64, 64) X(kFmtE4m3, 192, 128) AFFINE(4) AFFINE(8)
#undef AFFINE
#undef X
  return cudaErrorInvalidValue;
}

}  // namespace pkv
