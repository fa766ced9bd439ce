// Write side of e4m3 pages: appends a step's (or a prompt's) new K/V rows into pages that
// hold one f32 scale per (block, KV head) and plane.
//
// Per (sequence, KV head, plane, touched block), with a the largest magnitude of the block's
// new rows and s the block's scale (0 when no earlier row is in the block):
//     s'   = max(s, 2^ceil(log2(a / 448)))       448: the largest e4m3 value
//     code = e4m3(x / s')                         new rows, nearest even
//     code = e4m3(code * (s / s'))                earlier rows, when s' > s
// A power of two costs e4m3 nothing but range it does not need, and makes a grown scale an
// exact shift of the earlier codes (only their smallest values lose bits), so rows appended
// one by one end where rows appended together do.
//
// A block's new rows are contiguous in k_new/v_new and in the pool, so a unit is one run of
// 16-byte loads and 8-byte stores: bound by HBM, 2 bytes read and 1 written per value (8 sequences
// of 8192 new tokens, 8 KV heads, D=128: 60.6 us, 0.99 of a copy's rate; one token of 64
// sequences: 1.95 us, the launch).
#include <type_traits>

#include "pkv_e4m3.cuh"
#include "pkv_launch.h"

namespace pkv {

namespace {

// Grid (touched block x KV head x plane, sequence). kHold: 16-byte loads a thread keeps in
// registers between the two uses of the values (rows beyond those are read again).
template <int kHold>
__global__ void __launch_bounds__(128) pkv_append_blocks_kernel(const __grid_constant__ AppendBlockParams p) {
  __shared__ uint32_t red[4];
  wait_for_prerequisite_grids();
  const int plane = blockIdx.x & 1;
  const int unit = blockIdx.x >> 1;
  const int t = unit / p.num_kv_heads, h = unit - t * p.num_kv_heads, b = blockIdx.y;
  const int len = p.seq_lens[b];
  const long long end = static_cast<long long>(len) + p.n_new;
  if (len < 0 || end > static_cast<long long>(p.max_blocks) * p.block_size) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadSeqLen);
    return;
  }
  const int blk = len / p.block_size + t;
  const long long first = static_cast<long long>(blk) * p.block_size;  // the block's first position
  if (first >= end) return;
  const int r0 = first < len ? static_cast<int>(len - first) : 0;       // its first new row
  const int r1 = static_cast<int>(min(end - first, static_cast<long long>(p.block_size)));
  const int phys = p.block_tables[static_cast<size_t>(b) * p.max_blocks + blk];
  const int D = p.dim[plane];
  const uint4* src = reinterpret_cast<const uint4*>(
      p.src[plane] +
      ((static_cast<size_t>(b) * p.num_kv_heads + h) * p.n_new + static_cast<size_t>(first + r0 - len)) * D);
  const int n8 = (r1 - r0) * (D / 8);
  const int T = blockDim.x;

  uint4 v[kHold];
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    const int i = threadIdx.x + k * T;
    v[k] = i < n8 ? ld_nc_keep_v4(src + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  // the rows are in flight while the table's answer arrives
  if (static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_blocks)) {
    if (threadIdx.x == 0 && p.error_flag) atomicOr(p.error_flag, kDevErrBadBlock);
    return;
  }
  const size_t cell = static_cast<size_t>(phys) * p.num_kv_heads + h;
  uint8_t* block = p.pool[plane] + cell * p.block_size * D;
  uint2* dst = reinterpret_cast<uint2*>(block + static_cast<size_t>(r0) * D);
  const float old = r0 > 0 ? p.scales[plane][cell] : 0.f;
#pragma unroll
  for (int k = 0; k < kHold; ++k) m = max_abs(m, v[k]);
  for (int i = threadIdx.x + kHold * T; i < n8; i += T) m = max_abs(m, src[i]);
  m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
  if (T > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    m = max(max(red[0], red[1]), max(red[2], red[3]));
  } else {
    __syncwarp();  // every lane has read the old scale
  }
  const float need = pow2_scale(__uint_as_float(m << 16));
  const float s = fmaxf(old, need);
  if (threadIdx.x == 0) p.scales[plane][cell] = s;
  if (r0 > 0 && s > old) {  // the earlier rows' codes under the larger scale
    const float ratio = __fdiv_rn(old, s);
    uint2* row = reinterpret_cast<uint2*>(block);
    for (int i = threadIdx.x; i < r0 * (D / 8); i += T) {
      uint2 w = row[i];
      w.x = rescale4(w.x, ratio);
      w.y = rescale4(w.y, ratio);
      row[i] = w;
    }
  }
  const float inv = s > 0.f ? 1.f / s : 0.f;  // s = 0: every value is 0, and so is every code
  const float by = s > 0.f ? s : 1.f;
  auto write = [&](auto exact) {
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
      const int i = threadIdx.x + k * T;
      if (i < n8) dst[i] = quantize8<decltype(exact)::value>(v[k], by, inv);
    }
    for (int i = threadIdx.x + kHold * T; i < n8; i += T) dst[i] = quantize8<decltype(exact)::value>(src[i], by, inv);
  };
  if ((__float_as_uint(s) & 0x7FFFFFu) == 0u) {
    write(std::true_type{});
  } else {
    write(std::false_type{});
  }
}

}  // namespace

cudaError_t launch_append_blocks(const AppendBlockParams& p, int num_seqs, cudaStream_t stream) {
  if (p.n_new == 0) return cudaSuccess;
  const int most = (p.block_size - 1 + p.n_new - 1) / p.block_size + 1;  // blocks n_new rows can touch
  const int blocks = most < p.max_blocks ? most : p.max_blocks;
  const long long units = static_cast<long long>(blocks) * p.num_kv_heads * 2;
  if (units >= (1ll << 31)) return cudaErrorInvalidValue;
  const int rows = p.n_new < p.block_size ? p.n_new : p.block_size;
  const int loads = rows * (max(p.dim[0], p.dim[1]) / 8);  // 16-byte loads of a unit
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units), num_seqs);
  // One warp where it holds a unit's rows in registers (a few tokens), else four: with 4 loads
  // per thread while that covers a unit (fewer registers, more units per SM), else with 8.
  const bool one_warp = loads <= 4 * 32;
  cfg.blockDim = dim3(one_warp ? 32 : 128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernel waits before it touches memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return loads <= 4 * 128 ? cudaLaunchKernelEx(&cfg, pkv_append_blocks_kernel<4>, p)
                          : cudaLaunchKernelEx(&cfg, pkv_append_blocks_kernel<8>, p);
}

}  // namespace pkv
