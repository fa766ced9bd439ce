// Launches of the prompt attention kernel, shared by the translation units of the page formats.
#pragma once

#include <atomic>

#include "pkv_launch.h"
#include "pkv_prefill.cuh"

namespace pkv {

template <typename... Args>
inline cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream,
                             const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the kernels wait before they touch memory
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int DV, int FMT, bool HALF>
cudaError_t launch_prefill_of(const PrefillParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int units,
                      cudaStream_t stream, int device) {
  constexpr int smem = PrefillShape<D, DV, FMT>::kSmem;
  static std::atomic<bool> ready[256];  // per device; a second thread's call sets the same attribute again
  if (device < 0 || device >= 256 || !ready[device].load(std::memory_order_relaxed)) {
    const cudaError_t e =
        cudaFuncSetAttribute(pkv_prefill_kernel<D, DV, FMT, HALF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (device >= 0 && device < 256) ready[device].store(true, std::memory_order_relaxed);
  }
  return launch_dependent(pkv_prefill_kernel<D, DV, FMT, HALF>, dim3(units * p.num_kv_heads * p.splits), PrefillShape<D, DV, FMT>::kThreads, smem, stream,
                          p, tq, tk, tv);
}

template <int D, int DV, int FMT>
PrefillInfo prefill_info_of() {
  using T = PrefillShape<D, DV, FMT>;
  return PrefillInfo{true, T::kQ, T::KT, T::kSmem};
}

#define PKV_PREFILL_WIDE(X) X(64, 64) X(128, 128) X(256, 256) X(192, 128) X(256, 128) X(128, 256)
#define PKV_PREFILL_AFFINE(X) X(128, 128) X(256, 256) X(256, 128) X(128, 256)

// prefill_info_NAME and launch_prefill_NAME of a format and its pairs of head dims
#define PKV_PREFILL_INFO_OF(DK_, DV_) \
  if (dk == DK_ && dv == DV_) return prefill_info_of<DK_, DV_, kFmt>();
#define PKV_PREFILL_LAUNCH_OF(DK_, DV_) \
  if (dk == DK_ && dv == DV_) return launch_prefill_of<DK_, DV_, kFmt, kHalf>(p, tq, tk, tv, units, stream, device);
#define PKV_PREFILL_FORMAT(NAME, FMT, HALF, SHAPES)                                                                    \
  PrefillInfo prefill_info_##NAME(int dk, int dv) {                                                                    \
    constexpr int kFmt = FMT;                                                                                          \
    SHAPES(PKV_PREFILL_INFO_OF)                                                                                        \
    return PrefillInfo{};                                                                                              \
  }                                                                                                                    \
  cudaError_t launch_prefill_##NAME(int dk, int dv, const PrefillParams& p, const CUtensorMap& tq, const CUtensorMap& tk, \
                                    const CUtensorMap& tv, int units, cudaStream_t stream, int device) {               \
    constexpr int kFmt = FMT;                                                                                          \
    constexpr bool kHalf = HALF;                                                                                       \
    SHAPES(PKV_PREFILL_LAUNCH_OF)                                                                                      \
    return cudaErrorInvalidValue;                                                                                      \
  }

}  // namespace pkv
