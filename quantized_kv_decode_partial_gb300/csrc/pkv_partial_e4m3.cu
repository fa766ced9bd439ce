// e4m3 pages (one f32 scale per block and KV head): head dims 64 / 128 / 256 and key/value
// head dims 192/128, 256/128 and 128/256, each with up to 64 query rows per KV head.
// The SOLO instances serve grids of at most one CTA per SM (see PartialCfg).
#include "pkv_partial_instances.cuh"

namespace pkv {

#define PKV_E4M3_INSTANCES(X) \
  X(64, 64, 1, 1, false) X(64, 64, 2, 1, false) X(64, 64, 4, 1, false) X(64, 64, 4, 2, false) \
  X(128, 128, 1, 1, false) X(128, 128, 2, 1, false) X(128, 128, 2, 2, false) X(128, 128, 2, 4, false) \
  X(256, 256, 1, 1, false) X(256, 256, 1, 2, false) X(256, 256, 1, 4, false) X(256, 256, 1, 8, false) \
  X(192, 128, 1, 1, false) X(192, 128, 1, 2, false) X(192, 128, 1, 4, false) X(192, 128, 1, 8, false) \
  X(256, 128, 1, 1, false) X(256, 128, 1, 2, false) X(256, 128, 1, 4, false) X(256, 128, 1, 8, false) \
  X(128, 256, 1, 1, false) X(128, 256, 1, 2, false) X(128, 256, 1, 4, false) X(128, 256, 1, 8, false) \
  X(64, 64, 1, 1, true) X(128, 128, 1, 1, true) X(256, 256, 1, 1, true)

PartialInfo partial_info_e4m3(int dk, int dv, int nq, bool solo) {
  int nt, wq;
  tiles_for(dk, dv, nq, nt, wq);
#define X(DK_, DV_, NT_, WQ_, SOLO_) \
  if (dk == DK_ && dv == DV_ && nt == NT_ && wq == WQ_ && solo == SOLO_) \
    return info_of<kFmtE4m3, DK_, DV_, NT_, WQ_, SOLO_>();
  PKV_E4M3_INSTANCES(X)
#undef X
  return PartialInfo{};
}

cudaError_t launch_partial_e4m3(int dk, int dv, int nq, bool solo, const PartialParams& p, const CUtensorMap& tk,
                                const CUtensorMap& tv, dim3 grid, cudaStream_t s, int dev) {
  int nt, wq;
  tiles_for(dk, dv, nq, nt, wq);
#define X(DK_, DV_, NT_, WQ_, SOLO_) \
  if (dk == DK_ && dv == DV_ && nt == NT_ && wq == WQ_ && solo == SOLO_) \
    return launch_of<kFmtE4m3, DK_, DV_, NT_, WQ_, SOLO_>(p, tk, tv, grid, s, dev);
  PKV_E4M3_INSTANCES(X)
#undef X
  return cudaErrorInvalidValue;
}

}  // namespace pkv
