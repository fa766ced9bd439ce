// Prompt attention over 4-bit affine pages.
#include "pkv_prefill_instances.cuh"

namespace pkv {

PKV_PREFILL_FORMAT(u4, 4, PKV_PREFILL_AFFINE)

}  // namespace pkv
