// Prompt attention over 8-bit affine pages.
#include "pkv_prefill_instances.cuh"

namespace pkv {

PKV_PREFILL_FORMAT(u8, 8, PKV_PREFILL_AFFINE)

}  // namespace pkv
