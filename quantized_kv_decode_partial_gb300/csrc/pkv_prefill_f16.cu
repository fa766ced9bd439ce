// Prompt attention over fp16 values (of affine pages).
#include "pkv_prefill_instances.cuh"

namespace pkv {

PKV_PREFILL_FORMAT(f16, 16, true, PKV_PREFILL_AFFINE)

}  // namespace pkv
