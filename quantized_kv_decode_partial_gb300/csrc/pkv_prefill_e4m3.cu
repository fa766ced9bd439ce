// Prompt attention over e4m3 pages.
#include "pkv_prefill_instances.cuh"

namespace pkv {

PKV_PREFILL_FORMAT(e4m3, kFmtE4m3, false, PKV_PREFILL_WIDE)

}  // namespace pkv
