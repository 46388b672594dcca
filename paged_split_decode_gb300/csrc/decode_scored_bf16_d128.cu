// decode_scored_bf16_d128.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(bf16_128, 128, kKvBf16)
}  // namespace pd
