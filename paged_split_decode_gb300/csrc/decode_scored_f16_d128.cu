// decode_scored_f16_d128.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(f16_128, 128, kKvF16)
}  // namespace pd
