// decode_scored_f16_d256.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(f16_256, 256, kKvF16)
}  // namespace pd
