// decode_scored_fp8_d256.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(fp8_256, 256, kKvFp8)
}  // namespace pd
