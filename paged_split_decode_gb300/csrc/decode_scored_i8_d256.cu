// decode_scored_i8_d256.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(i8_256, 256, kKvInt8)
}  // namespace pd
