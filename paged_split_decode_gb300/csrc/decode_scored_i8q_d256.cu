// decode_scored_i8q_d256.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(i8q_256, 256, kKvInt8Bq)
}  // namespace pd
