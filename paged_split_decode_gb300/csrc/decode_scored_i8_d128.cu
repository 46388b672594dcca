// decode_scored_i8_d128.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(i8_128, 128, kKvInt8)
}  // namespace pd
