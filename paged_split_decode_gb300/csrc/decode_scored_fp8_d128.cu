// decode_scored_fp8_d128.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(fp8_128, 128, kKvFp8)
}  // namespace pd
