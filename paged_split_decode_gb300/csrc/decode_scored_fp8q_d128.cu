// decode_scored_fp8q_d128.cu -- the scored decode's instantiations for one cache kind
// and head size (a translation unit each, compiled in parallel).
#include "scored_launch.h"

namespace pd {
PD_SCORED_UNIT(fp8q_128, 128, kKvFp8Bq)
}  // namespace pd
