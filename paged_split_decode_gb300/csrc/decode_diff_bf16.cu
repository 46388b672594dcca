// decode_diff_bf16.cu -- instantiations of the differential decode for bfloat16
// caches, D = 128 and 256 (one translation unit per kind, compiled in parallel).
#include "diff_launch.h"

namespace pd {
namespace {
using S128 = DiffShapes<128, kKvBf16>;
using S256 = DiffShapes<256, kKvBf16>;
}  // namespace

bool diff_shape_bf16(int D, int ntm, int grouped, KernelShape* out) {
  return D == 128 ? S128::shape(ntm, grouped, out) : D == 256 && S256::shape(ntm, grouped, out);
}
cudaError_t diff_launch_bf16(int D, int ntm, int grouped, const CUtensorMap& tk, const CUtensorMap& tv,
                           const DiffParams& p, int grid, cudaStream_t s) {
  return D == 128 ? S128::launch(ntm, grouped, tk, tv, p, grid, s) : S256::launch(ntm, grouped, tk, tv, p, grid, s);
}

}  // namespace pd
