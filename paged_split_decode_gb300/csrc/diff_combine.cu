// diff_combine.cu -- launches the join of the differential decode's partials
// right behind the decode kernel (programmatic dependent launch), and picks
// the decode's instantiation by cache kind.
#include "diff_launch.h"

namespace pd {

bool diff_kernel_shape(int D, int kv, int ntm, int grouped, KernelShape* out) {
  switch (cache_kind(kv)) {
    case kKvF16: return diff_shape_f16(D, ntm, grouped, out);
    case kKvBf16: return diff_shape_bf16(D, ntm, grouped, out);
    case kKvFp8: return diff_shape_fp8(D, ntm, grouped, out);
    default: return diff_shape_i8(D, ntm, grouped, out);
  }
}

cudaError_t launch_diff(int D, int kv, int ntm, int grouped, const CUtensorMap& tk, const CUtensorMap& tv,
                        const DiffParams& p, int grid, cudaStream_t s) {
  switch (cache_kind(kv)) {
    case kKvF16: return diff_launch_f16(D, ntm, grouped, tk, tv, p, grid, s);
    case kKvBf16: return diff_launch_bf16(D, ntm, grouped, tk, tv, p, grid, s);
    case kKvFp8: return diff_launch_fp8(D, ntm, grouped, tk, tv, p, grid, s);
    default: return diff_launch_i8(D, ntm, grouped, tk, tv, p, grid, s);
  }
}

cudaError_t launch_diff_combine(int D, const DiffParams& p, int n_units, int row_chunks, int rows_at_once, int groups, bool many,
                                cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_units), static_cast<unsigned>(row_chunks),
                     static_cast<unsigned>(p.d.hg));
  cfg.blockDim = dim3(many ? kJoinThreadsMany : kJoinThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = D == 128 ? (many ? diff_combine_kernel<128, kJoinThreadsMany, 2> : diff_combine_kernel<128, kJoinThreads, 3>)
                               : (many ? diff_combine_kernel<256, kJoinThreadsMany, 2> : diff_combine_kernel<256, kJoinThreads, 3>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, rows_at_once, groups);
  if (e != cudaSuccess) return e;
  return cudaPeekAtLastError();
}

}  // namespace pd
