// decode_fp4.cu -- instantiations of the decode over 4-bit caches.
#include "scored_launch.h"

namespace pd {
namespace {

// Shapes by row tiles of 8 query rows per KV head: row tiles of a warp, row groups, key groups, steps in the ring,
// CTAs per SM. One row tile, L = 4096, B = 1 / 8 / 32: D = 256, two CTAs of six warps 10.1 / 17.8 / 42.5 us, four of
// four 11.2 / 18.6 / 42.9 (128 registers), two of eight 10.6 / 18.8 / 44.0, one of 16 50.4 at B = 32; D = 128, four of
// four 9.8 / 12.3 / 28.7, five 10.6 / 13.6 / 31.0, two of eight 9.1 / 13.0 / 26.6 (at L = 1024 15.8 against 12.7). Three
// tiles in one warp read and convert a tile once: D = 128, 18 rows, B = 32, L = 4096 50.6 us, two groups of two
// 62.6 (D = 256 103 and 118; at L = 512 36.3 and 34.0); four tiles, D = 128, 58.3 and 65.8 (D = 256: their sums do
// not fit the registers).
template <int D, bool QB>
struct Shapes {
  using C1 = std::conditional_t<D == 256, Fp4Cfg<256, 1, 1, 6, 2, 2, QB>, Fp4Cfg<128, 1, 1, 4, 3, 4, QB>>;
  using C2 = std::conditional_t<D == 256, Fp4Cfg<256, 2, 1, 8, 4, 1, QB>, Fp4Cfg<128, 2, 1, 6, 6, 2, QB>>;
  using C3 = std::conditional_t<D == 256, Fp4Cfg<256, 3, 1, 6, 6, 1, QB>, Fp4Cfg<128, 3, 1, 6, 6, 2, QB>>;
  using C4 = std::conditional_t<D == 256, Fp4Cfg<256, 2, 2, 4, 4, 1, QB>, Fp4Cfg<128, 4, 1, 4, 8, 2, QB>>;

  template <class C>
  static bool shape_one(KernelShape* out) {
    static_assert(C::kSmemBytes <= smem_limit(C::kMinBlocks), "the rings fit");
    out->threads = C::kThreads;
    out->smem_bytes = C::kSmemBytes;
    out->rows_padded = C::RP;
    out->ctas_per_sm = C::kMinBlocks;
    out->heads = 1;
    // a piece's start and end, in tiles (one row tile, 32 ragged sequences of up to 16384 keys: D = 128 8 heads 16 / 32 /
    // 48 tiles 74.0 / 60.5 / 65.1 us, D = 256 4 heads 16 / 24 / 40 72.8 / 61.2 / 62.3; 32 x 8192 keys 65.6 / 68.5 / 72.5
    // and 67.4 / 66.9 / 68.4; two row tiles, D = 256 8 / 16 / 24 122 / 114 / 102)
    out->unit_cost = D == 128 && C::NT * C::RG == 1 ? 32 : 24;
    out->fixed_pieces = 0;
    for (int& c : out->max_clusters) c = 0;  // split units go through the combine
    return true;
  }
  template <class C>
  static cudaError_t launch_one(const Fp4Params& p, int grid, cudaStream_t s) {
    static unsigned long long attr_ctx[64] = {};
    const cudaError_t e =
        once_per_context(attr_ctx, [] { return set_kernel_attributes(decode_fp4_kernel<C>, C::kSmemBytes); });
    if (e != cudaSuccess) return e;
    return launch_pdl(decode_fp4_kernel<C>, grid, C::kThreads, C::kSmemBytes, s, 1, p);
  }
  static bool shape(int nt, KernelShape* out) {
    return nt == 1 ? shape_one<C1>(out) : nt == 2 ? shape_one<C2>(out) : nt == 3 ? shape_one<C3>(out) : nt == 4 && shape_one<C4>(out);
  }
  static cudaError_t launch(int nt, const Fp4Params& p, int grid, cudaStream_t s) {
    return nt == 1 ? launch_one<C1>(p, grid, s)
           : nt == 2 ? launch_one<C2>(p, grid, s)
           : nt == 3 ? launch_one<C3>(p, grid, s)
           : nt == 4 ? launch_one<C4>(p, grid, s)
                     : cudaErrorInvalidValue;
  }
};

}  // namespace

bool fp4_shape(int D, bool q_bf16, int nt, KernelShape* out) {
  if (D == 128) return q_bf16 ? Shapes<128, true>::shape(nt, out) : Shapes<128, false>::shape(nt, out);
  return D == 256 && (q_bf16 ? Shapes<256, true>::shape(nt, out) : Shapes<256, false>::shape(nt, out));
}
cudaError_t fp4_launch(int D, bool q_bf16, int nt, const Fp4Params& p, int grid, cudaStream_t s) {
  if (D == 128) return q_bf16 ? Shapes<128, true>::launch(nt, p, grid, s) : Shapes<128, false>::launch(nt, p, grid, s);
  return q_bf16 ? Shapes<256, true>::launch(nt, p, grid, s) : Shapes<256, false>::launch(nt, p, grid, s);
}

bool scored_kernel_shape(int D, int kv, int nt, int grouped, KernelShape* out) {
  if (D != 128 && D != 256) return false;
  if (is_fp4(kv)) return !grouped && fp4_shape(D, kv == kKvFp4Bq, nt, out);
  switch (kv) {
    case kKvF16: return D == 128 ? scored_shape_f16_128(nt, grouped, out) : scored_shape_f16_256(nt, grouped, out);
    case kKvBf16: return D == 128 ? scored_shape_bf16_128(nt, grouped, out) : scored_shape_bf16_256(nt, grouped, out);
    case kKvFp8: return D == 128 ? scored_shape_fp8_128(nt, grouped, out) : scored_shape_fp8_256(nt, grouped, out);
    case kKvInt8: return D == 128 ? scored_shape_i8_128(nt, grouped, out) : scored_shape_i8_256(nt, grouped, out);
    case kKvFp8Bq: return D == 128 ? scored_shape_fp8q_128(nt, grouped, out) : scored_shape_fp8q_256(nt, grouped, out);
    case kKvInt8Bq: return D == 128 ? scored_shape_i8q_128(nt, grouped, out) : scored_shape_i8q_256(nt, grouped, out);
    default: return false;
  }
}
cudaError_t launch_scored(int D, int kv, int nt, int grouped, const CUtensorMap& k, const CUtensorMap& v,
                          const Fp4Params& p, int grid, cudaStream_t s) {
  if (is_fp4(kv)) return fp4_launch(D, kv == kKvFp4Bq, nt, p, grid, s);
  switch (kv) {
    case kKvF16:
      return D == 128 ? scored_launch_f16_128(nt, grouped, k, v, p, grid, s) : scored_launch_f16_256(nt, grouped, k, v, p, grid, s);
    case kKvBf16:
      return D == 128 ? scored_launch_bf16_128(nt, grouped, k, v, p, grid, s) : scored_launch_bf16_256(nt, grouped, k, v, p, grid, s);
    case kKvFp8:
      return D == 128 ? scored_launch_fp8_128(nt, grouped, k, v, p, grid, s) : scored_launch_fp8_256(nt, grouped, k, v, p, grid, s);
    case kKvInt8:
      return D == 128 ? scored_launch_i8_128(nt, grouped, k, v, p, grid, s) : scored_launch_i8_256(nt, grouped, k, v, p, grid, s);
    case kKvFp8Bq:
      return D == 128 ? scored_launch_fp8q_128(nt, grouped, k, v, p, grid, s) : scored_launch_fp8q_256(nt, grouped, k, v, p, grid, s);
    case kKvInt8Bq:
      return D == 128 ? scored_launch_i8q_128(nt, grouped, k, v, p, grid, s) : scored_launch_i8q_256(nt, grouped, k, v, p, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pd
