// scored_launch.h -- internal interface between the host layer and the scored
// decode's instantiation units (one per cache element kind and head size) and the
// 4-bit caches' (decode_fp4.cu).
#pragma once
#include "decode_fp4.cuh"
#include "decode_scored.cuh"
#include "decode_tci8.cuh"
#include "launch.h"

namespace pd {

// 4-bit caches under an fp16 and a bfloat16 q (beside the kinds of decode_kernel.cuh).
constexpr int kKvFp4 = 6, kKvFp4Bq = 7;
constexpr bool is_fp4(int kv) { return kv == kKvFp4 || kv == kKvFp4Bq; }

// As kernel_shape and launch_decode. (4-bit caches take no tensor maps.)
bool scored_kernel_shape(int D, int kv, int nt, int grouped, KernelShape* out);
cudaError_t launch_scored(int D, int kv, int nt, int grouped, const CUtensorMap& tk, const CUtensorMap& tv,
                          const Fp4Params& p, int grid, cudaStream_t stream);
cudaError_t launch_scored_combine(int D, const ScoredParams& p, int n_units, int dim_chunks, int batch, int threads,
                                  cudaStream_t stream);

// Adds the softmax weights of a scored decode, from the scores and the rows' (m, l) that it left
// in the workspace, to the keys' sums (key_weights.cu).
struct KeyWeightParams {
  ScoredParams d;
  const float* in;  // [num_blocks, Hkv, block_size]
  float* out;       // the same, may be in
  int row_tiles;    // row tiles of a unit's head in the scores
  int chunks;       // CTAs of a unit (set by the launch)
};
cudaError_t launch_key_weights(KeyWeightParams p, int sms, cudaStream_t stream);

// The deepest ring (at most 32 stages, a multiple of the key groups) that lets MINB CTAs share an SM.
template <int D, int KV, int HG, int RG, int KG, int MINB, int NS = 32>
constexpr int scored_stages() {
  if constexpr (NS <= KG || NS <= 2)
    return KG > 2 ? KG : 2;
  else if constexpr (NS % KG != 0)
    return scored_stages<D, KV, HG, RG, KG, MINB, NS - 1>();
  else if constexpr (ScoredCfg<D, KV, HG, RG, KG, NS, MINB>::kSmemBytes <= smem_limit(MINB))
    return NS;
  else
    return scored_stages<D, KV, HG, RG, KG, MINB, NS - 1>();
}
template <int D, int KV, int HG, int RG, int KG, int MINB>
using ScoredCfgFor = ScoredCfg<D, KV, HG, RG, KG, scored_stages<D, KV, HG, RG, KG, MINB>(), MINB>;

template <int D, int KV>
struct ScoredShapes {
  // heads per tile, row tiles per head, key groups, CTAs per SM. C4, 30 rows over fp16 caches, B = 8: two key groups in
  // one CTA 40.3 us at L = 4096 and 16.6 at 512, two CTAs of one group 46.4 and 16.1 (C2, C3 the other way round:
  // 42.4 and 37.3 against 32.8 and 33.1).
  using C1H = ScoredCfgFor<D, KV, 4, 1, 1, 1>;
  using C1 = ScoredCfgFor<D, KV, 1, 1, 3, 2>;
  using C2 = ScoredCfgFor<D, KV, 1, 2, 1, 2>;
  using C3 = ScoredCfgFor<D, KV, 1, 3, 1, 2>;
  using C4 = ScoredCfgFor<D, KV, 1, 4, 2, 1>;

  template <class C>
  static bool shape_one(KernelShape* out) {
    static_assert(C::kSmemBytes <= smem_limit(C::kMinBlocks), "the ring fits");
    out->threads = C::kThreads;
    out->smem_bytes = C::kSmemBytes;
    out->rows_padded = C::RP;
    out->ctas_per_sm = C::kMinBlocks;
    out->heads = C::HG;
    out->step_tiles = C::KG;
    out->key_groups = C::KG;
    out->whole_tile = 1;
    // (key groups, 14 x 2 heads, D = 128, fp16, 128 ragged sequences of up to 1024 keys: 12 / 24 tiles 25.3 / 22.0 us, 32 of
    // up to 16384 44.7 / 43.5; four heads a tile 4 / 8 51.6 / 49.5 and 143.9 / 144.9, whole 4096 keys 88.4 / 89.1)
    out->unit_cost = C::KG > 1 ? 24 : 4;
    out->fixed_pieces = 0;
    for (int& c : out->max_clusters) c = 0;  // split units go through the combine
    return true;
  }
  template <class C>
  static cudaError_t launch_one(const CUtensorMap& tk, const CUtensorMap& tv, const ScoredParams& p, int grid,
                                cudaStream_t s) {
    static unsigned long long attr_ctx[64] = {};
    const cudaError_t e =
        once_per_context(attr_ctx, [] { return set_kernel_attributes(decode_scored_kernel<C>, C::kSmemBytes); });
    if (e != cudaSuccess) return e;
    return launch_pdl(decode_scored_kernel<C>, grid, C::kThreads, C::kSmemBytes, s, 1, tk, tv, p);
  }
  // Two to four row tiles over e4m3 caches, and over int8 caches under a bfloat16 q (an fp16 output wants more bits
  // of P than the int8 kernel's products take): the kernels of tensor memory. 18 rows, B = 8, L = 4096: e4m3 20.5 us
  // against C3's 34.8, int8 26.4 against 40.0.
  static constexpr bool kTc = cache_kind(KV) == kKvFp8 || KV == kKvInt8Bq;
  template <int NG>
  using Tc = std::conditional_t<cache_kind(KV) == kKvFp8, Tc8<D, q_is_bf16(KV), NG, true>, Tci8<D, true, NG, true>>;
  template <int NG>
  static bool shape_tc(KernelShape* out) {
    if constexpr (cache_kind(KV) == kKvFp8) return shape_tc8<Tc<NG>>(NG, out);
    else return shape_tci8<Tc<NG>>(NG, out);
  }
  template <int NG>
  static cudaError_t launch_tc(const CUtensorMap& tk, const CUtensorMap& tv, const ScoredParams& p, int grid, cudaStream_t s) {
    if constexpr (cache_kind(KV) == kKvFp8) return launch_tc8<Tc<NG>>(tk, tv, p, grid, s);
    else return launch_tci8<Tc<NG>>(tk, tv, p, grid, s);
  }
  static bool shape(int nt, int grouped, KernelShape* out) {
    if (grouped) return nt == 1 && shape_one<C1H>(out);
    if constexpr (kTc) {
      if (nt > 1) return nt == 2 ? shape_tc<2>(out) : nt == 3 ? shape_tc<3>(out) : nt == 4 && shape_tc<4>(out);
      return shape_one<C1>(out);
    } else
    switch (nt) {
      case 1: return shape_one<C1>(out);
      case 2: return shape_one<C2>(out);
      case 3: return shape_one<C3>(out);
      case 4: return shape_one<C4>(out);
      default: return false;
    }
  }
  static cudaError_t launch(int nt, int grouped, const CUtensorMap& tk, const CUtensorMap& tv, const ScoredParams& p,
                            int grid, cudaStream_t s) {
    if (grouped) return nt == 1 ? launch_one<C1H>(tk, tv, p, grid, s) : cudaErrorInvalidValue;
    if constexpr (kTc) {
      return nt == 1   ? launch_one<C1>(tk, tv, p, grid, s)
             : nt == 2 ? launch_tc<2>(tk, tv, p, grid, s)
             : nt == 3 ? launch_tc<3>(tk, tv, p, grid, s)
             : nt == 4 ? launch_tc<4>(tk, tv, p, grid, s)
                       : cudaErrorInvalidValue;
    } else
    switch (nt) {
      case 1: return launch_one<C1>(tk, tv, p, grid, s);
      case 2: return launch_one<C2>(tk, tv, p, grid, s);
      case 3: return launch_one<C3>(tk, tv, p, grid, s);
      case 4: return launch_one<C4>(tk, tv, p, grid, s);
      default: return cudaErrorInvalidValue;
    }
  }
};

#define PD_SCORED_UNIT(name, D, KV)                                                                              \
  bool scored_shape_##name(int nt, int grouped, KernelShape* out) { return ScoredShapes<D, KV>::shape(nt, grouped, out); } \
  cudaError_t scored_launch_##name(int nt, int grouped, const CUtensorMap& tk, const CUtensorMap& tv,            \
                                   const ScoredParams& p, int grid, cudaStream_t s) {                            \
    return ScoredShapes<D, KV>::launch(nt, grouped, tk, tv, p, grid, s);                                         \
  }
#define PD_SCORED_DECL(name)                                                                                     \
  bool scored_shape_##name(int nt, int grouped, KernelShape* out);                                               \
  cudaError_t scored_launch_##name(int nt, int grouped, const CUtensorMap&, const CUtensorMap&, const ScoredParams&, int, \
                                   cudaStream_t);
PD_SCORED_DECL(f16_128)
PD_SCORED_DECL(f16_256)
PD_SCORED_DECL(bf16_128)
PD_SCORED_DECL(bf16_256)
PD_SCORED_DECL(fp8_128)
PD_SCORED_DECL(fp8_256)
PD_SCORED_DECL(i8_128)
PD_SCORED_DECL(i8_256)
PD_SCORED_DECL(fp8q_128)
PD_SCORED_DECL(fp8q_256)
PD_SCORED_DECL(i8q_128)
PD_SCORED_DECL(i8q_256)
bool fp4_shape(int D, bool q_bf16, int nt, KernelShape* out);
cudaError_t fp4_launch(int D, bool q_bf16, int nt, const Fp4Params& p, int grid, cudaStream_t s);

}  // namespace pd
