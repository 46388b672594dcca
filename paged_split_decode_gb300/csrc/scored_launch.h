// scored_launch.h -- internal interface between the host layer and the scored
// decode's instantiation units (one per cache element kind and head size) and the
// 4-bit caches' (decode_fp4.cu).
#pragma once
#include "decode_fp4.cuh"
#include "decode_scored.cuh"
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

// The deepest ring (at most 32 stages, a multiple of the key groups' steps) that lets MINB CTAs share an SM.
template <int D, int KV, int NT, int HG, int W, int KG, int KT, int MINB, int NS = 32>
constexpr int scored_stages() {
  constexpr int unit = KG > 1 ? KG * KT : 1;
  if constexpr (NS <= unit || NS <= 2)
    return unit > 2 ? unit : 2;
  else if constexpr (NS % unit != 0)
    return scored_stages<D, KV, NT, HG, W, KG, KT, MINB, NS - 1>();
  else if constexpr (ScoredCfg<D, KV, NT, HG, W, KG, KT, NS, MINB>::kSmemBytes <= smem_limit(MINB))
    return NS;
  else
    return scored_stages<D, KV, NT, HG, W, KG, KT, MINB, NS - 1>();
}
template <int D, int KV, int NT, int HG, int W, int KG, int KT, int MINB>
using ScoredCfgFor = ScoredCfg<D, KV, NT, HG, W, KG, KT, scored_stages<D, KV, NT, HG, W, KG, KT, MINB>(), MINB>;

template <int D, int KV>
struct ScoredShapes {
  // row tiles, heads per tile, warps per head, key groups, tiles per step, CTAs per SM
  using C1H = ScoredCfgFor<D, KV, 1, 4, 1, 1, 1, 1>;
  using C1 = ScoredCfgFor<D, KV, 1, 1, 1, 3, 1, 2>;
  using C2 = ScoredCfgFor<D, KV, 2, 1, 2, 4, 1, 1>;
  using C3 = ScoredCfgFor<D, KV, 3, 1, 4, 2, 1, 1>;
  using C4 = ScoredCfgFor<D, KV, 4, 1, 4, 2, 1, 1>;

  template <class C>
  static bool shape_one(KernelShape* out) {
    static_assert(C::kSmemBytes <= smem_limit(C::kMinBlocks), "the ring fits");
    out->threads = C::kThreads;
    out->smem_bytes = C::kSmemBytes;
    out->rows_padded = C::RP;
    out->ctas_per_sm = C::kMinBlocks;
    out->heads = C::HG;
    out->step_tiles = C::KG * C::KT;
    out->key_groups = C::KG;
    out->whole_tile = 1;
    out->unit_cost = C::KG > 1 ? 12 : 4;
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
  static bool shape(int nt, int grouped, KernelShape* out) {
    if (grouped) return nt == 1 && shape_one<C1H>(out);
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
