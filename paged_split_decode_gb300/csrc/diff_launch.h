// diff_launch.h -- internal interface between the host layer and the
// differential decode's instantiation units (one per cache element kind).
#pragma once
#include "decode_diff.cuh"
#include "decode_diff_tc.cuh"
#include "launch.h"

namespace pd {

// Shape of the instantiation for (D, cache element kind, ntm row tiles of 8
// query rows per map, grouped); false when there is none.
bool diff_kernel_shape(int D, int kv, int ntm, int grouped, KernelShape* out);
cudaError_t launch_diff(int D, int kv, int ntm, int grouped, const CUtensorMap& tk, const CUtensorMap& tv,
                        const DiffParams& p, int grid, cudaStream_t stream);
cudaError_t launch_diff_combine(int D, const DiffParams& p, int n_units, int row_chunks, int rows_at_once, int groups, bool many,
                                cudaStream_t stream);

bool diff_shape_f16(int D, int ntm, int grouped, KernelShape* out);
bool diff_shape_bf16(int D, int ntm, int grouped, KernelShape* out);
bool diff_shape_fp8(int D, int ntm, int grouped, KernelShape* out);
bool diff_shape_i8(int D, int ntm, int grouped, KernelShape* out);
cudaError_t diff_launch_f16(int D, int ntm, int grouped, const CUtensorMap&, const CUtensorMap&, const DiffParams&,
                            int, cudaStream_t);
cudaError_t diff_launch_bf16(int D, int ntm, int grouped, const CUtensorMap&, const CUtensorMap&, const DiffParams&,
                             int, cudaStream_t);
cudaError_t diff_launch_fp8(int D, int ntm, int grouped, const CUtensorMap&, const CUtensorMap&, const DiffParams&,
                            int, cudaStream_t);
cudaError_t diff_launch_i8(int D, int ntm, int grouped, const CUtensorMap&, const CUtensorMap&, const DiffParams&,
                           int, cudaStream_t);

// The deepest ring (at most 32 stages, a multiple of the key groups' steps) that
// lets MINB CTAs share an SM.
template <int D, int KV, int NTM, int HG, int W, int KG, int KT, int MINB, int NS = 32>
constexpr int diff_stages() {
  constexpr int unit = KG > 1 ? KG * KT : 1;
  if constexpr (NS <= unit || NS <= 2)
    return unit > 2 ? unit : 2;
  else if constexpr (NS % unit != 0)
    return diff_stages<D, KV, NTM, HG, W, KG, KT, MINB, NS - 1>();
  else if constexpr (DiffCfg<D, KV, NTM, HG, W, KG, KT, NS, MINB>::kSmemBytes <= smem_limit(MINB))
    return NS;
  else
    return diff_stages<D, KV, NTM, HG, W, KG, KT, MINB, NS - 1>();
}
template <int D, int KV, int NTM, int HG, int W, int KG, int KT, int MINB>
using DiffCfgFor = DiffCfg<D, KV, NTM, HG, W, KG, KT, diff_stages<D, KV, NTM, HG, W, KG, KT, MINB>(), MINB>;

template <class Cfg>
bool diff_shape_of(KernelShape* out) {
  static_assert(Cfg::kSmemBytes <= smem_limit(Cfg::kMinBlocks), "the ring fits");
  out->threads = Cfg::kThreads;
  out->smem_bytes = Cfg::kSmemBytes;
  out->rows_padded = Cfg::RP;
  out->ctas_per_sm = Cfg::kMinBlocks;
  out->heads = Cfg::HG;
  out->step_tiles = Cfg::KG * Cfg::KT;
  out->key_groups = Cfg::KG;
  out->whole_tile = 1;
  // what a piece's end costs, in tiles: 1 us from the accumulators, 5 us where key
  // groups merge first (measured, D = 256 GQA 6:1, L = 8192, B = 8, qlen = 3, 4 /
  // 10 / 16 / 24 / 48 tiles: fp16 61.0 / 59.2 / 57.2 / 56.8 / 57.5 us; without key
  // groups 4 to 12 tiles are within 1 %)
  out->unit_cost = Cfg::KG > 1 ? 20 : 4;
  out->fixed_pieces = 0;
  for (int& c : out->max_clusters) c = 0;  // split units go through the combine
  return true;
}

template <class Cfg>
cudaError_t diff_launch_cfg(const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p, int grid,
                            cudaStream_t stream) {
  static unsigned long long attr_ctx[64] = {};
  const cudaError_t e =
      once_per_context(attr_ctx, [] { return set_kernel_attributes(decode_diff_kernel<Cfg>, Cfg::kSmemBytes); });
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_diff_kernel<Cfg>, grid, Cfg::kThreads, Cfg::kSmemBytes, stream, 1, tk, tv, p);
}

// The shapes of one cache kind, as measured fastest on GB300 (D = 256 GQA 6:1
// L = 4096 B = 32 unless said):
//  * C1H, one row tile per map and Hkv a multiple of four: a warp per head, four
//    heads a tile, one CTA per SM. Two tiles a step at D = 128 (e4m3, 32 x 8
//    heads, ragged: 108 -> 100 us); at D = 256 two tiles' scores spill (e4m3 54
//    -> 60 us). Two warps per head that swap P took 66 us at e4m3, four 77.
//  * C1, other head counts: per-head tiles, three key groups of one warp on two
//    CTAs per SM (two CTAs' producers: one tile's copies take 0.2 us to issue).
//  * C2 to C4, two to four row tiles per map: four warps a head, two key groups,
//    one CTA per SM; two tiles a step while the fragments fit (qlen = 3, e4m3, L
//    = 8192, B = 8: 69 -> 65 us before those had the tensor-memory engine below).
template <int D, int KV>
struct DiffShapes {
  // row tiles per map, heads per tile, warps per head, key groups, tiles per step, CTAs per SM
  using C1H = DiffCfgFor<D, KV, 1, 4, 1, 1, (D == 128 ? 2 : 1), 1>;
  using C1 = DiffCfgFor<D, KV, 1, 1, 1, 3, 1, 2>;
  using C2 = DiffCfgFor<D, KV, 2, 1, 4, 2, 2, 1>;
  using C3 = DiffCfgFor<D, KV, 3, 1, 4, 2, 2, 1>;
  using C4 = DiffCfgFor<D, KV, 4, 1, 4, 2, 1, 1>;

  // byte caches, two or more row tiles per map, where shared memory holds it: the
  // tensor-memory engine (L = 8192, B = 8, qlen = 2 / 3 / 5: e4m3 45.9 / 58.7 / 76.7
  // here, 33.2 / 35.3 / 44.3 us there, int8 51.4 / 63.4 here, 40.9 / 45.4 there)
  template <class C>
  static constexpr bool kTc = KV == kKvFp8 || (KV == kKvInt8 && (D == 128 || C::NTM < 4));
  template <class C>
  static bool rows_shape(KernelShape* out) {
    if constexpr (kTc<C>) return diff_tc_shape_of<DiffTc<D, KV, C::NTM>>(out);
    else return diff_shape_of<C>(out);
  }
  template <class C>
  static cudaError_t rows_launch(const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p, int grid,
                                 cudaStream_t s) {
    if constexpr (kTc<C>) return launch_diff_tc<DiffTc<D, KV, C::NTM>>(tk, tv, p, grid, s);
    else return diff_launch_cfg<C>(tk, tv, p, grid, s);
  }

  static bool shape(int ntm, int grouped, KernelShape* out) {
    if (grouped) return ntm == 1 && diff_shape_of<C1H>(out);
    switch (ntm) {
      case 1: return diff_shape_of<C1>(out);
      case 2: return rows_shape<C2>(out);
      case 3: return rows_shape<C3>(out);
      case 4: return rows_shape<C4>(out);
      default: return false;
    }
  }
  static cudaError_t launch(int ntm, int grouped, const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p,
                            int grid, cudaStream_t s) {
    if (grouped) return ntm == 1 ? diff_launch_cfg<C1H>(tk, tv, p, grid, s) : cudaErrorInvalidValue;
    switch (ntm) {
      case 1: return diff_launch_cfg<C1>(tk, tv, p, grid, s);
      case 2: return rows_launch<C2>(tk, tv, p, grid, s);
      case 3: return rows_launch<C3>(tk, tv, p, grid, s);
      case 4: return rows_launch<C4>(tk, tv, p, grid, s);
      default: return cudaErrorInvalidValue;
    }
  }
};

}  // namespace pd
