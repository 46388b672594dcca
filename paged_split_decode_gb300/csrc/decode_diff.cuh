// decode_diff.cuh -- differential decode over the paged caches for sm_103a.
//
// Computes, for every sequence, query token and query head h, with q and K
// rows of two halves q1|q2 and k1|k2,
//   out = softmax(c q1 . k1) V - lambda_h softmax(c q2 . k2) V,
// optionally followed by the head's root-mean-square norm
//   out * rsqrt(mean(out^2) + eps) * weight * gain,
// over caches laid out as the plain decode's. HBM-bound: K and V are read once
// (2 L Hkv D elements) for 6 L Hq D flops per query token.
//
// The decode's structure is kept (decode_kernel.cuh: persistent CTAs over
// balanced ranges of 16-key tiles, one TMA producer warp, a ring of
// 128B-swizzled stages, S^T = K Q^T and O^T = V^T P^T with mma.sync, bounded
// waits). What differs is what the two maps make possible: a half of a K row
// belongs to one map only, so the two maps' scores cost one pass over K, and
// both maps' P meet the same V fragments: every K and V byte is read from
// shared memory, and a one-byte code widened, once for both maps.
//  * W = 1: a warp serves a head alone (both maps, all of V's dims): no
//    exchange between warps at all. KT = 2 takes two tiles a step, which halves
//    the shuffles and gives the tensor pipe independent chains.
//  * W = 4 (more row tiles than one warp's registers hold): warp (map m, row
//    group h) scores map m for its row tiles over that map's whole
//    contraction (no partial scores to add), and the four swap their packed
//    P fragments (8 bytes per lane, tile and row tile, one
//    barrier per step); each warp accumulates both maps over a quarter of V's dims.
//  * KG key groups of such warps take the ring's steps in turn and merge their
//    (m, l, O) through shared memory at the end of a piece.
// A tile is one box of a 4-D tensor map that puts keys before heads: a head's
// 16 keys are 16 adjacent 128-byte rows of a slab and meet all eight swizzle
// phases whatever the heads per tile.
//
// A unit covered by one piece is finished here, the difference and the norm in
// fp32; a split unit's pieces write fp32 (m, l, O) partials of both maps, which
// diff_combine_kernel joins.
#pragma once
#include <cuda_bf16.h>

#include <type_traits>

#include "decode_kernel.cuh"

namespace pd {

struct DiffParams {
  DecodeParams d;
  const void* v_cache;      // V beside its tensor map (for the rare look at single elements)
  const float* lambda;      // [Hq]
  const void* norm_weight;  // [D] or null
  int norm_f32;             // norm_weight is fp32 (else q's type)
  float norm_eps, norm_gain;
};

template <int D_, int KV_, int NTM_, int HG_, int W_, int KG_, int KT_, int NS_, int MINB_>
struct DiffCfg {
  static constexpr int D = D_, KV = KV_, NTM = NTM_, HG = HG_, W = W_, KG = KG_, KT = KT_, NS = NS_;
  static constexpr int kMinBlocks = MINB_;
  static constexpr bool BYTE = KV == kKvFp8 || KV == kKvInt8;
  static constexpr bool BF16 = KV == kKvBf16;  // bfloat16 operands; byte kinds use fp16 ones
  static constexpr int kElem = BYTE ? 1 : 2;
  static constexpr int kSlabElems = 128 / kElem;
  static constexpr int kSlabs = D / kSlabElems;
  static constexpr int kHeadBytes = kTileKeys * 128;  // one head's keys of a slab
  static constexpr int kSlabBytes = HG * kHeadBytes;  // [head][key][128 B]
  static constexpr int kTileBytes = kSlabs * kSlabBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  // 16-bit caches, up to 16 query rows per map: P is carried as the sum of two
  // operands (the rounded value and the rounded rest), which makes the output as
  // exact as one rounding allows (error against 64 bits, relative to its norm: fp16
  // 2.1e-4, bfloat16 1.66e-3, as in 32 bits throughout). Elsewhere P is rounded to the
  // operands' type once (fp16 3.2e-4, bfloat16 2.5e-3; byte caches, whose operands are
  // fp16, 3.2e-4 under an fp16 q, 1.69e-3 under a bfloat16 one): the second products
  // cost 2 % with two row tiles (qlen = 2, B = 8, L = 8192, D = 256: 50.0 -> 51.1 us), 26
  // and 30 % with three and four (56.1 -> 71.0, 74.6 -> 97.1), 28 % over byte caches
  // with one (e4m3, B = 32, L = 4096: 53.8 -> 69.8).
  static constexpr int PP = !BYTE && NTM <= 2 ? 2 : 1;
  static constexpr int MPW = W == 1 ? 2 : 1;             // maps a warp scores
  static constexpr int RG = W == 4 ? 2 : 1;              // row groups
  static constexpr int NTR = (NTM + RG - 1) / RG;        // row tiles (per map) a warp scores
  static constexpr int kGroupWarps = HG * W;             // warps of a key group
  static constexpr int kConsumerWarps = kGroupWarps * KG;
  static constexpr int kConsumerThreads = kConsumerWarps * 32;
  // Eight consumer warps alone on an SM take the registers that the producer's
  // warpgroup gives up (256 x 216 + 128 x 56 of the launch's 384 x 168).
  static constexpr bool kSplitRegs = kConsumerWarps == 8 && MINB_ == 1;
  static constexpr int kThreads = kConsumerThreads + (kSplitRegs ? 128 : 32);
  static constexpr int RM = NTM * 8;      // partial rows per map of a head
  static constexpr int RH = 2 * RM;       // per head
  static constexpr int RP = HG * RH;      // per unit
  static constexpr bool kMerge = KG > 1;                 // the epilogue goes through shared memory
  static constexpr int kDP = D + 4;                      // merge row pitch (floats)
  static constexpr int kMergeO = kMerge ? RP * kDP * 4 : 0;
  static constexpr int kMergeML = kMerge ? KG * RP * 8 : 0;
  // a head's exchange, double-buffered: packed P [map][row tile][lane], rescale
  // factors [map][row tile][row], a flag per warp
  static constexpr int kXTiles = 2 * RG * NTR;
  static constexpr int kXPlane = kXTiles * 32 * 8 * KT;
  static constexpr int kXP = kXPlane * PP;
  static constexpr int kXOne = kXP + kXTiles * 8 * 4 + 16;
  static constexpr int kXHead = 2 * kXOne;
  static constexpr int kX = W > 1 ? HG * KG * kXHead : 0;
  static constexpr int kOffMergeML = NS * kStageBytes + kMergeO;
  static constexpr int kOffX = kOffMergeML + kMergeML;
  static constexpr int kOffBars = kOffX + kX;
  static constexpr int kOffPre = kOffBars + 2 * NS * 8;
  static constexpr int kSmemBytes = (kOffPre + (kMaxAutoB + 1) * 4 + 15) / 16 * 16 + 1024;
  // a stage always belongs to the same key group (see Cfg), which takes KT
  // consecutive ring positions a step
  static_assert(KG == 1 || NS % (KG * KT) == 0, "ring stages must be a multiple of the key groups' steps");
  static_assert(KT == 1 || KT == 2, "one or two tiles a step");
  static_assert(W == 1 || W == 4, "one or four warps per head");
  // the straight epilogue has no exchange between a head's warps, and no barrier
  // that keeps a fast warp's next piece out of the buffers that a slow one still reads
  static_assert(W == 1 || kMerge, "a head's warps end a piece in the merge's barriers");
  static_assert(HG * KG <= 14, "named barriers 2.. serve the heads' warps");
};

__device__ __forceinline__ float norm_weight_at(const DiffParams& p, int d) {
  if (p.norm_f32) return __ldg(static_cast<const float*>(p.norm_weight) + d);
  const uint16_t w = __ldg(static_cast<const uint16_t*>(p.norm_weight) + d);
  return p.d.out_bf16 ? __uint_as_float(static_cast<uint32_t>(w) << 16) : __half2float(__ushort_as_half(w));
}

// x rounded to the 16-bit operand type.
template <bool BF16>
__device__ __forceinline__ float round16(float x) {
  if constexpr (BF16) return __bfloat162float(__float2bfloat16_rn(x));
  else return __half2float(__float2half_rn(x));
}

__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A map's output where its sum of weights l is a positive number, else nothing: a
// map without a visible key, or with a NaN among its scores, contributes zeros.
__device__ __forceinline__ float map_out(float l, float o) { return l > 0.f ? o : 0.f; }

__device__ __forceinline__ uint32_t pack_out(bool bf16, float lo, float hi) {
  return bf16 ? pack_bf162(lo, hi) : pack_half2(lo, hi);
}

// The factor of a row of D elements whose squares sum to ss. (A row of zeros with eps =
// 0 stays zero; one with a NaN is NaN throughout, its zeros too.)
template <int D>
__device__ __forceinline__ float norm_factor(const DiffParams& p, float ss) {
  const float t = ss / static_cast<float>(D) + p.norm_eps;
  return t == 0.f ? 0.f : rsqrtf(t) * p.norm_gain;
}

// Four dims d .. d + 3 of an output row, normalised by f where there is a norm.
__device__ __forceinline__ void store_row4(const DiffParams& p, uint16_t* dst, int d, float4 v, float f) {
  if (p.norm_weight != nullptr) {
    v.x *= f * norm_weight_at(p, d);
    v.y *= f * norm_weight_at(p, d + 1);
    v.z *= f * norm_weight_at(p, d + 2);
    v.w *= f * norm_weight_at(p, d + 3);
  }
  const bool bf = p.d.out_bf16 != 0;
  *reinterpret_cast<uint2*>(dst + d) = make_uint2(pack_out(bf, v.x, v.y), pack_out(bf, v.z, v.w));
}

// NaN and infinities in V of keys that not every row of a unit sees -- the newest
// keys under several query tokens, those about a window's start -- would reach the
// rows that do not see them, whose weight of zero times them is NaN. Such keys are
// in a unit's first and last tiles only: there they are taken out of the product's
// operand, and a piece that had one marks the outputs of the rows that see it at its
// end.

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, Cfg::kMinBlocks)
    decode_diff_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const DiffParams dp) {
  const DecodeParams& p = dp.d;
  constexpr int D = Cfg::D, NS = Cfg::NS, NTM = Cfg::NTM;
  constexpr bool BYTE = Cfg::BYTE, BF16 = Cfg::BF16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);  // full[NS], empty[NS]
  int* s_pre = reinterpret_cast<int*>(smem + Cfg::kOffPre);
  // (what a warp's branches depend on is broadcast, so that they compile to
  // uniform ones without reconvergence around the matrix instructions)
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const bool is_producer = warp == Cfg::kConsumerWarps;
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + NS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, Cfg::kGroupWarps);
    }
    fence_mbar_init();
  }
  if (is_producer && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // nothing above touches global memory (programmatic dependent launch)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.num_splits == 0 && warp == 0) balanced_prefix(p, s_pre, lane);
  __syncthreads();

  WorkIter it;
  work_init(p, s_pre, it);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Piece pc;

  if constexpr (Cfg::kSplitRegs) {
    if (warp < Cfg::kConsumerWarps) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (!is_producer) return;  // the rest of the producer's warpgroup
    }
  }
  if (is_producer) {
    // One elected lane issues two copies a tile, K and V, each one box of the 4-D map
    // (128 bytes, 16 keys, HG heads, all slabs): copies issued by several lanes
    // are serialised, which at four to eight boxes a tile held the ring back.
    // Each lane translates its own of the next 32 tiles.
    const uint64_t pol = l2_policy_evict_first();
    uint32_t q = 0, issued = 0;
    bool ok = true;
    while (work_next(p, s_pre, it, pc)) {
      if (pc.ntiles == 0) continue;
      const int32_t* row = p.block_table + static_cast<long long>(pc.b) * p.max_blocks;
      auto load_group = [&](int t) -> int {  // lane i: physical block of tile t + i
        int blk = 0;
        if (t + lane < pc.ntiles) blk = __ldg(row + (pc.first_tile + t + lane) / p.tiles_per_block);
        return blk;
      };
      int cur = load_group(0);
      for (int t = 0; t < pc.ntiles; t += 32) {
        const int nxt = (t + 32 < pc.ntiles) ? load_group(t + 32) : 0;
        const int n = min(32, pc.ntiles - t);
        if (cur < 0 || cur >= p.num_blocks) {
          raise_error(p.error_flag, kErrBlockId);
          cur = 0;
        }
        const int row0 = cur * p.block_size + ((pc.first_tile + t + lane) % p.tiles_per_block) * kTileKeys;
        for (int i = 0; i < n; ++i, ++q) {
          const int z = __shfl_sync(0xffffffffu, row0, i);
          if (elect_one()) {
            const int stage = q % NS;
            const uint32_t fb = full0 + 8 * stage;
            if (ok && q >= NS) ok = mbar_wait(empty0 + 8 * stage, ((q / NS) - 1) & 1, p.timeout_ns);
            if (ok && p.inject == 1) ok = false;
            if (ok) {
              mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
              const uint32_t dst = smem_u32(smem + stage * Cfg::kStageBytes);
              tma_load_4d(dst, &tm_k, fb, 0, z, pc.kh, 0, pol);
              tma_load_4d(dst + Cfg::kTileBytes, &tm_v, fb, 0, z, pc.kh, 0, pol);
              issued = q + 1;
            }
          }
        }
        cur = nxt;
      }
    }
    if (elect_one()) {
      if (!ok) raise_error(p.error_flag, kErrTimeout);
      // every issued load lands before the CTA's shared memory is released
      const uint32_t first = issued > NS ? issued - NS : 0;
      for (uint32_t k = first; k < issued; ++k)
        if (!mbar_wait(full0 + 8 * (k % NS), (k / NS) & 1, kDrainLimitNs)) break;
    }
    __syncwarp();
    return;
  }

  // -------------------------------------------------------------- consumers
  constexpr int W = Cfg::W, KG = Cfg::KG, KT = Cfg::KT, HG = Cfg::HG, MPW = Cfg::MPW, NTR = Cfg::NTR;
  const int w = warp % W;                    // warp of the head: its 1 / W of V's dims
  const int kg = (warp / W) % KG;            // key group
  const int th = warp / (W * KG);            // head of the tile
  const int map = w & 1, rt0 = (w >> 1) * NTR;  // W > 1: the map and first row tile it scores
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int KSW = D / 32;                // k-steps of one map (D / 2 dims)
  constexpr int MTW = D / 16 / W;            // m-tiles of 16 output dims of this warp
  float* merge_o = reinterpret_cast<float*>(smem + NS * Cfg::kStageBytes);
  float* merge_ml = reinterpret_cast<float*>(smem + Cfg::kOffMergeML);
  const uint32_t smem0 = smem_u32(smem);
  const uint32_t xch = smem0 + Cfg::kOffX + (th * KG + kg) * Cfg::kXHead;
  // One-byte tiles: 16-byte chunk 4 s + t4 of a 64-dim super-step s. The eight
  // lanes of a shared-memory phase hold two accumulator rows of four chunks, so
  // rows 2i and 2i + 1 stand for keys whose swizzle phases differ by 4; and the
  // four keys that a V read touches (rows 2 t4) differ in their phases' upper
  // two bits: no bank conflict on either.
  auto key_of = [](int r) { return BYTE ? static_cast<int>((0x37621540u >> (4 * r)) & 15u) : r; };
  const int kg0 = key_of(g);                 // key of accumulator row g (row g + 8: + 8)
  // Per-lane offsets within a stage. 16-bit: the row that this lane addresses for
  // ldmatrix (K; V transposed) with the swizzled chunk of k-step (m-tile) 0; that
  // of step s is 32 s away by exclusive or, since the rows are 128-byte aligned.
  // One-byte: row key_of(g) with chunk t4 of super-step 0 (64 s away by exclusive
  // or); V's two keys (and those + 8) with the first chunk of the 32-dim group.
  uint32_t k_off, v_off[2];
  if constexpr (!BYTE) {
    const int kk = lane & 15, kv = (lane & 7) + (lane >> 4) * 8;
    k_off = th * Cfg::kHeadBytes + kk * 128 + (((lane >> 4) ^ (kk & 7)) << 4);
    v_off[0] = Cfg::kTileBytes + th * Cfg::kHeadBytes + kv * 128 + ((((lane >> 3) & 1) ^ (kv & 7)) << 4);
  } else {
    k_off = th * Cfg::kHeadBytes + kg0 * 128 + ((t4 ^ (kg0 & 7)) << 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int kv = key_of(2 * t4 + i);
      v_off[i] = Cfg::kTileBytes + th * Cfg::kHeadBytes + kv * 128 + (((g >> 2) ^ (kv & 7)) << 4) + ((4 * g) & 15);
    }
  }
  // a negative score factor is taken as a positive one on -q; a factor of zero
  // as one too small to matter, so that a masked score (-inf) stays -inf
  const float sl2 = fmaxf(fabsf(p.sl2), 1e-30f);
  const uint32_t flip = p.sl2 < 0.f ? 0x80008000u : 0u;
  uint32_t qf[MPW][KSW][NTR][2];
  float o[2][MTW][NTM][4];
  uint32_t q = 0;                            // ring position of the piece's first tile
  bool ok = true;

  while (uniform(work_next(p, s_pre, it, pc))) {
    const int ntiles = uniform(pc.ntiles), first_tile = uniform(pc.first_tile), seq_len = uniform(pc.L);
    const int lo_all = uniform(pc.tile_lo_all), hi_all = uniform(pc.tile_hi_all);
    constexpr bool kScreen = Cfg::KV != kKvInt8;
    const int screen_hi = pc.qlen > 1 ? hi_all : 0x7fffffff;
    uint32_t odd = 0;                        // elements that were taken out
    // ---- q fragments of the rows and maps this warp scores
    float sl2r[MPW][NTR][2];                 // score factors (log2 units), positive
    int hi_r[NTR][2];                        // last visible key of a row
    float m_r[MPW][NTR][2], l_r[MPW][NTR][2];  // reference maxima (scaled) and sums
#pragma unroll
    for (int n = 0; n < NTR; ++n) {
      const int r = (rt0 + n) * 8 + g;
      const __half* qrow = nullptr;
      if (r < pc.R && pc.ntiles > 0) {
        const int i = r / p.G, hl = r % p.G;
        qrow = p.q + (static_cast<long long>(pc.q0 + i) * p.Hq + (pc.kh + th) * p.G + hl) * D;
      }
#pragma unroll
      for (int m = 0; m < MPW; ++m) {
        sl2r[m][n][0] = sl2r[m][n][1] = sl2;
        m_r[m][n][0] = m_r[m][n][1] = -INFINITY;
        l_r[m][n][0] = l_r[m][n][1] = 0.f;
        const int half = (W == 1 ? m : map) * (D / 2);
#pragma unroll
        for (int ks = 0; ks < KSW; ++ks) {
          const int d0 = half + (BYTE ? 64 * (ks >> 2) + 16 * t4 + 4 * (ks & 3) : ks * 16 + 2 * t4);
          const int d1 = d0 + (BYTE ? 2 : 8);
          qf[m][ks][n][0] = qrow ? __ldg(reinterpret_cast<const uint32_t*>(qrow + d0)) ^ flip : 0u;
          qf[m][ks][n][1] = qrow ? __ldg(reinterpret_cast<const uint32_t*>(qrow + d1)) ^ flip : 0u;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rc = (rt0 + n) * 8 + 2 * t4 + c;
        hi_r[n][c] = pc.L - pc.qlen + rc / p.G;  // (padded rows: q = 0, never written)
      }
    }
    if constexpr (BYTE) {
      if (p.out_bf16) {
        // bfloat16 q over byte caches: the half row scaled by 2^e into fp16,
        // exactly; 2^-e joins the row's score factor
#pragma unroll
        for (int m = 0; m < MPW; ++m)
#pragma unroll
          for (int n = 0; n < NTR; ++n) {
            float mx = 0.f;
#pragma unroll
            for (int ks = 0; ks < KSW; ++ks)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t v = qf[m][ks][n][h];
                mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(v << 16)), fabsf(__uint_as_float(v & 0xffff0000u))));
              }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int e = q_row_exponent(mx);
            sl2r[m][n][0] = fmaxf(sl2 * pow2f(-__shfl_sync(0xffffffffu, e, 8 * t4)), 0x1p-126f);
            sl2r[m][n][1] = fmaxf(sl2 * pow2f(-__shfl_sync(0xffffffffu, e, 8 * t4 + 4)), 0x1p-126f);
            const float up = pow2f(e);
#pragma unroll
            for (int ks = 0; ks < KSW; ++ks)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t v = qf[m][ks][n][h];
                qf[m][ks][n][h] = pack_half2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xffff0000u) * up);
              }
          }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int mt = 0; mt < MTW; ++mt)
#pragma unroll
        for (int n = 0; n < NTM; ++n) o[m][mt][n][0] = o[m][mt][n][1] = o[m][mt][n][2] = o[m][mt][n][3] = 0.f;

    // ---- this key group's steps: KT ring positions each, dealt to the groups
    // by ring position (a piece may start or end inside a step)
    const int lead = KG > 1 && KT > 1 ? static_cast<int>(q % KT) : 0;
    const uint32_t step0 = (q - lead) / KT;
    // (a piece without tiles has no step, not even the one that it would start in:
    // that one's stage is not its to give back)
    const int last = ntiles > 0 ? ntiles + lead : 0;
    // A step is compiled twice: for tiles that every row sees whole, and for the others
    // (EDGE: masks, values, a missing tile), so that the common one has no branch (B = 32,
    // L = 4096, D = 256: int8 61.0 -> 57.8 us, e4m3 53.8 -> 53.2; fp16, qlen = 3, B = 8, L =
    // 8192: 56.6 before values were looked at, 58.0 so, 62.6 in one copy). int8 caches have
    // no values to look at, and four warps a head gain nothing there.
    auto step = [&](const int st, auto edge_step) __attribute__((always_inline)) {
      constexpr bool EDGE = decltype(edge_step)::value;
      const int k0 = st * KT - lead;
      bool have[KT];
      int tile[KT];  // a step's missing tile is its other one over again, masked: no branch splits the step
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        have[j] = !EDGE || (k0 + j >= 0 && k0 + j < ntiles);
        if (ok && have[j])
          ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * ((q + k0 + j) % NS), ((q + k0 + j) / NS) & 1, p.timeout_ns));
      }
#pragma unroll
      for (int j = 0; j < KT; ++j) tile[j] = have[j] ? k0 + j : k0 + (KT - 1 - j);
      if (!ok) {  // gave up: keep the head's barrier sequence
        if constexpr (W > 1) named_bar_sync(2 + th * KG + kg, W * 32);
        return;
      }
      constexpr int PP = Cfg::PP;
      uint32_t pf[KT][2][NTM][2 * PP];  // P^T fragments of both maps
      float x[KT][MPW][NTR][4];    // raw scores
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        // ---- S^T: 16 keys x 8 rows per row tile and map
        const uint32_t ka = smem0 + ((q + tile[j]) % NS) * Cfg::kStageBytes + k_off;
        float sa[MPW][NTR][4], sb[MPW][NTR][4];
#pragma unroll
        for (int m = 0; m < MPW; ++m)
#pragma unroll
          for (int n = 0; n < NTR; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sa[m][n][e] = sb[m][n][e] = 0.f;
        if constexpr (!BYTE) {
          // (KSW is 4 or 8: a map's k-steps start a slab)
#pragma unroll
          for (int m = 0; m < MPW; ++m) {
            const uint32_t km = ka + (W == 1 ? m : map) * (KSW / 4) * Cfg::kSlabBytes;
#pragma unroll
            for (int ksl = 0; ksl < KSW; ++ksl) {
              uint32_t a[4];
              ldsm_x4((km ^ ((ksl & 3) * 32)) + (ksl >> 2) * Cfg::kSlabBytes, a);
#pragma unroll
              for (int n = 0; n < NTR; ++n) {
                if (ksl & 1) mma_op<BF16>(sb[m][n], a, qf[m][ksl][n][0], qf[m][ksl][n][1]);
                else mma_op<BF16>(sa[m][n], a, qf[m][ksl][n][0], qf[m][ksl][n][1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int m = 0; m < MPW; ++m)
#pragma unroll
            for (int sup = 0; sup < KSW / 4; ++sup) {
              // 64-dim super-steps: two a slab
              const uint32_t half = static_cast<uint32_t>(W == 1 ? m : map);
              const uint32_t at = D == 256 ? (ka ^ (sup * 64)) + half * Cfg::kSlabBytes : ka ^ (half * 64);
              const uint4 w0 = lds_v4_tile(at), w8 = lds_v4_tile(at + 8 * 128);
              const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w};
              const uint32_t wb[4] = {w8.x, w8.y, w8.z, w8.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int ksl = sup * 4 + i;
                uint32_t a[4];
                const uint32_t xa = byte_word_prep<Cfg::KV>(wa[i]), xb = byte_word_prep<Cfg::KV>(wb[i]);
                a[0] = byte_pair_to_half2<Cfg::KV>(xa, false);
                a[1] = byte_pair_to_half2<Cfg::KV>(xb, false);
                a[2] = byte_pair_to_half2<Cfg::KV>(xa, true);
                a[3] = byte_pair_to_half2<Cfg::KV>(xb, true);
#pragma unroll
                for (int n = 0; n < NTR; ++n) {
                  if (i & 1) mma_op<BF16>(sb[m][n], a, qf[m][ksl][n][0], qf[m][ksl][n][1]);
                  else mma_op<BF16>(sa[m][n], a, qf[m][ksl][n][0], qf[m][ksl][n][1]);
                }
              }
            }
        }
        const int key0 = (first_tile + tile[j]) * kTileKeys;
        const bool interior = !EDGE || (have[j] && key0 >= lo_all && key0 + kTileKeys - 1 <= hi_all);
        const int j0 = key0 + kg0, j1 = j0 + 8;
#pragma unroll
        for (int n = 0; n < NTR; ++n) {
#pragma unroll
          for (int m = 0; m < MPW; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][m][n][e] = sa[m][n][e] + sb[m][n][e];
          if (!interior) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int hi = have[j] ? hi_r[n][c] : -1, lo = p.window > 0 ? hi - p.window + 1 : 0;
#pragma unroll
              for (int m = 0; m < MPW; ++m) {
                if (j0 < lo || j0 > hi) x[j][m][n][c] = -INFINITY;
                if (j1 < lo || j1 > hi) x[j][m][n][2 + c] = -INFINITY;
              }
            }
          }
        }
      }
      // ---- online softmax. P = 2^(x sl2 - m + kUp) is relative to a reference m that
      // is raised to the running maximum only when a score passes it by more than
      // 2^kLazy: P stays within the 16-bit operands' range (at most 2^15), the
      // result does not depend on m, and the common step needs no shuffle, no
      // rescaling and, between warps, no factors. 2^kUp moves fp16's last bit from
      // 2^-24 to 2^-31 of the reference's weight: in a map with one key 16 nats above
      // 32767 others a tenth of a percent was lost below it. (l and O carry the factor,
      // in every piece; their quotient does not.)
      constexpr float kLazy = 8.f, kUp = 15.f - kLazy;
      bool raise = false;
#pragma unroll
      for (int m = 0; m < MPW; ++m)
#pragma unroll
        for (int n = 0; n < NTR; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(x[0][m][n][c], x[0][m][n][2 + c]);
            if constexpr (KT > 1) mx = fmaxf(mx, fmaxf(x[KT - 1][m][n][c], x[KT - 1][m][n][2 + c]));
            raise |= fmaf(mx, sl2r[m][n][c], -m_r[m][n][c]) > kLazy;  // (no key seen: m = -inf)
          }
      raise = __any_sync(0xffffffffu, raise);
      const uint32_t xcur = xch + (static_cast<uint32_t>(st / KG) & 1u) * Cfg::kXOne;
      const uint32_t xa = xcur + Cfg::kXP, flags = xa + Cfg::kXTiles * 32;
      if (raise) {
#pragma unroll
        for (int m = 0; m < MPW; ++m)
#pragma unroll
          for (int n = 0; n < NTR; ++n) {
            float al[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = fmaxf(x[0][m][n][c], x[0][m][n][2 + c]);
              if constexpr (KT > 1) mx = fmaxf(mx, fmaxf(x[KT - 1][m][n][c], x[KT - 1][m][n][2 + c]));
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
              const float old = m_r[m][n][c], mn = fmaxf(old, mx * sl2r[m][n][c]);
              // nothing accumulated yet: O and l are zero, keep factor 1
              al[c] = old == -INFINITY ? 1.f : ex2(old - mn);
              m_r[m][n][c] = mn;
              l_r[m][n][c] *= al[c];
            }
            if constexpr (W == 1) {
#pragma unroll
              for (int mt = 0; mt < MTW; ++mt) {
                o[m][mt][n][0] *= al[0]; o[m][mt][n][1] *= al[1];
                o[m][mt][n][2] *= al[0]; o[m][mt][n][3] *= al[1];
              }
            } else if (g == 0) {
              sts_f2(xa + (map * Cfg::RG * NTR + rt0 + n) * 32 + 8 * t4, al[0], al[1]);
            }
          }
      }
      // P rounded to the operands' 16-bit type (tensor-core products), the sum
      // l of the unrounded exponentials
#pragma unroll
      for (int m = 0; m < MPW; ++m)
#pragma unroll
        for (int n = 0; n < NTR; ++n) {
          float nb[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) nb[c] = m_r[m][n][c] == -INFINITY ? 0.f : kUp - m_r[m][n][c];
          uint32_t pk[KT][2 * PP];
#pragma unroll
          for (int j = 0; j < KT; ++j) {
            const float p00 = ex2(fmaf(x[j][m][n][0], sl2r[m][n][0], nb[0]));
            const float p01 = ex2(fmaf(x[j][m][n][1], sl2r[m][n][1], nb[1]));
            const float p10 = ex2(fmaf(x[j][m][n][2], sl2r[m][n][0], nb[0]));
            const float p11 = ex2(fmaf(x[j][m][n][3], sl2r[m][n][1], nb[1]));
            l_r[m][n][0] += p00 + p10;
            l_r[m][n][1] += p01 + p11;
            pk[j][0] = movmatrix_trans(pack2<BF16>(p00, p01));
            pk[j][1] = movmatrix_trans(pack2<BF16>(p10, p11));
            if constexpr (PP == 2) {
              pk[j][PP] = movmatrix_trans(pack2<BF16>(p00 - round16<BF16>(p00), p01 - round16<BF16>(p01)));
              pk[j][PP + 1] = movmatrix_trans(pack2<BF16>(p10 - round16<BF16>(p10), p11 - round16<BF16>(p11)));
            }
            if constexpr (W == 1) {
#pragma unroll
              for (int i = 0; i < 2 * PP; ++i) pf[j][m][n][i] = pk[j][i];
            }
          }
          if constexpr (W > 1) {
            const uint32_t at = xcur + ((map * Cfg::RG * NTR + rt0 + n) * 32 + lane) * 8 * KT;
#pragma unroll
            for (int h = 0; h < PP; ++h) {
              if constexpr (KT == 1) sts_v2(at + h * Cfg::kXPlane, pk[0][2 * h], pk[0][2 * h + 1]);
              else sts_v4(at + h * Cfg::kXPlane, pk[0][2 * h], pk[0][2 * h + 1], pk[KT - 1][2 * h], pk[KT - 1][2 * h + 1]);
            }
          }
        }
      if constexpr (W > 1) {
        if (lane == 0) sts_b32(flags + 4 * w, raise ? 1u : 0u);
        named_bar_sync(2 + th * KG + kg, W * 32);
        const uint4 fl = lds_v4(flags);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NTM; ++n) {
            const uint32_t at = xcur + ((m * Cfg::RG * NTR + n) * 32 + lane) * 8 * KT;
#pragma unroll
            for (int h = 0; h < PP; ++h) {
              if constexpr (KT == 1) {
                const uint2 v = lds_v2(at + h * Cfg::kXPlane);
                pf[0][m][n][2 * h] = v.x;
                pf[0][m][n][2 * h + 1] = v.y;
              } else {
                const uint4 v = lds_v4(at + h * Cfg::kXPlane);
                pf[0][m][n][2 * h] = v.x;
                pf[0][m][n][2 * h + 1] = v.y;
                pf[KT - 1][m][n][2 * h] = v.z;
                pf[KT - 1][m][n][2 * h + 1] = v.w;
              }
            }
          }
        if (uniform(fl.x | fl.y | fl.z | fl.w)) {
          const uint32_t of[4] = {fl.x, fl.y, fl.z, fl.w};
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NTM; ++n) {
              if (of[(m + 2 * (n / NTR)) % W] == 0u) continue;
              const float2 al = lds_f2(xa + (m * Cfg::RG * NTR + n) * 32 + 8 * t4);
#pragma unroll
              for (int mt = 0; mt < MTW; ++mt) {
                o[m][mt][n][0] *= al.x; o[m][mt][n][1] *= al.y;
                o[m][mt][n][2] *= al.x; o[m][mt][n][3] *= al.y;
              }
            }
        }
      }

      // ---- O^T += V^T P^T of both maps over this warp's dims; V of keys at or
      // past the sequence end is zeroed (its bits may be NaN)
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        const uint32_t stage = (q + tile[j]) % NS, sbase = smem0 + stage * Cfg::kStageBytes;
        const int key0 = (first_tile + tile[j]) * kTileKeys;
        const bool tail = EDGE && key0 + kTileKeys > seq_len;
        const bool screen = EDGE && kScreen && (key0 < lo_all || key0 + kTileKeys - 1 > screen_hi);
        auto screened = [&](uint32_t (&a)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t bad = not_finite_16<BF16>(a[i]);
            odd |= bad;
            a[i] &= ~bad;
          }
        };
        if constexpr (!BYTE) {
          // this warp's m-tiles: a part of a slab's four, or whole slabs
          const uint32_t va = (sbase + v_off[0] + (MTW >= 4 ? w * (MTW / 4) * Cfg::kSlabBytes : (w * MTW >> 2) * Cfg::kSlabBytes)) ^
                              (MTW >= 4 ? 0 : (w * MTW & 3) * 32);
          uint32_t vm01 = 0xffffffffu, vm23 = 0xffffffffu;
          if (tail) {
            const int kt = key0 + 2 * t4;
            vm01 = (kt < seq_len ? 0x0000ffffu : 0u) | (kt + 1 < seq_len ? 0xffff0000u : 0u);
            vm23 = (kt + 8 < seq_len ? 0x0000ffffu : 0u) | (kt + 9 < seq_len ? 0xffff0000u : 0u);
          }
#pragma unroll
          for (int mtl = 0; mtl < MTW; ++mtl) {
            uint32_t a[4];
            ldsm_x4_trans((va ^ ((mtl & 3) * 32)) + (mtl >> 2) * Cfg::kSlabBytes, a);
            if (tail) {
              a[0] &= vm01; a[1] &= vm01; a[2] &= vm23; a[3] &= vm23;
            }
            if (screen) screened(a);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NTM; ++n)
#pragma unroll
                for (int h = 0; h < PP; ++h) mma_op<BF16>(o[m][mtl][n], a, pf[j][m][n][2 * h], pf[j][m][n][2 * h + 1]);
          }
        } else {
          // 32-dim group P32: lane reads 4 codes at dims 32 P32 + 4 g of keys
          // key_of(2 t4), key_of(2 t4 + 1) and those + 8; m-tile 2 P32 takes
          // dims 4 g (row g) and 4 g + 1 (row g + 8), m-tile 2 P32 + 1 the next two
          const int kA = key_of(2 * t4), kB = key_of(2 * t4 + 1), kC = kA + 8, kD = kB + 8;
#pragma unroll
          for (int pl = 0; pl < MTW / 2; ++pl) {
            const int P32 = w * (MTW / 2) + pl;
            const uint32_t x32 = (P32 & 3) * 32, slab = sbase + (P32 >> 2) * Cfg::kSlabBytes;
            const uint32_t vA = slab + (v_off[0] ^ x32), vB = slab + (v_off[1] ^ x32);
            uint32_t wA = lds_b32_tile(vA), wB = lds_b32_tile(vB);
            uint32_t wC = lds_b32_tile(vA + 8 * 128), wD = lds_b32_tile(vB + 8 * 128);
            if (tail) {  // code 0 is the value 0 in both byte formats
              if (key0 + kA >= seq_len) wA = 0u;
              if (key0 + kB >= seq_len) wB = 0u;
              if (key0 + kC >= seq_len) wC = 0u;
              if (key0 + kD >= seq_len) wD = 0u;
            }
            wA = byte_word_prep<Cfg::KV>(wA); wB = byte_word_prep<Cfg::KV>(wB);
            wC = byte_word_prep<Cfg::KV>(wC); wD = byte_word_prep<Cfg::KV>(wD);
            const uint32_t ab01 = prmt(wA, wB, 0x5140u), ab23 = prmt(wA, wB, 0x7362u);
            const uint32_t cd01 = prmt(wC, wD, 0x5140u), cd23 = prmt(wC, wD, 0x7362u);
            uint32_t a[4];
            a[0] = byte_pair_to_half2<Cfg::KV>(ab01, false);
            a[1] = byte_pair_to_half2<Cfg::KV>(ab01, true);
            a[2] = byte_pair_to_half2<Cfg::KV>(cd01, false);
            a[3] = byte_pair_to_half2<Cfg::KV>(cd01, true);
            if (screen) screened(a);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NTM; ++n) mma_op<BF16>(o[m][2 * pl][n], a, pf[j][m][n][0], pf[j][m][n][1]);
            a[0] = byte_pair_to_half2<Cfg::KV>(ab23, false);
            a[1] = byte_pair_to_half2<Cfg::KV>(ab23, true);
            a[2] = byte_pair_to_half2<Cfg::KV>(cd23, false);
            a[3] = byte_pair_to_half2<Cfg::KV>(cd23, true);
            if (screen) screened(a);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int n = 0; n < NTM; ++n) mma_op<BF16>(o[m][2 * pl + 1][n], a, pf[j][m][n][0], pf[j][m][n][1]);
          }
        }
        __syncwarp();
        // (a stage taken twice is given back after the second time)
        if (lane == 0 && (j == KT - 1 || (have[0] && have[KT - 1]))) mbar_arrive(empty0 + 8 * stage);
      }
    };
    for (int st = (kg - static_cast<int>(step0 % KG) + KG) % KG; st * KT < last; st += KG) {
      const int key0 = (first_tile + st * KT - lead) * kTileKeys;
      if ((W == 1 || kScreen) && st * KT >= lead && (st + 1) * KT <= last && key0 >= lo_all && key0 + KT * kTileKeys - 1 <= hi_all)
        step(st, std::false_type());
      else
        step(st, std::true_type());
    }
    q += ntiles;

    // ---- end of the piece: row sums over the lanes of each row
#pragma unroll
    for (int m = 0; m < MPW; ++m)
#pragma unroll
      for (int n = 0; n < NTR; ++n)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l_r[m][n][0] += __shfl_xor_sync(0xffffffffu, l_r[m][n][0], off);
          l_r[m][n][1] += __shfl_xor_sync(0xffffffffu, l_r[m][n][1], off);
        }
    // output dims of accumulator registers e = 0/1 and 2/3 of m-tile mtl
    auto dim0 = [&](int mtl) {
      const int mt = w * MTW + mtl;
      return BYTE ? (mt >> 1) * 32 + 4 * g + 2 * (mt & 1) : mt * 16 + g;
    };
    constexpr int kStep = BYTE ? 1 : 8;
    const bool direct = pc.npieces == 1;
    if constexpr (kScreen) {
      if (__any_sync(0xffffffffu, odd != 0u)) {
#pragma unroll 1
        for (int j = max(0, (p.window > 0 ? hi_all - p.window + 1 : 0)) / kTileKeys * kTileKeys; j < seq_len; ++j) {
          const int key0 = j / kTileKeys * kTileKeys;
          if (key0 >= lo_all && key0 + kTileKeys - 1 <= screen_hi) {  // tiles that nothing was taken out of
            j = max(key0 + kTileKeys, screen_hi / kTileKeys * kTileKeys) - 1;
            continue;
          }
          const int blk = __ldg(p.block_table + static_cast<long long>(pc.b) * p.max_blocks + j / p.block_size);
          const long long slot = static_cast<long long>(blk >= 0 && blk < p.num_blocks ? blk : 0) * p.block_size + j % p.block_size;
          const uint8_t* row = static_cast<const uint8_t*>(dp.v_cache) + (slot * p.Hkv + pc.kh + th) * (D * Cfg::kElem);
#pragma unroll
          for (int mtl = 0; mtl < MTW; ++mtl) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = dim0(mtl) + e * kStep;
              const bool bad = BYTE ? (row[d] & 0x7fu) == 0x7fu
                                    : not_finite_16<BF16>(reinterpret_cast<const uint16_t*>(row)[d]) != 0u;
#pragma unroll
              for (int n = 0; n < NTM; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const int hi = hi_all + (n * 8 + 2 * t4 + c) / p.G;
                  const bool mark = bad && j <= hi && (p.window <= 0 || j > hi - p.window);
                  o[0][mtl][n][2 * e + c] = mark ? NAN : o[0][mtl][n][2 * e + c];
                  o[1][mtl][n][2 * e + c] = mark ? NAN : o[1][mtl][n][2 * e + c];
                }
            }
          }
        }
      }
    }

    if constexpr (!Cfg::kMerge) {
      // straight from the accumulators
      if (!direct) {
#pragma unroll
        for (int n = 0; n < NTM; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = n * 8 + 2 * t4 + c;
            if (r >= pc.R) continue;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const long long prow = static_cast<long long>(pc.slot) * Cfg::RP + th * Cfg::RH + m * Cfg::RM + r;
              float* dst = p.ws_o + prow * D;
#pragma unroll
              for (int mtl = 0; mtl < MTW; ++mtl) {
                const int d0 = dim0(mtl);
                if constexpr (BYTE) {
                  __stcg(reinterpret_cast<float2*>(dst + d0), make_float2(o[m][mtl][n][c], o[m][mtl][n][2 + c]));
                } else {
                  __stcg(dst + d0, o[m][mtl][n][c]);
                  __stcg(dst + d0 + 8, o[m][mtl][n][2 + c]);
                }
              }
            }
          }
        if (g == 0) {  // the maxima and sums
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NTM; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int r = n * 8 + 2 * t4 + c;
                const long long prow = static_cast<long long>(pc.slot) * Cfg::RP + th * Cfg::RH + m * Cfg::RM + r;
                if (r < pc.R)
                  __stcg(reinterpret_cast<float2*>(p.ws_ml + prow * 2), make_float2(m_r[m][n][c], l_r[m][n][c]));
              }
        }
        continue;
      }
      // the whole unit: the difference of both maps, the norm (W = 1: the warp holds
      // the rows' sums and all of V's dims)
      float ss[NTM][2];
#pragma unroll
      for (int n = 0; n < NTM; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = n * 8 + 2 * t4 + c;
          const float lam = r < pc.R ? __ldg(dp.lambda + (pc.kh + th) * p.G + r % p.G) : 0.f;
          const float l1 = l_r[0][n][c], l2 = l_r[1][n][c];
          const float inv1 = l1 > 0.f ? p.out_scale / l1 : 0.f;
          const float inv2 = l2 > 0.f ? p.out_scale / l2 * lam : 0.f;
          float s = 0.f;
#pragma unroll
          for (int mtl = 0; mtl < MTW; ++mtl)
#pragma unroll
            for (int e = c; e < 4; e += 2) {
              const float v = map_out(l1, o[0][mtl][n][e]) * inv1 - map_out(l2, o[1][mtl][n][e]) * inv2;
              o[0][mtl][n][e] = v;
              s += v * v;
            }
          ss[n][c] = s;
        }
      if (dp.norm_weight != nullptr) {
#pragma unroll
        for (int n = 0; n < NTM; ++n) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            ss[n][0] += __shfl_xor_sync(0xffffffffu, ss[n][0], off);
            ss[n][1] += __shfl_xor_sync(0xffffffffu, ss[n][1], off);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NTM; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = n * 8 + 2 * t4 + c;
          if (r >= pc.R) continue;
          const float f = norm_factor<D>(dp, ss[n][c]);
          uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) +
                          (static_cast<long long>(pc.q0 + r / p.G) * p.Hq + (pc.kh + th) * p.G + r % p.G) * D;
#pragma unroll
          for (int mtl = 0; mtl < MTW; ++mtl) {
            const int d0 = dim0(mtl);
            float a = o[0][mtl][n][c], b = o[0][mtl][n][2 + c];
            if (dp.norm_weight != nullptr) {
              a *= f * norm_weight_at(dp, d0);
              b *= f * norm_weight_at(dp, d0 + kStep);
            }
            const uint32_t v = pack_out(p.out_bf16 != 0, a, b);
            if constexpr (BYTE) {
              *reinterpret_cast<uint32_t*>(dst + d0) = v;
            } else {
              dst[d0] = static_cast<uint16_t>(v & 0xffffu);
              dst[d0 + kStep] = static_cast<uint16_t>(v >> 16);
            }
          }
        }
    } else {
      // ---- through shared memory: rows [head][map][row], a row's key groups
      // weighted by 2^(m - max m) and added in group order
      if (g == 0) {
#pragma unroll
        for (int m = 0; m < MPW; ++m)
#pragma unroll
          for (int n = 0; n < NTR; ++n) {
            if (rt0 + n >= NTM) continue;
            float* ml = merge_ml + (kg * Cfg::RP + th * Cfg::RH + (W == 1 ? m : map) * Cfg::RM + (rt0 + n) * 8 + 2 * t4) * 2;
            ml[0] = m_r[m][n][0];
            ml[1] = l_r[m][n][0];
            ml[2] = m_r[m][n][1];
            ml[3] = l_r[m][n][1];
          }
      }
      named_bar_sync(1, Cfg::kConsumerThreads);
#pragma unroll 1
      for (int k = 0; k < KG; ++k) {
        if (kg == k) {
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NTM; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int row = th * Cfg::RH + m * Cfg::RM + n * 8 + 2 * t4 + c;
                float M = -INFINITY;
#pragma unroll
                for (int kk = 0; kk < KG; ++kk) M = fmaxf(M, merge_ml[(kk * Cfg::RP + row) * 2]);
                const float mk = merge_ml[(k * Cfg::RP + row) * 2];
                const float f = mk == -INFINITY ? 0.f : ex2(mk - M);
                float* mo = merge_o + row * Cfg::kDP;
#pragma unroll
                for (int mtl = 0; mtl < MTW; ++mtl) {
                  const int d0 = dim0(mtl);
                  const float a = f * o[m][mtl][n][c], b = f * o[m][mtl][n][2 + c];
                  if (k == 0) {
                    mo[d0] = a;
                    mo[d0 + kStep] = b;
                  } else {
                    mo[d0] += a;
                    mo[d0 + kStep] += b;
                  }
                }
              }
        }
        named_bar_sync(1, Cfg::kConsumerThreads);
      }
      auto row_ml = [&](int row, float& M, float& L) {
        M = -INFINITY;
        L = 0.f;
#pragma unroll
        for (int k = 0; k < KG; ++k) M = fmaxf(M, merge_ml[(k * Cfg::RP + row) * 2]);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const float mk = merge_ml[(k * Cfg::RP + row) * 2], lk = merge_ml[(k * Cfg::RP + row) * 2 + 1];
          if (lk != 0.f) L += ex2(mk - M) * lk;  // (0: no key; a NaN goes on into the sum)
        }
      };
      constexpr int V4 = D / 128;  // float4 groups per lane of a row
      // a warp per row: (head, map, row) partials, or (head, row) results
      const int rows = HG * pc.R * (direct ? 1 : 2);
      for (int i = warp; i < rows; i += Cfg::kConsumerWarps) {
        const int r = i % pc.R;
        if (!direct) {
          const int row = i / pc.R / 2 * Cfg::RH + (i / pc.R & 1) * Cfg::RM + r;
          float M, L;
          row_ml(row, M, L);
          const long long prow = static_cast<long long>(pc.slot) * Cfg::RP + row;
#pragma unroll
          for (int v = 0; v < V4; ++v)
            __stcg(reinterpret_cast<float4*>(p.ws_o + prow * D) + v * 32 + lane,
                   *(reinterpret_cast<const float4*>(merge_o + row * Cfg::kDP) + v * 32 + lane));
          if (lane == 0) __stcg(reinterpret_cast<float2*>(p.ws_ml + prow * 2), make_float2(M, L));
        } else {
          const int hh = i / pc.R, row1 = hh * Cfg::RH + r, row2 = row1 + Cfg::RM;
          float M, l1, l2;
          row_ml(row1, M, l1);
          row_ml(row2, M, l2);
          const int head = (pc.kh + hh) * p.G + r % p.G;
          const float inv1 = l1 > 0.f ? p.out_scale / l1 : 0.f;
          const float inv2 = l2 > 0.f ? p.out_scale / l2 * __ldg(dp.lambda + head) : 0.f;
          float4 y[V4];
          float ss = 0.f;
#pragma unroll
          for (int v = 0; v < V4; ++v) {
            const float4 a = *(reinterpret_cast<const float4*>(merge_o + row1 * Cfg::kDP) + v * 32 + lane);
            const float4 b = *(reinterpret_cast<const float4*>(merge_o + row2 * Cfg::kDP) + v * 32 + lane);
            y[v] = make_float4(map_out(l1, a.x) * inv1 - map_out(l2, b.x) * inv2, map_out(l1, a.y) * inv1 - map_out(l2, b.y) * inv2,
                               map_out(l1, a.z) * inv1 - map_out(l2, b.z) * inv2, map_out(l1, a.w) * inv1 - map_out(l2, b.w) * inv2);
            ss += y[v].x * y[v].x + y[v].y * y[v].y + y[v].z * y[v].z + y[v].w * y[v].w;
          }
          float f = 1.f;
          if (dp.norm_weight != nullptr) {
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
            f = norm_factor<D>(dp, ss);
          }
          uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + (static_cast<long long>(pc.q0 + r / p.G) * p.Hq + head) * D;
#pragma unroll
          for (int v = 0; v < V4; ++v) store_row4(dp, dst, 4 * (v * 32 + lane), y[v], f);
        }
      }
      named_bar_sync(1, Cfg::kConsumerThreads);  // the merge buffers are free again
    }
  }
  if (!ok && lane == 0) raise_error(p.error_flag, kErrTimeout);
}

// ---------------------------------------------------------------------------
// Joins the partials of every split unit, takes the difference of the two maps
// and, with a norm, normalises the row.
//   grid (units, row chunks, heads per tile), NT threads. A thread holds four
//   dims of one row for both maps, so that their difference is its own; RB rows
//   are taken at a time with PG threads per item, which share the item's pieces
//   (pg, pg + PG, ...; NB pieces' loads in flight). Adjacent lanes take adjacent
//   dims (lanes that take adjacent pieces instead touch a line each: B = 1, 64
//   pieces, 12 -> 19 us). The PG states of an item are scaled by their joint
//   maximum, which is a row's own, and added in pg order, so the result does not
//   depend on scheduling. What does not come from the decode kernel (the unit's
//   layout, lambda, the norm's weights) is read before the wait for it.
constexpr int kJoinThreads = 384, kJoinThreadsMany = 1024;

struct JoinState {
  float m, l;
  float4 o;
};
// Adds a partial (m, l, O) to a state. l = 0: it saw no key. (A NaN score leaves a NaN
// l, with m = -inf where there is no other, which goes on into the sum.)
__device__ __forceinline__ void join_add(JoinState& s, float2 ml, float4 o) {
  if (ml.y == 0.f) return;
  if (ml.x > s.m) {
    const float f = s.m == -INFINITY ? 0.f : ex2(s.m - ml.x);
    s.l *= f;
    s.o.x *= f; s.o.y *= f; s.o.z *= f; s.o.w *= f;
    s.m = ml.x;
  }
  const float w = ex2(ml.x - s.m);
  s.l += w * ml.y;
  s.o.x += w * o.x; s.o.y += w * o.y; s.o.z += w * o.z; s.o.w += w * o.w;
}
template <int D, int NT, int NB>
__global__ void __launch_bounds__(NT, NT <= 384 ? 2 : 1) diff_combine_kernel(const DiffParams dp, int RB, int PG) {
  const DecodeParams& p = dp.d;
  constexpr int S4 = D / 4;
  __shared__ float4 s_o[2][NT];
  __shared__ float2 s_ml[2][NT / S4];  // [map][pg * RB + row]: (m, l), then (weight, joint sum)
  __shared__ float s_ss[NT / 32];
  __shared__ long long s_red[2][NT / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int u = blockIdx.x;
  int P, step;
  long long slot0, slot_base;
  unit_layout(p, u, s_red, P, slot0, slot_base, step);
  const int b = u / p.hgn;
  int q0, qn;
  seq_queries(p, b, false, q0, qn);
  const int kh = (u % p.hgn) * p.hg + blockIdx.z;
  const int live = p.G * qn;
  const int chunk = (live + gridDim.y - 1) / gridDim.y;
  const int r_begin = blockIdx.y * chunk, r_end = min(live, r_begin + chunk);
  const int t = threadIdx.x, c4 = t % S4, pg = t / S4 / RB, j = t / S4 % RB;  // (pg >= PG: a thread without an item)
  float4 wt = make_float4(1.f, 1.f, 1.f, 1.f);
  if (dp.norm_weight != nullptr)
    wt = make_float4(norm_weight_at(dp, 4 * c4), norm_weight_at(dp, 4 * c4 + 1), norm_weight_at(dp, 4 * c4 + 2),
                     norm_weight_at(dp, 4 * c4 + 3));
  float lam = r_begin + j < r_end ? __ldg(dp.lambda + kh * p.G + (r_begin + j) % p.G) : 0.f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (P <= 1) return;
  const long long RP = p.rows_padded;
  const int rbase = blockIdx.z * p.rows_head, rmap = p.rows_head / 2;
  for (int r0 = r_begin; r0 < r_end; r0 += RB) {
    const int r = r0 + j;
    const bool on = pg < PG && r < r_end;
    if (r0 > r_begin) lam = on ? __ldg(dp.lambda + kh * p.G + r % p.G) : 0.f;
    JoinState st[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) st[m] = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (on) {
#pragma unroll 1
      for (int k0 = pg; k0 < P; k0 += NB * PG) {
        float2 ml[NB][2];
        float4 v[NB][2];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int k = k0 + i * PG;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            ml[i][m] = make_float2(-INFINITY, 0.f);
            if (k < P) {
              const long long row = (k == 0 ? slot0 : slot_base + static_cast<long long>(step) * k) * RP + rbase + m * rmap + r;
              ml[i][m] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml + row * 2));
              v[i][m] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + row * D) + c4);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m) join_add(st[m], ml[i][m], v[i][m]);
      }
    }
    if (PG > 1) {
      if (r0 > r_begin) __syncthreads();  // the last rows' states have been read
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        s_o[m][t] = st[m].o;
        if (pg < PG && c4 == 0) s_ml[m][t / S4] = make_float2(st[m].m, st[m].l);
      }
      __syncthreads();
      // a warp per (map, row): the groups' weights and the joint sum
      const int lane = t & 31;
      for (int i = t >> 5; i < 2 * RB; i += NT / 32) {
        float2* ml = &s_ml[i / RB][i % RB];
        const float2 a = lane < PG ? ml[lane * RB] : make_float2(-INFINITY, 0.f);
        float M = a.x;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float w = a.x == -INFINITY ? 0.f : ex2(a.x - M);
        float l = w * a.y;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane < PG) ml[lane * RB] = make_float2(w, l);
      }
      __syncthreads();
      if (pg == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < PG; ++k) {
            const float w = s_ml[m][k * RB + j].x;
            const float4 a = s_o[m][k * RB * S4 + t];
            o.x += w * a.x; o.y += w * a.y; o.z += w * a.z; o.w += w * a.w;
          }
          st[m].o = o;
          st[m].l = s_ml[m][j].y;
        }
      }
    }
    const float i1 = st[0].l > 0.f ? p.out_scale / st[0].l : 0.f, i2 = st[1].l > 0.f ? p.out_scale / st[1].l * lam : 0.f;
    const float l1 = st[0].l, l2 = st[1].l;
    const float4 a = st[0].o, b2 = st[1].o;
    float4 v = make_float4(map_out(l1, a.x) * i1 - map_out(l2, b2.x) * i2, map_out(l1, a.y) * i1 - map_out(l2, b2.y) * i2,
                           map_out(l1, a.z) * i1 - map_out(l2, b2.z) * i2, map_out(l1, a.w) * i1 - map_out(l2, b2.w) * i2);
    if (dp.norm_weight != nullptr) {
      float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (S4 > 32) {  // a row spans two warps
        if (r0 > r_begin) __syncthreads();
        if ((t & 31) == 0) s_ss[t >> 5] = ss;
        __syncthreads();
        ss = s_ss[(t >> 5) & ~1] + s_ss[(t >> 5) | 1];
      }
      const float f = norm_factor<D>(dp, ss);
      v.x *= f * wt.x;
      v.y *= f * wt.y;
      v.z *= f * wt.z;
      v.w *= f * wt.w;
    }
    if (on && pg == 0)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) +
                                (static_cast<long long>(q0 + r / p.G) * p.Hq + kh * p.G + r % p.G) * D + 4 * c4) =
          make_uint2(pack_out(p.out_bf16 != 0, v.x, v.y), pack_out(p.out_bf16 != 0, v.z, v.w));
  }
}

}  // namespace pd
