// decode_scored.cuh -- the scored decode over 16-bit and one-byte caches for sm_103a:
// the paged decode with capped scores, distance biases, prefixes, the rows' log-sum-exp
// and, for the keys' weights, the scores themselves.
//
//   y = c q . k;  y = cap tanh(y / cap);  y -= slope_h |p - j|;  out = softmax(y) V
//
// HBM-bound: K and V are read once (fp16, 24 x 4 heads, D = 256, B = 32, L = 4096, capped: 85.4 us, 0.94 of the
// copy rate; 32 ragged sequences, D = 128, biased: 0.92 to 1.05). The decode's frame (decode_kernel.cuh: balanced
// ranges of 16-key tiles, one TMA producer warp, a ring of 128B-swizzled stages,
// bounded waits, partials and combine) with the differential decode's consumers, for one map:
//  * A warp serves one row tile of 8 query rows of one head, all of D, so that a score is
//    capped and biased by one lane only (two warps that split D would both do it) and no warp
//    waits for another. RG such warps read the same tile where a head has more rows. (Warps that
//    split V's dims and exchange their packed P at a barrier a step, 18 rows over e4m3 caches,
//    B = 8, L = 4096: 41.1 us against 34.8, fp16 caches 44.2 against 33.1.)
//  * KG key groups of such warps take the ring's tiles in turn and merge at the end of a piece.
// A tile is one box of a 4-D tensor map with keys before heads (no bank conflicts). The
// softmax reference is raised only when a score passes it by 2^8: the common step has
// no shuffles and no rescaling.
#pragma once
#include <type_traits>

#include "decode_kernel.cuh"

namespace pd {

template <int D_, int KV_, int HG_, int RG_, int KG_, int NS_, int MINB_>
struct ScoredCfg {
  static constexpr int D = D_, KV = cache_kind(KV_), HG = HG_, RG = RG_, KG = KG_, NS = NS_;
  static constexpr int kMinBlocks = MINB_;
  static constexpr bool BYTE = KV == kKvFp8 || KV == kKvInt8;
  static constexpr bool BF16 = KV == kKvBf16;   // bfloat16 operands; byte kinds use fp16 ones
  static constexpr bool QB = q_is_bf16(KV_);     // q and out in bfloat16
  static constexpr int kElem = BYTE ? 1 : 2;
  static constexpr int kSlabs = D * kElem / 128;
  static constexpr int kHeadBytes = kTileKeys * 128;  // one head's keys of a slab
  static constexpr int kSlabBytes = HG * kHeadBytes;  // [head][key][128 B]
  static constexpr int kTileBytes = kSlabs * kSlabBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  // P as the sum of two operands, the rounded value and the rounded rest, where one
  // rounding would show beside the output's own (error against 64 bits, relative to
  // the output's norm: fp16 3.2e-4 with one, 2.1e-4 with two, bfloat16 2.5e-3 and
  // 1.7e-3; a bfloat16 output over fp16 operands hides it).
  static constexpr int PP = QB && !BF16 ? 1 : 2;
  static constexpr int kGroupWarps = HG * RG;   // warps of a key group
  static constexpr int kConsumerWarps = kGroupWarps * KG;
  static constexpr int kConsumerThreads = kConsumerWarps * 32;
  // Eight consumer warps alone on an SM take the registers that the producer's
  // warpgroup gives up (256 x 216 + 128 x 56 of the launch's 384 x 168).
  static constexpr bool kSplitRegs = kConsumerWarps == 8 && MINB_ == 1;
  static constexpr int kThreads = kConsumerThreads + (kSplitRegs ? 128 : 32);
  static constexpr int RH = RG * 8;              // partial rows per head
  static constexpr int RP = HG * RH;             // per unit
  static constexpr bool kMerge = KG > 1;         // the epilogue goes through shared memory
  static constexpr int kDP = D + 4;              // merge row pitch (floats)
  static constexpr int kMergeO = kMerge ? RP * kDP * 4 : 0;
  static constexpr int kMergeML = kMerge ? KG * RP * 8 : 0;
  static constexpr int kOffMergeML = NS * kStageBytes + kMergeO;
  static constexpr int kOffBars = kOffMergeML + kMergeML;
  static constexpr int kOffPre = kOffBars + 2 * NS * 8;
  static constexpr int kSmemBytes = (kOffPre + (kMaxAutoB + 1) * 4 + 15) / 16 * 16 + 1024;
  // a stage always belongs to the same key group
  static_assert(NS % KG == 0, "ring stages must be a multiple of the key groups");
};

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, Cfg::kMinBlocks)
    decode_scored_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const ScoredParams p) {
  constexpr int D = Cfg::D, NS = Cfg::NS;
  constexpr bool BYTE = Cfg::BYTE, BF16 = Cfg::BF16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);  // full[NS], empty[NS]
  int* s_pre = reinterpret_cast<int*>(smem + Cfg::kOffPre);
  // (what a warp's branches depend on is broadcast, so that they compile to
  // uniform ones without reconvergence around the matrix instructions)
  const int warp = warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
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
    // One elected lane issues two copies a tile, K and V, each one box of the 4-D map;
    // each lane translates its own of the next 32 tiles.
    const uint64_t pol = l2_policy_evict_first();
    uint32_t q = 0, issued = 0;
    bool ok = true;
    while (work_next(p, s_pre, it, pc)) {
      if (pc.ntiles == 0) continue;
      const int32_t* row = p.block_table + static_cast<long long>(pc.b) * p.max_blocks;
      auto load_group = [&](int t) -> int {  // lane i: physical block of tile t + i
        int blk = 0;
        if (t + lane < pc.ntiles) blk = __ldg(row + piece_tile(p, pc, t + lane) / p.tiles_per_block);
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
        const int row0 = cur * p.block_size + (piece_tile(p, pc, t + lane) % p.tiles_per_block) * kTileKeys;
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
  constexpr int RG = Cfg::RG, KG = Cfg::KG, HG = Cfg::HG, PP = Cfg::PP;
  const int kg = warp % KG;                  // key group
  const int rt = (warp / KG) % RG;           // row tile
  const int th = warp / (KG * RG);           // head of the tile
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int KS = D / 16;                 // k-steps of S^T
  constexpr int MT = D / 16;                 // m-tiles of 16 output dims
  float* merge_o = reinterpret_cast<float*>(smem + NS * Cfg::kStageBytes);
  float* merge_ml = reinterpret_cast<float*>(smem + Cfg::kOffMergeML);
  const uint32_t smem0 = smem_u32(smem);
  // One-byte tiles: 16-byte chunk 4 s + t4 of a 64-dim super-step s. The eight lanes of a
  // shared-memory phase hold two accumulator rows of four chunks, so rows 2i and 2i + 1
  // stand for keys whose swizzle phases differ by 4; and the four keys that a V read
  // touches (rows 2 t4) differ in their phases' upper two bits.
  auto key_of = [](int r) { return BYTE ? static_cast<int>((0x37621540u >> (4 * r)) & 15u) : r; };
  const int kg0 = key_of(g);                 // key of accumulator row g (row g + 8: + 8)
  uint32_t k_off, v_off[2];                  // this lane's offsets within a stage
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
  uint32_t qf[KS][2];
  float o[MT][4];
  uint32_t q = 0;                            // ring position of the piece's first tile
  bool ok = true;

  while (warp_uniform(work_next(p, s_pre, it, pc))) {
    const int ntiles = warp_uniform(pc.ntiles), seq_len = warp_uniform(pc.L);
    const int lo_all = warp_uniform(pc.tile_lo_all), hi_all = warp_uniform(pc.tile_hi_all);
    const int prefix = warp_uniform(pc.prefix);
    // ---- q fragments, score factors and limits of this warp's row tile
    float sl2r[2] = {p.sl2, p.sl2}, slope[2] = {0.f, 0.f};
    int hi_r[2];                              // last causal key of rows 2 t4, 2 t4 + 1 (padded rows: -1)
    float m_r[2] = {-INFINITY, -INFINITY}, l_r[2] = {0.f, 0.f};
    {
      const int r = rt * 8 + g;
      const __half* qrow = nullptr;
      if (r < pc.R && pc.ntiles > 0)
        qrow = p.q + (static_cast<long long>(pc.q0 + r / p.G) * p.Hq + (pc.kh + th) * p.G + r % p.G) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int d0 = BYTE ? 64 * (ks >> 2) + 16 * t4 + 4 * (ks & 3) : ks * 16 + 2 * t4;
        const int d1 = d0 + (BYTE ? 2 : 8);
        qf[ks][0] = qrow ? __ldg(reinterpret_cast<const uint32_t*>(qrow + d0)) : 0u;
        qf[ks][1] = qrow ? __ldg(reinterpret_cast<const uint32_t*>(qrow + d1)) : 0u;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rc = rt * 8 + 2 * t4 + c;
        hi_r[c] = rc < pc.R ? pc.L - pc.qlen + rc / p.G : -1;
        if (p.slopes != nullptr && rc < pc.R) slope[c] = __ldg(p.slopes + (pc.kh + th) * p.G + rc % p.G) * kLog2e;
      }
    }
    if constexpr (BYTE && Cfg::QB) {
      // bfloat16 q over byte caches: the row scaled by 2^e into fp16, exactly; 2^-e
      // joins the row's score factor
      float mx = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(qf[ks][h] << 16)), fabsf(__uint_as_float(qf[ks][h] & 0xffff0000u))));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = q_row_exponent(mx);
      sl2r[0] = p.sl2 * pow2f(-__shfl_sync(0xffffffffu, e, 8 * t4));
      sl2r[1] = p.sl2 * pow2f(-__shfl_sync(0xffffffffu, e, 8 * t4 + 4));
      const float up = pow2f(e);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          qf[ks][h] = pack_half2(__uint_as_float(qf[ks][h] << 16) * up, __uint_as_float(qf[ks][h] & 0xffff0000u) * up);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    // ---- this key group's tiles, dealt to the groups by ring position
    // A step is compiled twice: for tiles that every row sees whole, and for the others
    // (EDGE: masks, values), so that the common one has no branch.
    auto step = [&](const int st, auto edge_step) __attribute__((always_inline)) {
      constexpr bool EDGE = decltype(edge_step)::value;
      const uint32_t stage = (q + st) % NS;
      const int key0 = piece_tile(p, pc, st) * kTileKeys;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * stage, ((q + st) / NS) & 1, p.timeout_ns));
      if (!ok) return;
      uint32_t pf[2 * PP];          // P^T fragments
      float x[4];                   // scores (log2 units)
      // ---- S^T: 16 keys x 8 rows
      const uint32_t ka = smem0 + stage * Cfg::kStageBytes + k_off;
      float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (!BYTE) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t a[4];
          ldsm_x4((ka ^ ((ks & 3) * 32)) + (ks >> 2) * Cfg::kSlabBytes, a);
          if (ks & 1) mma_op<BF16>(sb, a, qf[ks][0], qf[ks][1]);
          else mma_op<BF16>(sa, a, qf[ks][0], qf[ks][1]);
        }
      } else {
#pragma unroll
        for (int sup = 0; sup < KS / 4; ++sup) {  // 64-dim super-steps: two a slab
          const uint32_t at = (ka ^ ((sup & 1) * 64)) + (sup >> 1) * Cfg::kSlabBytes;
          const uint4 w0 = lds_v4_tile(at), w8 = lds_v4_tile(at + 8 * 128);
          const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w};
          const uint32_t wb[4] = {w8.x, w8.y, w8.z, w8.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t xa = byte_word_prep<Cfg::KV>(wa[i]), xb = byte_word_prep<Cfg::KV>(wb[i]);
            const uint32_t a[4] = {byte_pair_to_half2<Cfg::KV>(xa, false), byte_pair_to_half2<Cfg::KV>(xb, false),
                                   byte_pair_to_half2<Cfg::KV>(xa, true), byte_pair_to_half2<Cfg::KV>(xb, true)};
            if (i & 1) mma_op<BF16>(sb, a, qf[sup * 4 + i][0], qf[sup * 4 + i][1]);
            else mma_op<BF16>(sa, a, qf[sup * 4 + i][0], qf[sup * 4 + i][1]);
          }
        }
      }
      const int j0 = key0 + kg0;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (sa[e] + sb[e]) * sl2r[e & 1];
      if (p.cap_out > 0.f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = p.cap_out * tanh_f32(x[e] * p.cap_u);
      }
      if (p.slopes != nullptr) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] -= slope[e & 1] * static_cast<float>(abs(j0 + (e >> 1) * 8 - hi_r[e & 1]));
      }
      if constexpr (EDGE) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!row_sees(p, pc, rt * 8 + 2 * t4 + (e & 1), j0 + (e >> 1) * 8)) x[e] = -INFINITY;
      }
      if (p.scores != nullptr) {  // [key][row] of this tile and row tile
        float* dst = p.scores + ((static_cast<long long>(pc.b) * p.Hkv + pc.kh + th) * p.max_blocks *
                                     p.tiles_per_block + key0 / kTileKeys) * (RG * 128) + rt * 128 + kg0 * 8 + 2 * t4;
        __stcg(reinterpret_cast<float2*>(dst), make_float2(x[0], x[1]));
        __stcg(reinterpret_cast<float2*>(dst + 64), make_float2(x[2], x[3]));
      }
      // ---- online softmax. P = 2^(x - m + kUp) is relative to a reference m that is
      // raised to the running maximum only when a score passes it by more than
      // 2^kLazy: P stays at most 2^15, and 2^kUp moves fp16's last bit from 2^-24 to
      // 2^-31 of the reference's weight.
      constexpr float kLazy = 8.f, kUp = 15.f - kLazy;
      bool raise = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) raise |= x[e] - m_r[e & 1] > kLazy;  // (no key seen: m = -inf)
      if (__any_sync(0xffffffffu, raise)) {
        float al[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(x[c], x[2 + c]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          // (each row goes by its own scores: its bits do not depend on the tile's other rows)
          const float old = m_r[c], mn = mx - old > kLazy ? mx : old;
          al[c] = old == -INFINITY ? 1.f : ex2(old - mn);  // (nothing accumulated yet: keep factor 1)
          m_r[c] = mn;
          l_r[c] *= al[c];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          o[mt][0] *= al[0]; o[mt][1] *= al[1];
          o[mt][2] *= al[0]; o[mt][3] *= al[1];
        }
      }
      float nb[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) nb[c] = m_r[c] == -INFINITY ? 0.f : kUp - m_r[c];
      const float p00 = ex2(x[0] + nb[0]), p01 = ex2(x[1] + nb[1]), p10 = ex2(x[2] + nb[0]), p11 = ex2(x[3] + nb[1]);
      l_r[0] += p00 + p10;
      l_r[1] += p01 + p11;
      const uint32_t w0 = pack2<BF16>(p00, p01), w1 = pack2<BF16>(p10, p11);
      pf[0] = movmatrix_trans(w0);
      pf[1] = movmatrix_trans(w1);
      if constexpr (PP == 2) {
        const float2 h0 = unpack2<BF16>(w0), h1 = unpack2<BF16>(w1);
        pf[2] = movmatrix_trans(pack2<BF16>(p00 - h0.x, p01 - h0.y));
        pf[3] = movmatrix_trans(pack2<BF16>(p10 - h1.x, p11 - h1.y));
      }
      // ---- O^T += V^T P^T
      const uint32_t sbase = smem0 + stage * Cfg::kStageBytes;
      // V of keys at or past the sequence's end is zeroed (its bits may be anything)
      const bool tail = EDGE && key0 + kTileKeys > seq_len;
      auto product = [&](int mtl, uint32_t (&a)[4]) {
        if constexpr (EDGE && Cfg::KV != kKvInt8) {
          // Rows that do not see a key have a zero weight for it, which times a NaN or an
          // infinity of its V is NaN: such elements are taken out, and a product of ones (the
          // elements' places, the rows that see the key) marks the outputs that they belong to.
          uint32_t odd[4], any = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) any |= odd[i] = not_finite_16<BF16>(a[i]);
          if (__any_sync(0xffffffffu, any != 0)) {
            constexpr uint32_t kOne = BF16 ? 0x3f803f80u : 0x3c003c00u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] &= ~odd[i];
              odd[i] &= kOne;
            }
            const int ja = key0 + key_of(2 * t4), jb = key0 + key_of(2 * t4 + 1);
            const int r = rt * 8 + g;
            const uint32_t see[2] = {
                kOne & ((row_sees(p, pc, r, ja) ? 0xffffu : 0u) | (row_sees(p, pc, r, jb) ? 0xffff0000u : 0u)),
                kOne & ((row_sees(p, pc, r, ja + 8) ? 0xffffu : 0u) | (row_sees(p, pc, r, jb + 8) ? 0xffff0000u : 0u))};
            float mark[4] = {0.f, 0.f, 0.f, 0.f};
            mma_op<BF16>(mark, odd, see[0], see[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (mark[e] > 0.f) o[mtl][e] = __uint_as_float(0x7fffffffu);
          }
        }
#pragma unroll
        for (int h = 0; h < PP; ++h) mma_op<BF16>(o[mtl], a, pf[2 * h], pf[2 * h + 1]);
      };
      if constexpr (!BYTE) {
        const uint32_t va = sbase + v_off[0];
        uint32_t vm01 = 0xffffffffu, vm23 = 0xffffffffu;
        if (tail) {
          const int kt = key0 + 2 * t4;
          vm01 = (kt < seq_len ? 0x0000ffffu : 0u) | (kt + 1 < seq_len ? 0xffff0000u : 0u);
          vm23 = (kt + 8 < seq_len ? 0x0000ffffu : 0u) | (kt + 9 < seq_len ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int mtl = 0; mtl < MT; ++mtl) {
          uint32_t a[4];
          ldsm_x4_trans((va ^ ((mtl & 3) * 32)) + (mtl >> 2) * Cfg::kSlabBytes, a);
          if (tail) {
            a[0] &= vm01; a[1] &= vm01; a[2] &= vm23; a[3] &= vm23;
          }
          product(mtl, a);
        }
      } else {
        // 32-dim group P32: lane reads 4 codes at dims 32 P32 + 4 g of keys
        // key_of(2 t4), key_of(2 t4 + 1) and those + 8; m-tile 2 P32 takes
        // dims 4 g (row g) and 4 g + 1 (row g + 8), m-tile 2 P32 + 1 the next two
        const int kA = key_of(2 * t4), kB = key_of(2 * t4 + 1), kC = kA + 8, kD = kB + 8;
#pragma unroll
        for (int P32 = 0; P32 < MT / 2; ++P32) {
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
          uint32_t a[4] = {byte_pair_to_half2<Cfg::KV>(ab01, false), byte_pair_to_half2<Cfg::KV>(ab01, true),
                           byte_pair_to_half2<Cfg::KV>(cd01, false), byte_pair_to_half2<Cfg::KV>(cd01, true)};
          product(2 * P32, a);
          uint32_t b[4] = {byte_pair_to_half2<Cfg::KV>(ab23, false), byte_pair_to_half2<Cfg::KV>(ab23, true),
                           byte_pair_to_half2<Cfg::KV>(cd23, false), byte_pair_to_half2<Cfg::KV>(cd23, true)};
          product(2 * P32 + 1, b);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * stage);
    };
    for (int st = (kg - static_cast<int>(q % KG) + KG) % KG; st < ntiles; st += KG) {
      const int key0 = piece_tile(p, pc, st) * kTileKeys;
      if ((key0 >= lo_all && key0 + kTileKeys - 1 <= hi_all) || (key0 + kTileKeys <= prefix && hi_all >= 0))
        step(st, std::false_type());
      else
        step(st, std::true_type());
    }
    q += ntiles;

    // ---- end of the piece: row sums over the lanes of each row; m is what the weights are relative to
    constexpr float kUp = 7.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l_r[c] += __shfl_xor_sync(0xffffffffu, l_r[c], off);
      if (l_r[c] != l_r[c] && m_r[c] == -INFINITY) m_r[c] = 0.f;  // nothing but NaN: not an empty row
      m_r[c] -= kUp;
    }
    // output dims of accumulator registers e = 0/1 and 2/3 of m-tile mtl
    auto dim0 = [&](int mt) {
      return BYTE ? (mt >> 1) * 32 + 4 * g + 2 * (mt & 1) : mt * 16 + g;
    };
    constexpr int kStep = BYTE ? 1 : 8;
    const bool direct = pc.npieces == 1;
    if constexpr (!Cfg::kMerge) {
      // straight from the accumulators
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = rt * 8 + 2 * t4 + c;
        if (r >= pc.R) continue;
        if (direct) {
          const int head = (pc.kh + th) * p.G + r % p.G;
          const float inv = row_factor(p, l_r[c]);
          if (g == 0) store_row_sum(p, pc.b, pc.q0, r / p.G, head, m_r[c], l_r[c]);
          uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + (static_cast<long long>(pc.q0 + r / p.G) * p.Hq + head) * D;
#pragma unroll
          for (int mtl = 0; mtl < MT; ++mtl) {
            const int d0 = dim0(mtl);
            const uint32_t v = pack2<Cfg::QB>(o[mtl][c] * inv, o[mtl][2 + c] * inv);
            if constexpr (BYTE) {
              *reinterpret_cast<uint32_t*>(dst + d0) = v;
            } else {
              dst[d0] = static_cast<uint16_t>(v & 0xffffu);
              dst[d0 + kStep] = static_cast<uint16_t>(v >> 16);
            }
          }
        } else {
          const long long prow = static_cast<long long>(pc.slot) * Cfg::RP + th * Cfg::RH + r;
          float* dst = p.ws_o + prow * D;
#pragma unroll
          for (int mtl = 0; mtl < MT; ++mtl) {
            const int d0 = dim0(mtl);
            if constexpr (BYTE) {
              __stcg(reinterpret_cast<float2*>(dst + d0), make_float2(o[mtl][c], o[mtl][2 + c]));
            } else {
              __stcg(dst + d0, o[mtl][c]);
              __stcg(dst + d0 + 8, o[mtl][2 + c]);
            }
          }
          if (g == 0) __stcg(reinterpret_cast<float2*>(p.ws_ml + prow * 2), make_float2(m_r[c], l_r[c]));
        }
      }
    } else {
      // ---- through shared memory: a row's key groups weighted by 2^(m - max m) and added in group order
      if (g == 0) {
        float* ml = merge_ml + (kg * Cfg::RP + th * Cfg::RH + rt * 8 + 2 * t4) * 2;
        ml[0] = m_r[0];
        ml[1] = l_r[0];
        ml[2] = m_r[1];
        ml[3] = l_r[1];
      }
      named_bar_sync(1, Cfg::kConsumerThreads);
#pragma unroll 1
      for (int k = 0; k < KG; ++k) {
        if (kg == k) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int row = th * Cfg::RH + rt * 8 + 2 * t4 + c;
            float M = -INFINITY;
#pragma unroll
            for (int kk = 0; kk < KG; ++kk) M = fmaxf(M, merge_ml[(kk * Cfg::RP + row) * 2]);
            const float mk = merge_ml[(k * Cfg::RP + row) * 2];
            const float f = mk == -INFINITY ? 0.f : ex2(mk - M);
            float* mo = merge_o + row * Cfg::kDP;
#pragma unroll
            for (int mtl = 0; mtl < MT; ++mtl) {
              const int d0 = dim0(mtl);
              const float a = f * o[mtl][c], b = f * o[mtl][2 + c];
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
      constexpr int V4 = D / 128;  // float4 groups per lane of a row
      for (int i = warp; i < HG * pc.R; i += Cfg::kConsumerWarps) {  // a warp per row
        const int r = i % pc.R, hh = i / pc.R, row = hh * Cfg::RH + r;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < KG; ++k) M = fmaxf(M, merge_ml[(k * Cfg::RP + row) * 2]);
#pragma unroll
        for (int k = 0; k < KG; ++k) {
          const float mk = merge_ml[(k * Cfg::RP + row) * 2], lk = merge_ml[(k * Cfg::RP + row) * 2 + 1];
          if (lk != 0.f) L += ex2(mk - M) * lk;  // (0: no key; a NaN goes on into the sum)
        }
        const float4* src = reinterpret_cast<const float4*>(merge_o + row * Cfg::kDP);
        if (!direct) {
          const long long prow = static_cast<long long>(pc.slot) * Cfg::RP + row;
#pragma unroll
          for (int v = 0; v < V4; ++v) __stcg(reinterpret_cast<float4*>(p.ws_o + prow * D) + v * 32 + lane, src[v * 32 + lane]);
          if (lane == 0) __stcg(reinterpret_cast<float2*>(p.ws_ml + prow * 2), make_float2(M, L));
        } else {
          const int head = (pc.kh + hh) * p.G + r % p.G;
          const float inv = row_factor(p, L);
          if (lane == 0) store_row_sum(p, pc.b, pc.q0, r / p.G, head, M, L);
          uint2* dst = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) +
                                                (static_cast<long long>(pc.q0 + r / p.G) * p.Hq + head) * D);
#pragma unroll
          for (int v = 0; v < V4; ++v) {
            const float4 f = src[v * 32 + lane];
            dst[v * 32 + lane] = make_uint2(pack2<Cfg::QB>(f.x * inv, f.y * inv), pack2<Cfg::QB>(f.z * inv, f.w * inv));
          }
        }
      }
      named_bar_sync(1, Cfg::kConsumerThreads);  // merge buffers free again
    }
  }
  if (!ok && lane == 0) raise_error(p.error_flag, kErrTimeout);
}

}  // namespace pd
