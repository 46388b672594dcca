// decode_fp4.cuh -- paged split-K decode over 4-bit caches for sm_103a.
//
// The decode of decode_kernel.cuh (its units, balanced and fixed splits, partials
// and combine; the scored decode's caps, biases and prefixes) over caches of e2m1
// codes, two to a byte, with an e4m3 scale for every 16 values of a row and an fp32
// scale for each cache: codes [num_blocks, Hkv, block_size, D / 2], scales
// [num_blocks, Hkv, block_size, D / 16]. Heads before keys, so that a head's 16 keys
// are one run of 8 D bytes of codes and one of D bytes of scales: at 4 bits a single
// row is 64 or 128 bytes.
//
// 9/16 byte a value is so little that the tensor products' operands, not HBM, are
// what the consumers wait for: a tile of 16 keys of one head (D = 256) takes 128
// conversions e2m1 -> fp16, as many multiplications by the scales, and 32 to 48
// mma.sync for 4.6 KB: 616 instructions of a warp in all (24 x 4 heads, B = 32, L = 4096: 42.4 us, of which
// 8 lie around the loop; L = 16384 125 us, 0.72 of the copy rate). No unit of the SM is full while they run:
// instructions 1.9 of 4 a cycle, ALU 39 %, tensor 30, fp16 21, shared memory 29, conversions' unit below 3,
// DRAM 48. What bounds it is the latency of one chain after another in the three warps that a
// scheduler has (165 registers a thread; stalls: fixed latencies 1.3 warps an issue, math pipes 0.7, shared
// memory 0.6). So no warp does anything else, and none waits for another:
//  * A unit is (sequence, KV head). Its tiles go to the CTA's warps in turn; every
//    warp translates pages, copies, computes and keeps (m, l, O) on its own, and the
//    warps meet only at the end of a piece. No producer warp, no barriers in the loop.
//  * A lane copies (cp.async) the 16-byte pieces of codes that it will itself
//    multiply, into a ring of its warp's own: [piece][lane], no bank conflicts. Only
//    the scales, 16 bytes a key, are read across lanes.
//  * S^T = K Q^T: row g of the A operand is key g, and since the order of the
//    contraction is free a byte of codes converts straight to an operand register
//    (two adjacent dims of a key); q lies in shared memory in the same order.
//  * O^T = V^T P^T: an operand register is two keys of one dim. The nibbles of two
//    keys' words are exchanged first (four logical operations for 16 values), so that
//    a byte again converts to a register; rows g and g + 8 of an m-tile are two
//    adjacent dims.
//  * A code times its scale has at most six significant bits: exact in fp16, as
//    operands for K and V alike. The caches' fp32 scales go into the score factor and
//    the output.
//  * The softmax reference is raised only when a score passes it by 2^8, so that the
//    common step has no shuffles and no rescaling.
#pragma once
#include <type_traits>

#include "decode_kernel.cuh"

namespace pd {

struct Fp4Params : ScoredParams {
  const uint8_t *k_codes, *v_codes, *k_sf, *v_sf;
};

// NT: row tiles of 8 query rows that a warp computes, RG: row groups of that many
// (warps that read the same tiles), KG: key groups, ST: tiles in a warp's ring.
template <int D_, int NT_, int RG_, int KG_, int ST_, int MINB_, bool QB_>
struct Fp4Cfg {
  static constexpr int D = D_, NT = NT_, RG = RG_, KG = KG_, ST = ST_, kMinBlocks = MINB_;
  static constexpr bool QB = QB_;
  // P as two operands unless a bfloat16 output's own rounding hides one (see decode_kernel.cuh)
  static constexpr int PP = QB ? 1 : 2;
  static constexpr int kWarps = KG * RG, kThreads = kWarps * 32;
  static constexpr int kCodes = kTileKeys * D / 2, kScales = kTileKeys * D / 16;
  static constexpr int kTile = 2 * kCodes + 2 * kScales;  // K codes, V codes, K scales, V scales
  static constexpr int kStage = kTile;
  static constexpr int kRing = ST * kStage;               // a warp's
  static constexpr int MT = D / 16;                       // m-tiles (pairs of dims by lane)
  static constexpr int kPitch = 33;                       // float4 pitch of an m-tile's fragments in the merge
  static constexpr int kMerge = NT * MT * kPitch * 16;    // a warp's (m, l, O) fragments, over its ring
  static_assert(kMerge <= kRing, "the merge buffer lies over the ring");
  static constexpr int RP = RG * NT * 8;
  static constexpr int kOffQ = kWarps * kRing;            // q fragments
  static constexpr int kQ = RG * NT * MT * 32 * 8;
  static constexpr int kOffML = kOffQ + kQ;               // [warp][NT * 8] (m, l)
  static constexpr int kOffFactor = kOffML + kWarps * NT * 8 * 8;  // rows' score factors
  static constexpr int kOffPre = kOffFactor + RP * 4;
  static constexpr int kSmemBytes = kOffPre + (kMaxAutoB + 1) * 4 + 12;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The four bytes of a word of e2m1 codes as four fp16 pairs (low nibble -> low half), exact.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint16_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
  return v;
}

// O^T += V^T P^T for a tile of 16 keys from `key0` on, whose codes lie at vt as the copies left them and whose
// scales at sf: P operands pb[n] of NT row tiles (the query rows from row0 on), and with PP = 2 what their rounding left,
// pl[n]. EDGE: not every row sees all of its keys.
template <int D, int NT, int PP, bool EDGE>
__device__ __forceinline__ void fp4_pv(const ScoredParams& p, const Piece& pc, int row0, uint32_t vt, uint32_t sf, int lane,
                                       int key0, int seq_len, const uint32_t (&pb)[NT][2], const uint32_t (&pl)[NT][2],
                                       float (&o)[D / 16][NT][4]) {
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int NG = D / 128;  // groups of 16 dims that a lane holds
  constexpr int NWD = D / 64;  // words of a key that a lane holds
  // scales of keys (2 t4, 2 t4 + 1) and (2 t4 + 8, 2 t4 + 9) for groups NG g ..
  uint32_t f01[NG], f89[NG], w[4][NWD];
  if constexpr (NG == 2) {
    const uint32_t at = sf + 2 * t4 * 16 + 2 * g;
    const uint32_t a = e4m3x2_to_half2(lds_u16(at)), b = e4m3x2_to_half2(lds_u16(at + 16)),
                   c = e4m3x2_to_half2(lds_u16(at + 128)), d = e4m3x2_to_half2(lds_u16(at + 144));
    f01[0] = prmt(a, b, 0x5410u); f01[1] = prmt(a, b, 0x7632u);
    f89[0] = prmt(c, d, 0x5410u); f89[1] = prmt(c, d, 0x7632u);
  #pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 v = lds_v4(vt + q * 512 + lane * 16);
      w[q][0] = v.x; w[q][1] = v.y; w[q][2] = v.z; w[q][3] = v.w;
    }
  } else {
    // rows of 8 scales: a byte for this lane's group of each key
    const uint32_t at = sf + 2 * t4 * 8 + (g & ~1);
    const uint32_t a = lds_u16(at), b = lds_u16(at + 8), c = lds_u16(at + 64), d = lds_u16(at + 72);
    const uint32_t sel = (g & 1) ? 0x0051u : 0x0040u;
    f01[0] = e4m3x2_to_half2(static_cast<uint16_t>(prmt(a, b, sel)));
    f89[0] = e4m3x2_to_half2(static_cast<uint16_t>(prmt(c, d, sel)));
  #pragma unroll
    for (int q = 0; q < 4; ++q) {
      // key 2 t4 + (q & 1) + 8 (q >> 1): line t4 + 4 (q >> 1)
      const uint32_t at_v = vt + t4 * 128 + (((g >> 1) ^ (2 * t4)) << 4) + (g & 1) * 8;
      const uint2 v = lds_v2((at_v ^ ((q & 1) * 64)) + (q >> 1) * 512);
      w[q][0] = v.x; w[q][1] = v.y;
    }
  }
  // Keys at or past the sequence's end may hold any bits: a scale of NaN must not meet a
  // weight of zero. Nor must one of a key that only some rows see: it is taken out, and a
  // product of ones marks the outputs of the rows that see it.
  if constexpr (EDGE) {
    const int ka = key0 + 2 * t4;
    const uint32_t in01 = (ka < seq_len ? 0x0000ffffu : 0u) | (ka + 1 < seq_len ? 0xffff0000u : 0u);
    const uint32_t in89 = (ka + 8 < seq_len ? 0x0000ffffu : 0u) | (ka + 9 < seq_len ? 0xffff0000u : 0u);
  #pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
      f01[gr] &= in01;
      f89[gr] &= in89;
      const uint32_t o01 = not_finite_16<false>(f01[gr]), o89 = not_finite_16<false>(f89[gr]);
      if (__any_sync(0xffffffffu, (o01 | o89) != 0)) {
        f01[gr] &= ~o01;
        f89[gr] &= ~o89;
        const uint32_t a[4] = {o01 & 0x3c003c00u, o01 & 0x3c003c00u, o89 & 0x3c003c00u, o89 & 0x3c003c00u};
  #pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int r = row0 + n * 8 + g;
          const uint32_t see0 = (row_sees(p, pc, r, ka) ? 0x3c00u : 0u) | (row_sees(p, pc, r, ka + 1) ? 0x3c000000u : 0u);
          const uint32_t see1 = (row_sees(p, pc, r, ka + 8) ? 0x3c00u : 0u) | (row_sees(p, pc, r, ka + 9) ? 0x3c000000u : 0u);
          float mark[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816(mark, a, see0, see1);
  #pragma unroll
          for (int mt = 0; mt < 8; ++mt)
  #pragma unroll
            for (int e = 0; e < 4; ++e)
              if (mark[e] > 0.f) o[gr * 8 + mt][n][e] = __uint_as_float(0x7fffffffu);
        }
      }
    }
  }
  #pragma unroll
  for (int q = 0; q < NWD; ++q) {  // a word: 8 dims, four m-tiles
    constexpr uint32_t M = 0x0f0f0f0fu;
    const uint32_t e01 = (w[0][q] & M) | ((w[1][q] << 4) & ~M), d01 = ((w[0][q] >> 4) & M) | (w[1][q] & ~M);
    const uint32_t e89 = (w[2][q] & M) | ((w[3][q] << 4) & ~M), d89 = ((w[2][q] >> 4) & M) | (w[3][q] & ~M);
    uint32_t he[4], hd[4], je[4], jd[4];
    e2m1x8_to_half2(e01, he);
    e2m1x8_to_half2(d01, hd);
    e2m1x8_to_half2(e89, je);
    e2m1x8_to_half2(d89, jd);
    const uint32_t s01 = f01[q / 2], s89 = f89[q / 2];
  #pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t a[4] = {hmul2_u(he[b], s01), hmul2_u(hd[b], s01), hmul2_u(je[b], s89), hmul2_u(jd[b], s89)};
  #pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16816(o[4 * q + b][n], a, pb[n][0], pb[n][1]);
        if constexpr (PP == 2) mma_16816(o[4 * q + b][n], a, pl[n][0], pl[n][1]);
      }
    }
  }
}

// Dims d and d + 1 of row r of a piece, whose weights are relative to ml.x and add up to ml.y: the
// unit's output, or the piece's partial.
template <class Cfg>
__device__ __forceinline__ void fp4_store(const ScoredParams& p, const Piece& pc, int r, int d, float v0, float v1, float2 ml,
                                          bool direct) {
  if (direct) {
    const int q = r / p.G, head = pc.kh * p.G + r % p.G;
    const float inv = row_factor(p, ml.y);
    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(p.out) +
                                 (static_cast<long long>(pc.q0 + q) * p.Hq + head) * Cfg::D + d) =
        Cfg::QB ? pack_bf162(v0 * inv, v1 * inv) : pack_half2(v0 * inv, v1 * inv);
    if (d == 0) store_row_sum(p, pc.b, pc.q0, q, head, ml.x, ml.y);
  } else {
    const long long prow = static_cast<long long>(pc.slot) * Cfg::RP + r;
    __stcg(reinterpret_cast<float2*>(p.ws_o + prow * Cfg::D + d), make_float2(v0, v1));
    if (d == 0) __stcg(reinterpret_cast<float2*>(p.ws_ml + prow * 2), ml);
  }
}

// The warps' accumulator fragments, (n MT + mt) kPitch + lane in each warp's ring, and (m, l) joined into the piece's
// output or partial. Warp k RG + rw: key group k, row group rw of NT row tiles.
template <class Cfg, int D, int NT, int RG, int KG, int THREADS>
__device__ __forceinline__ void fp4_join(const ScoredParams& p, const Piece& pc, const uint8_t* rings, const float2* s_ml) {
  constexpr int MT = D / 16;
  static_assert(THREADS % (4 * MT) == 0, "a thread's fragments of a row tile are of the same two rows");
  const bool direct = pc.npieces == 1;
#pragma unroll 1
  for (int tile = 0; tile < RG * NT; ++tile) {
    const int rw = tile / NT, n = tile % NT, r0 = tile * 8 + 2 * (threadIdx.x / MT % 4);
    if (r0 >= pc.R) continue;
    // the key groups' factors and the rows' (m, l)
    float f[KG][2];
    float2 row[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float2 ml[KG];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        ml[k] = s_ml[(k * RG + rw) * NT * 8 + n * 8 + 2 * (threadIdx.x / MT % 4) + c];
        M = fmaxf(M, ml[k].x);
      }
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        f[k][c] = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
        L += f[k][c] * ml[k].y;
      }
      row[c] = make_float2(M, L);
    }
    for (int item = threadIdx.x; item < MT * 32; item += THREADS) {  // two dims of two rows: an accumulator fragment
      const int mt = item % MT, ln = item / MT;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < KG; ++k) {
        const float4 v = reinterpret_cast<const float4*>(rings + (k * RG + rw) * Cfg::kRing)[(n * MT + mt) * Cfg::kPitch + ln];
        acc.x += f[k][0] * v.x; acc.y += f[k][1] * v.y; acc.z += f[k][0] * v.z; acc.w += f[k][1] * v.w;
      }
      const int d = D / 8 * (ln >> 2) + 2 * mt;  // dims d, d + 1 of rows r0, r0 + 1
      fp4_store<Cfg>(p, pc, r0, d, acc.x, acc.z, row[0], direct);
      if (r0 + 1 < pc.R) fp4_store<Cfg>(p, pc, r0 + 1, d, acc.y, acc.w, row[1], direct);
    }
  }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, Cfg::kMinBlocks) decode_fp4_kernel(const Fp4Params p) {
  constexpr int D = Cfg::D, NT = Cfg::NT, RG = Cfg::RG, KG = Cfg::KG, ST = Cfg::ST, MT = Cfg::MT;
  constexpr int PP = Cfg::PP;
  extern __shared__ __align__(128) uint8_t smem[];
  float2* s_ml = reinterpret_cast<float2*>(smem + Cfg::kOffML);
  float* s_factor = reinterpret_cast<float*>(smem + Cfg::kOffFactor);
  int* s_pre = reinterpret_cast<int*>(smem + Cfg::kOffPre);
  const int warp = warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rg = warp % RG, kg = warp / RG;
  const int g = lane >> 2, t4 = lane & 3;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.num_splits == 0 && warp == 0) balanced_prefix(p, s_pre, lane);
  __syncthreads();
  WorkIter it;
  work_init(p, s_pre, it);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Piece pc;

  const uint32_t ring = smem_u32(smem) + warp * Cfg::kRing;
  // this lane's pieces of a tile. D = 256: K chunks t4 and t4 + 4 of keys g and g + 8; V chunk g of
  // keys 2 t4, 2 t4 + 1 and those + 8; scales of key lane % 16. D = 128: K chunk t4; V and the
  // scales in 16-byte pieces of two keys' rows.
  const uint8_t* k_src = p.k_codes + (D == 256 ? g * 128 + t4 * 16 : g * 64 + t4 * 16);
  const uint8_t* v_src = p.v_codes + (D == 256 ? 2 * t4 * 128 + g * 16 : lane * 16);
  constexpr int kSfLanes = D / 16;  // lanes that copy scales of K (as many of V)
  const uint8_t* sf_src = (lane < kSfLanes ? p.k_sf : p.v_sf) + lane % kSfLanes * 16;
  const uint32_t q_frags = smem_u32(smem + Cfg::kOffQ) + rg * NT * MT * 32 * 8;

  while (warp_uniform(work_next(p, s_pre, it, pc))) {
    const int kh = pc.kh, ntiles = warp_uniform(pc.ntiles), seq_len = warp_uniform(pc.L);
    const int lo_all = warp_uniform(pc.tile_lo_all), hi_all = warp_uniform(pc.tile_hi_all);
    const int prefix = warp_uniform(pc.prefix);
    // ---- copies of the warp's steps: step i is tile i KG + kg
    const int steps = (ntiles - kg + KG - 1) / KG;  // (<= 0: none)
    const int32_t* row = p.block_table + static_cast<long long>(pc.b) * p.max_blocks;
    auto load_block = [&](int i0) -> int {  // lane: the physical block of step i0 + lane
      const int k = (i0 + lane) * KG + kg;
      return k < ntiles ? __ldg(row + piece_tile(p, pc, k) / p.tiles_per_block) : 0;
    };
    int cur = 0, nxt = load_block(0);  // lane: the tile in the caches' order, of step (i & ~31) + lane; blocks of the steps after
    auto to_tile = [&](int i0, int blk) -> int {
      if (blk < 0 || blk >= p.num_blocks) {
        raise_error(p.error_flag, kErrBlockId);
        blk = 0;
      }
      return (blk * p.Hkv + kh) * p.tiles_per_block + piece_tile(p, pc, (i0 + lane) * KG + kg) % p.tiles_per_block;
    };
    int next = 0;              // the step whose copies are next
    uint32_t fill = ring;      // and its stage
    auto issue = [&]() {
      if (next < steps) {
        if ((next & 31) == 0) {
          cur = to_tile(next, nxt);
          nxt = load_block(next + 32);
        }
        const long long tile = __shfl_sync(0xffffffffu, cur, next & 31);
        const uint8_t* kc = k_src + tile * Cfg::kCodes;
        const uint8_t* vc = v_src + tile * Cfg::kCodes;
        const uint8_t* sf = sf_src + tile * Cfg::kScales;
        const uint32_t dst = fill + lane * 16;
        if constexpr (D == 256) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            cp_async16(dst + q * 512, kc + (q >> 1) * 1024 + (q & 1) * 64);
            cp_async16(dst + Cfg::kCodes + q * 512, vc + (q >> 1) * 1024 + (q & 1) * 128);
          }
          cp_async16(dst + 2 * Cfg::kCodes, sf);
        } else {
          // V: 16-byte piece c of line l (two keys' rows) lies at c ^ 2 l of its line: the lanes of
          // a read (keys 2 t4, 8-byte chunks g) meet all banks
          const int line = lane >> 3;
          const uint32_t vd = fill + Cfg::kCodes + line * 128 + (((lane & 7) ^ (2 * line)) << 4);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            cp_async16(dst + q * 512, kc + q * 512);
            cp_async16(vd + q * 512, vc + q * 512);
          }
          if (lane < 2 * kSfLanes) cp_async16(dst + 2 * Cfg::kCodes, sf);
        }
      }
      cp_async_commit();
      ++next;
      fill = fill == ring + (ST - 1) * Cfg::kStage ? ring : fill + Cfg::kStage;
    };
    // q rows are loaded while the table's entries come
    uint2 qv[NT][MT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = (rg * NT + n) * 8 + g;
      const uint32_t* qrow = nullptr;
      if (kg == 0 && r < pc.R && ntiles > 0)
        qrow = reinterpret_cast<const uint32_t*>(
            p.q + (static_cast<long long>(pc.q0 + r / p.G) * p.Hq + kh * p.G + r % p.G) * D);
#pragma unroll
      for (int ks = 0; ks < MT; ++ks) {
        // chunk of 32 dims (t4, then t4 + 4), four dims of it a k-step
        const int d = D == 256 ? (ks >> 3) * 128 + 32 * t4 + (ks & 7) * 4 : 32 * t4 + ks * 4;
        qv[n][ks] = qrow ? __ldg(reinterpret_cast<const uint2*>(qrow + d / 2)) : make_uint2(0u, 0u);
      }
    }
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) issue();

    // ---- q fragments, in the order that the codes' bytes give the contraction: lane's k-steps
    // 2 i and 2 i + 1 side by side, [row group][row tile][i][lane] 16 bytes
    float sl2r[NT][2];
    int hi_r[NT][2];          // last causal key of rows 2 t4, 2 t4 + 1 of a row tile (padded rows: -1)
    float m_r[NT][2], l_r[NT][2];
    float o[MT][NT][4];
    if (kg == 0) {  // (the key groups share the row group's)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (Cfg::QB) {
          float m = 0.f;
#pragma unroll
          for (int ks = 0; ks < MT; ++ks)
            m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(qv[n][ks].x << 16)), fabsf(__uint_as_float(qv[n][ks].x & 0xffff0000u))),
                               fmaxf(fabsf(__uint_as_float(qv[n][ks].y << 16)), fabsf(__uint_as_float(qv[n][ks].y & 0xffff0000u)))));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const int eq = q_row_exponent(m);
          const float up = pow2f(eq);
          if (t4 == 0) s_factor[(rg * NT + n) * 8 + g] = p.sl2 * pow2f(-eq);
#pragma unroll
          for (int ks = 0; ks < MT; ++ks) {
            uint2& v = qv[n][ks];
            v.x = pack_half2(__uint_as_float(v.x << 16) * up, __uint_as_float(v.x & 0xffff0000u) * up);
            v.y = pack_half2(__uint_as_float(v.y << 16) * up, __uint_as_float(v.y & 0xffff0000u) * up);
          }
        }
#pragma unroll
        for (int i = 0; i < MT / 2; ++i)
          sts_v4(q_frags + ((n * MT / 2 + i) * 32 + lane) * 16, qv[n][2 * i].x, qv[n][2 * i].y, qv[n][2 * i + 1].x,
                 qv[n][2 * i + 1].y);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rr = (rg * NT + n) * 8 + 2 * t4 + c;
        hi_r[n][c] = rr < pc.R ? pc.L - pc.qlen + rr / p.G : -1;
        m_r[n][c] = -INFINITY;
        l_r[n][c] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) sl2r[n][c] = Cfg::QB ? s_factor[(rg * NT + n) * 8 + 2 * t4 + c] : p.sl2;

    uint32_t stage = ring;
    // A step is compiled twice: for tiles that every row sees whole, and for the others (EDGE:
    // masks, scales that are no numbers).
    auto step = [&](const int i, auto edge_step) __attribute__((always_inline)) {
      constexpr bool EDGE = decltype(edge_step)::value;
      const int key0 = piece_tile(p, pc, i * KG + kg) * kTileKeys;
      // ---- S^T = K Q^T: 16 keys x 8 rows for each row tile
      float x[NT][4];
      {
        float sa[NT][4], sb[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sa[n][e] = sb[n][e] = 0.f;
        const uint32_t kt = stage;
        constexpr int NC = D / 128;  // 16-byte chunks of a key that a lane holds
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          // scales of the two groups of 16 dims of the chunk, for keys g and g + 8
          const uint32_t sf = kt + 2 * Cfg::kCodes + g * (D / 16) + c * 8 + 2 * t4;
          const uint32_t s0 = e4m3x2_to_half2(lds_u16(sf)), s8 = e4m3x2_to_half2(lds_u16(sf + D / 2));
          const uint32_t s00 = prmt(s0, s0, 0x1010u), s01 = prmt(s0, s0, 0x3232u);
          const uint32_t s80 = prmt(s8, s8, 0x1010u), s81 = prmt(s8, s8, 0x3232u);
          const uint4 w0 = lds_v4(kt + c * 512 + lane * 16), w8 = lds_v4(kt + (NC + c) * 512 + lane * 16);
          const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w}, wb[4] = {w8.x, w8.y, w8.z, w8.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {  // a word: 8 dims, two k-steps; words 0, 1 are the first group
            uint32_t ha[4], hb[4];
            e2m1x8_to_half2(wa[w], ha);
            e2m1x8_to_half2(wb[w], hb);
            const uint32_t f0 = w < 2 ? s00 : s01, f8 = w < 2 ? s80 : s81;
            const uint32_t a0[4] = {hmul2_u(ha[0], f0), hmul2_u(hb[0], f8), hmul2_u(ha[1], f0), hmul2_u(hb[1], f8)};
            const uint32_t a1[4] = {hmul2_u(ha[2], f0), hmul2_u(hb[2], f8), hmul2_u(ha[3], f0), hmul2_u(hb[3], f8)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 b = lds_v4_tile(q_frags + ((n * MT / 2 + c * 4 + w) * 32 + lane) * 16);
              mma_16816(sa[n], a0, b.x, b.y);
              mma_16816(sb[n], a1, b.z, b.w);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = (sa[n][e] + sb[n][e]) * sl2r[n][e & 1];
      }
      // ---- caps, biases, masks
      const int j0 = key0 + g;
      if (p.cap_out > 0.f) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = p.cap_out * tanh_f32(x[n][e] * p.cap_u);
      }
      if (p.slopes != nullptr) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = (rg * NT + n) * 8 + 2 * t4 + c;
            const float slope = r < pc.R ? __ldg(p.slopes + kh * p.G + r % p.G) * kLog2e : 0.f;
            x[n][c] -= slope * static_cast<float>(abs(j0 - hi_r[n][c]));
            x[n][c + 2] -= slope * static_cast<float>(abs(j0 + 8 - hi_r[n][c]));
          }
      }
      if constexpr (EDGE) {  // (padded rows: q = 0, never written)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!row_sees(p, pc, (rg * NT + n) * 8 + 2 * t4 + (e & 1), j0 + (e >> 1) * 8))
              x[n][e] = -INFINITY;
      }
      if (p.scores != nullptr) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* dst = p.scores + ((static_cast<long long>(pc.b) * p.Hkv + kh) * p.max_blocks * p.tiles_per_block +
                                   key0 / kTileKeys) * (RG * NT * 128) + (rg * NT + n) * 128 + g * 8 + 2 * t4;
          __stcg(reinterpret_cast<float2*>(dst), make_float2(x[n][0], x[n][1]));
          __stcg(reinterpret_cast<float2*>(dst + 64), make_float2(x[n][2], x[n][3]));
        }
      }
      // ---- softmax: weights relative to a reference that is at most 2^8 below a score,
      // times 2^7, so that they stay below fp16's end and its last bit is 2^-31 of the
      // reference's weight
      bool up = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          up |= fmaxf(x[n][c], x[n][c + 2]) - m_r[n][c] > 8.f;  // (no key seen: m = -inf)
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(x[n][c], x[n][c + 2]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            // (each row goes by its own scores: its bits do not depend on the tiles' other rows)
            mx = mx - m_r[n][c] > 8.f ? mx : m_r[n][c];
            const float al = m_r[n][c] == -INFINITY ? 1.f : ex2(m_r[n][c] - mx);  // (O and l are zero before the first)
            m_r[n][c] = mx;
            l_r[n][c] *= al;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[mt][n][c] *= al;
              o[mt][n][c + 2] *= al;
            }
          }
      }
      uint32_t pb[NT][2], pl[NT][2] = {};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float b0 = m_r[n][0] == -INFINITY ? 0.f : 7.f - m_r[n][0];
        const float b1 = m_r[n][1] == -INFINITY ? 0.f : 7.f - m_r[n][1];
        const float p0 = ex2(x[n][0] + b0), p1 = ex2(x[n][1] + b1), p2 = ex2(x[n][2] + b0), p3 = ex2(x[n][3] + b1);
        l_r[n][0] += p0 + p2;
        l_r[n][1] += p1 + p3;
        const uint32_t w0 = pack_half2(p0, p1), w1 = pack_half2(p2, p3);
        pb[n][0] = movmatrix_trans(w0);
        pb[n][1] = movmatrix_trans(w1);
        if constexpr (PP == 2) {
          const float2 h0 = unpack2<false>(w0), h1 = unpack2<false>(w1);
          pl[n][0] = movmatrix_trans(pack_half2(p0 - h0.x, p1 - h0.y));
          pl[n][1] = movmatrix_trans(pack_half2(p2 - h1.x, p3 - h1.y));
        }
      }
      // ---- O^T += V^T P^T
      fp4_pv<D, NT, PP, EDGE>(p, pc, rg * NT * 8, stage + Cfg::kCodes, stage + 2 * Cfg::kCodes + Cfg::kScales, lane, key0,
                              seq_len, pb, pl, o);
    };
    for (int i = 0; i < steps; ++i) {
      cp_async_wait<ST - 2>();
      __syncwarp();  // the step's scales are there, and every lane is done with the stage that is filled next
      issue();
      const int key0 = piece_tile(p, pc, i * KG + kg) * kTileKeys;
      if ((key0 >= lo_all && key0 + kTileKeys - 1 <= hi_all) || (key0 + kTileKeys <= prefix && hi_all >= 0))
        step(i, std::false_type());
      else
        step(i, std::true_type());
      stage = stage == ring + (ST - 1) * Cfg::kStage ? ring : stage + Cfg::kStage;
    }

    // ---- the warps' (m, l, O) meet; m becomes what the weights are relative to
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l_r[n][c] += __shfl_xor_sync(0xffffffffu, l_r[n][c], off);
        if (l_r[n][c] != l_r[n][c] && m_r[n][c] == -INFINITY) m_r[n][c] = 0.f;  // nothing but NaN: not an empty row
        if (g == 0) s_ml[warp * NT * 8 + n * 8 + 2 * t4 + c] = make_float2(m_r[n][c] - 7.f, l_r[n][c]);
      }
    cp_async_wait<0>();
    __syncwarp();  // (every lane is done with the warp's ring)
    float4* mine = reinterpret_cast<float4*>(smem + warp * Cfg::kRing);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        mine[(n * MT + mt) * Cfg::kPitch + lane] = make_float4(o[mt][n][0], o[mt][n][1], o[mt][n][2], o[mt][n][3]);
    __syncthreads();
    fp4_join<Cfg, D, NT, RG, KG, Cfg::kThreads>(p, pc, smem, s_ml);
    __syncthreads();  // the rings are free again
  }
}

}  // namespace pd
