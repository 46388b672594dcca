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
// waits). What differs is what the two maps make possible: the two warps of a
// head's pair split D in halves, and a half of a K row belongs to one map
// only. So warp m scores map m over its whole contraction (no partial scores to
// add) and runs that map's softmax alone; the pair then swaps its packed P
// fragments and rescale factors through shared memory (16 bytes per lane and
// row tile, one 64-thread barrier per tile) and each warp accumulates both
// maps over its own half of V's dims. Every K and V byte is thus read from
// shared memory, and a one-byte code widened, once for both maps.
// Each warp pair holds one to four tiles of 8 query rows per map (G * qlen <=
// 32), dealt to RG row groups.
//
// A unit covered by one piece is finished from the accumulators: the pair
// exchanges row sums, takes the difference in fp32 and, with a norm, the sums
// of squares. A split unit's pieces write fp32 (m, l, O) partials of both
// maps, which diff_combine_kernel joins.
#pragma once
#include <cuda_bf16.h>

#include "decode_kernel.cuh"

namespace pd {

struct DiffParams {
  DecodeParams d;
  const float* lambda;      // [Hq]
  const void* norm_weight;  // [D] or null
  int norm_f32;             // norm_weight is fp32 (else q's type)
  float norm_eps, norm_gain;
};

template <int D_, int KV_, int NTM_, int RG_, int NS_, int MINB_, int HG_>
struct DiffCfg {
  static constexpr int D = D_, KV = KV_, NTM = NTM_, RG = RG_, NS = NS_, HG = HG_;
  static constexpr int kMinBlocks = MINB_;
  static constexpr bool BYTE = KV == kKvFp8 || KV == kKvInt8;
  static constexpr bool BF16 = KV == kKvBf16;  // bfloat16 operands; byte kinds use fp16 ones
  static constexpr int kElem = BYTE ? 1 : 2;
  static constexpr int kSlabElems = 128 / kElem;
  static constexpr int kSlabs = D / kSlabElems;
  static constexpr int kSlabBytes = kTileKeys * HG * 128;  // [key][head][128 B]
  static constexpr int kTileBytes = kSlabs * kSlabBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static_assert(NTM % RG == 0, "row groups take equal shares of the row tiles");
  static constexpr int NTW = NTM / RG;  // row tiles (per map) of a warp
  static constexpr int kPairs = HG * RG;
  static constexpr int kConsumerWarps = 2 * kPairs;
  static constexpr int kThreads = kConsumerWarps * 32 + 32;
  static constexpr int RM = NTM * 8;      // partial rows per map of a head
  static constexpr int RH = 2 * RM;       // per head
  static constexpr int RP = HG * RH;      // per unit
  // a pair's exchange: two buffers of (own fragments of each map), and the
  // epilogue's row sums
  static constexpr int kXBuf = 32 * NTW * 16;  // one warp's 16 bytes per lane and row tile
  static constexpr int kXPair = 2 * 2 * kXBuf + 2 * kXBuf;
  static constexpr int kOffX = NS * kStageBytes;
  static constexpr int kOffBars = kOffX + kPairs * kXPair;
  static constexpr int kOffPre = kOffBars + 2 * NS * 8;
  static constexpr int kSmemBytes = (kOffPre + (kMaxAutoB + 1) * 4 + 15) / 16 * 16 + 1024;
  static_assert(kPairs <= 14, "named barriers 2..");
};

// Output value of row sums: the difference of the two maps.
__device__ __forceinline__ float diff_of(float o1, float o2, float inv1, float inv2l) { return o1 * inv1 - o2 * inv2l; }

__device__ __forceinline__ float norm_weight_at(const DiffParams& p, int d) {
  if (p.norm_f32) return __ldg(static_cast<const float*>(p.norm_weight) + d);
  const uint16_t w = __ldg(static_cast<const uint16_t*>(p.norm_weight) + d);
  return p.d.out_bf16 ? __uint_as_float(static_cast<uint32_t>(w) << 16) : __half2float(__ushort_as_half(w));
}

__device__ __forceinline__ uint32_t pack_out(bool bf16, float lo, float hi) {
  return bf16 ? pack_bf162(lo, hi) : pack_half2(lo, hi);
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, Cfg::kMinBlocks)
    decode_diff_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const DiffParams dp) {
  const DecodeParams& p = dp.d;
  constexpr int D = Cfg::D, NS = Cfg::NS, HG = Cfg::HG, NTW = Cfg::NTW, RG = Cfg::RG;
  constexpr bool BYTE = Cfg::BYTE, BF16 = Cfg::BF16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kOffBars);  // full[NS], empty[NS]
  int* s_pre = reinterpret_cast<int*>(smem + Cfg::kOffPre);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_producer = warp == Cfg::kConsumerWarps;
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + NS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, Cfg::kConsumerWarps);
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

  if (is_producer) {
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
        const int nxt = (t + 32 < pc.ntiles) ? load_group(t + 32) : -1;
        const int n = min(32, pc.ntiles - t);
        for (int i = 0; i < n; ++i, ++q) {
          int blk = __shfl_sync(0xffffffffu, cur, i);
          if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) raise_error(p.error_flag, kErrBlockId);
            blk = 0;
          }
          const int stage = q % NS;
          const uint32_t fb = full0 + 8 * stage;
          if (lane == 0) {
            if (ok && q >= NS) ok = mbar_wait(empty0 + 8 * stage, ((q / NS) - 1) & 1, p.timeout_ns);
            if (ok && p.inject == 1) ok = false;
            if (ok) mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) continue;
          if (lane < 2 * Cfg::kSlabs) {
            const int tile = pc.first_tile + t + i;
            const int z = blk * p.block_size + (tile % p.tiles_per_block) * kTileKeys;
            const int sl = lane % Cfg::kSlabs;
            const bool is_v = lane >= Cfg::kSlabs;
            const uint32_t dst = smem_u32(smem + stage * Cfg::kStageBytes) + (is_v ? Cfg::kTileBytes : 0) +
                                 sl * Cfg::kSlabBytes;
            tma_load_3d(dst, is_v ? &tm_v : &tm_k, fb, sl * Cfg::kSlabElems, pc.kh, z, pol);
          }
          issued = q + 1;
        }
        cur = nxt;
      }
    }
    if (lane == 0) {
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
  const int map = warp & 1;                  // the map this warp scores; its half of V's dims
  const int pair = warp >> 1, rg = pair % RG, th = pair / RG;
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int KSW = D / 32;                // k-steps of one map (D / 2 dims)
  constexpr int MTW = D / 32;                // m-tiles of 16 output dims of this warp
  uint8_t* xch = smem + Cfg::kOffX + pair * Cfg::kXPair;
  float4* xend = reinterpret_cast<float4*>(xch + 4 * Cfg::kXBuf);  // [map][tile][lane] row sums
  // One-byte tiles at D = 128: a map's half of a slab row is four 16-byte
  // chunks, and the eight lanes of a shared-memory phase hold two rows of
  // four; rows whose swizzle phases differ in their high bit use different
  // halves of the banks, so lane row g stands for key (g & 1) * 4 + (g >> 1).
  constexpr bool kPermute = BYTE && D == 128;
  auto key_of = [](int r) { return kPermute ? (r & 1) * 4 + (r >> 1) : r; };
  const int kg0 = key_of(g);                 // key of accumulator row g (row g + 8: + 8)
  uint32_t qf[KSW][NTW][2];
  float o[2][MTW][NTW][4];                   // [own map, other map]
  uint32_t q = 0;
  bool ok = true;

  while (work_next(p, s_pre, it, pc)) {
    // ---- q fragments of this warp's map
    float sl2r[NTW][2];
#pragma unroll
    for (int n = 0; n < NTW; ++n) {
      sl2r[n][0] = sl2r[n][1] = p.sl2;
      const int r = (rg * NTW + n) * 8 + g;
      const __half* qrow = nullptr;
      if (r < pc.R && pc.ntiles > 0) {
        const int i = r / p.G, hl = r % p.G;
        qrow = p.q + (static_cast<long long>(pc.q0 + i) * p.Hq + (pc.kh + th) * p.G + hl) * D + map * (D / 2);
      }
#pragma unroll
      for (int ks = 0; ks < KSW; ++ks) {
        int d0, d1;  // dims within the half
        if constexpr (!BYTE) {
          d0 = ks * 16 + 2 * t4;
          d1 = d0 + 8;
        } else if constexpr (D == 256) {
          // super-step ss = ks / 4 of the half's slab: chunk 2 t4 + ss
          d0 = 16 * (2 * t4 + (ks >> 2)) + 4 * (ks & 3);
          d1 = d0 + 2;
        } else {
          d0 = 16 * t4 + 4 * ks;
          d1 = d0 + 2;
        }
        qf[ks][n][0] = qrow ? __ldg(reinterpret_cast<const uint32_t*>(qrow + d0)) : 0u;
        qf[ks][n][1] = qrow ? __ldg(reinterpret_cast<const uint32_t*>(qrow + d1)) : 0u;
      }
    }
    if constexpr (BYTE) {
      if (p.out_bf16) {
        // bfloat16 q over byte caches: the half row scaled by 2^e into fp16,
        // exactly; 2^-e joins the row's score factor
#pragma unroll
        for (int n = 0; n < NTW; ++n) {
          float m = 0.f;
#pragma unroll
          for (int ks = 0; ks < KSW; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = qf[ks][n][h];
              m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
            }
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const int e = q_row_exponent(m);
          sl2r[n][0] = p.sl2 * pow2f(-__shfl_sync(0xffffffffu, e, 8 * t4));
          sl2r[n][1] = p.sl2 * pow2f(-__shfl_sync(0xffffffffu, e, 8 * t4 + 4));
          const float up = pow2f(e);
#pragma unroll
          for (int ks = 0; ks < KSW; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = qf[ks][n][h];
              qf[ks][n][h] = pack_half2(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
            }
        }
      }
    }
    int lo_r[NTW][2], hi_r[NTW][2];
    float m_r[NTW][2], l_r[NTW][2];
#pragma unroll
    for (int n = 0; n < NTW; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = (rg * NTW + n) * 8 + 2 * t4 + c;
        if (r < pc.R) {
          const int pos = pc.L - pc.qlen + r / p.G;
          hi_r[n][c] = pos;
          lo_r[n][c] = (p.window > 0) ? max(0, pos - p.window + 1) : 0;
        } else {
          hi_r[n][c] = -1;
          lo_r[n][c] = 0;
        }
        m_r[n][c] = -INFINITY;
        l_r[n][c] = 0.f;
      }
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int mt = 0; mt < MTW; ++mt) o[w][mt][n][0] = o[w][mt][n][1] = o[w][mt][n][2] = o[w][mt][n][3] = 0.f;
    }

    for (int k = 0; k < pc.ntiles; ++k) {
      const uint32_t qq = q + k;
      const int stage = qq % NS;
      if (ok) ok = mbar_wait(full0 + 8 * stage, (qq / NS) & 1, p.timeout_ns);
      if (!ok) {
        named_bar_sync(2 + pair, 64);  // keep the pair's barrier sequence
        continue;
      }
      const uint32_t kb = smem_u32(smem + stage * Cfg::kStageBytes);
      const uint32_t vb = kb + Cfg::kTileBytes;
      const int key0 = (pc.first_tile + k) * kTileKeys;

      // ---- S^T of this warp's map: 16 keys x 8 rows per row tile, over D / 2
      float sa[NTW][4], sb[NTW][4];
#pragma unroll
      for (int n = 0; n < NTW; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sa[n][e] = sb[n][e] = 0.f;
      if constexpr (!BYTE) {
        const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
        const int srow = key * HG + th;
        const uint32_t rowb = kb + srow * 128;
#pragma unroll
        for (int ksl = 0; ksl < KSW; ++ksl) {
          const int ks = map * KSW + ksl;
          const int slab = ks >> 2, chunk = (ks & 3) * 2 + (lane >> 4);
          uint32_t a[4];
          ldsm_x4(rowb + slab * Cfg::kSlabBytes + ((chunk ^ (srow & 7)) << 4), a);
#pragma unroll
          for (int n = 0; n < NTW; ++n) {
            if (ksl & 1) mma_op<BF16>(sb[n], a, qf[ksl][n][0], qf[ksl][n][1]);
            else mma_op<BF16>(sa[n], a, qf[ksl][n][0], qf[ksl][n][1]);
          }
        }
      } else {
        const int srow = kg0 * HG + th;
        const uint32_t r0 = kb + srow * 128, r8 = kb + (srow + 8 * HG) * 128;
#pragma unroll
        for (int sup = 0; sup < KSW / 4; ++sup) {
          const int slab = D == 256 ? map : 0;
          const int chunk = (D == 256 ? 2 * t4 + sup : 4 * map + t4) ^ (srow & 7);
          uint4 w0, w8;
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(w0.x), "=r"(w0.y), "=r"(w0.z), "=r"(w0.w)
                       : "r"(r0 + slab * Cfg::kSlabBytes + (chunk << 4)));
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(w8.x), "=r"(w8.y), "=r"(w8.z), "=r"(w8.w)
                       : "r"(r8 + slab * Cfg::kSlabBytes + (chunk << 4)));
          const uint32_t wa[4] = {w0.x, w0.y, w0.z, w0.w};
          const uint32_t wb[4] = {w8.x, w8.y, w8.z, w8.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int ksl = sup * 4 + j;
            uint32_t a[4];
            const uint32_t xa = byte_word_prep<Cfg::KV>(wa[j]), xb = byte_word_prep<Cfg::KV>(wb[j]);
            a[0] = byte_pair_to_half2<Cfg::KV>(xa, false);
            a[1] = byte_pair_to_half2<Cfg::KV>(xb, false);
            a[2] = byte_pair_to_half2<Cfg::KV>(xa, true);
            a[3] = byte_pair_to_half2<Cfg::KV>(xb, true);
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
              if (j & 1) mma_op<BF16>(sb[n], a, qf[ksl][n][0], qf[ksl][n][1]);
              else mma_op<BF16>(sa[n], a, qf[ksl][n][0], qf[ksl][n][1]);
            }
          }
        }
      }
      // ---- mask and online softmax of this map; P rounded to the operands'
      // 16-bit type (the sum l is of the unrounded exponentials)
      uint32_t pf[2][NTW][2];  // [own, other] P^T fragments
      float al[2][NTW][2];     // [own, other] rescale factors
      const bool interior = key0 >= pc.tile_lo_all && key0 + kTileKeys - 1 <= pc.tile_hi_all;
      uint4* buf = reinterpret_cast<uint4*>(xch + (qq & 1) * 2 * Cfg::kXBuf);  // [map][tile][lane]
#pragma unroll
      for (int n = 0; n < NTW; ++n) {
        const int j0 = key0 + kg0, j1 = j0 + 8;
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = (sa[n][e] + sb[n][e]) * sl2r[n][e & 1];
        if (interior) {
          if (hi_r[n][0] < 0) x[0] = x[2] = -INFINITY;  // padded rows stay masked
          if (hi_r[n][1] < 0) x[1] = x[3] = -INFINITY;
        } else {
          if (!(j0 >= lo_r[n][0] && j0 <= hi_r[n][0])) x[0] = -INFINITY;
          if (!(j0 >= lo_r[n][1] && j0 <= hi_r[n][1])) x[1] = -INFINITY;
          if (!(j1 >= lo_r[n][0] && j1 <= hi_r[n][0])) x[2] = -INFINITY;
          if (!(j1 >= lo_r[n][1] && j1 <= hi_r[n][1])) x[3] = -INFINITY;
        }
        float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
        }
        const float mn0 = fmaxf(m_r[n][0], mx0), mn1 = fmaxf(m_r[n][1], mx1);
        const float base0 = (mn0 == -INFINITY) ? 0.f : mn0;
        const float base1 = (mn1 == -INFINITY) ? 0.f : mn1;
        al[0][n][0] = (m_r[n][0] == -INFINITY) ? 1.f : ex2(m_r[n][0] - base0);
        al[0][n][1] = (m_r[n][1] == -INFINITY) ? 1.f : ex2(m_r[n][1] - base1);
        const float p00 = ex2(x[0] - base0), p01 = ex2(x[1] - base1);
        const float p10 = ex2(x[2] - base0), p11 = ex2(x[3] - base1);
        m_r[n][0] = mn0;
        m_r[n][1] = mn1;
        l_r[n][0] = l_r[n][0] * al[0][n][0] + (p00 + p10);
        l_r[n][1] = l_r[n][1] * al[0][n][1] + (p01 + p11);
        pf[0][n][0] = movmatrix_trans(pack2<BF16>(p00, p01));
        pf[0][n][1] = movmatrix_trans(pack2<BF16>(p10, p11));
        buf[(map * NTW + n) * 32 + lane] = make_uint4(pf[0][n][0], pf[0][n][1], __float_as_uint(al[0][n][0]),
                                                      __float_as_uint(al[0][n][1]));
      }
      named_bar_sync(2 + pair, 64);
      bool rescale = false;
#pragma unroll
      for (int n = 0; n < NTW; ++n) {
        const uint4 w = buf[((map ^ 1) * NTW + n) * 32 + lane];
        pf[1][n][0] = w.x;
        pf[1][n][1] = w.y;
        al[1][n][0] = __uint_as_float(w.z);
        al[1][n][1] = __uint_as_float(w.w);
        rescale |= al[0][n][0] != 1.f || al[0][n][1] != 1.f || al[1][n][0] != 1.f || al[1][n][1] != 1.f;
      }
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int mt = 0; mt < MTW; ++mt)
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
              o[w][mt][n][0] *= al[w][n][0]; o[w][mt][n][1] *= al[w][n][1];
              o[w][mt][n][2] *= al[w][n][0]; o[w][mt][n][3] *= al[w][n][1];
            }
      }

      // ---- O^T += V^T P^T of both maps over this warp's half of the dims; V
      // of keys at or past the sequence end is zeroed (its bits may be NaN)
      const bool tail = key0 + kTileKeys > pc.L;
      if constexpr (!BYTE) {
        const int key = (lane & 7) + (lane >> 4) * 8;
        const int srow = key * HG + th;
        const uint32_t rowb = vb + srow * 128;
        uint32_t vm01 = 0xffffffffu, vm23 = 0xffffffffu;
        if (tail) {
          const int k0 = key0 + 2 * t4;
          vm01 = (k0 < pc.L ? 0x0000ffffu : 0u) | (k0 + 1 < pc.L ? 0xffff0000u : 0u);
          vm23 = (k0 + 8 < pc.L ? 0x0000ffffu : 0u) | (k0 + 9 < pc.L ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int mtl = 0; mtl < MTW; ++mtl) {
          const int mt = map * MTW + mtl;
          const int slab = mt >> 2, chunk = (mt & 3) * 2 + ((lane >> 3) & 1);
          uint32_t a[4];
          ldsm_x4_trans(rowb + slab * Cfg::kSlabBytes + ((chunk ^ (srow & 7)) << 4), a);
          if (tail) {
            a[0] &= vm01; a[1] &= vm01; a[2] &= vm23; a[3] &= vm23;
          }
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int n = 0; n < NTW; ++n) mma_op<BF16>(o[w][mtl][n], a, pf[w][n][0], pf[w][n][1]);
        }
      } else {
        const int kA = key_of(2 * t4), kB = key_of(2 * t4 + 1), kC = kA + 8, kD = kB + 8;
        const int rA = kA * HG + th, rB = kB * HG + th, rC = kC * HG + th, rD = kD * HG + th;
#pragma unroll
        for (int pl = 0; pl < MTW / 2; ++pl) {
          const int P32 = map * (MTW / 2) + pl;
          const int slab = P32 >> 2;
          const int chunk = (P32 & 3) * 2 + (g >> 2);
          const int byte = (4 * g) & 15;
          const uint32_t sb0 = vb + slab * Cfg::kSlabBytes + byte;
          uint32_t wA, wB, wC, wD;
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wA) : "r"(sb0 + rA * 128 + ((chunk ^ (rA & 7)) << 4)));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wB) : "r"(sb0 + rB * 128 + ((chunk ^ (rB & 7)) << 4)));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wC) : "r"(sb0 + rC * 128 + ((chunk ^ (rC & 7)) << 4)));
          asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wD) : "r"(sb0 + rD * 128 + ((chunk ^ (rD & 7)) << 4)));
          if (tail) {  // code 0 is the value 0 in both byte formats
            if (key0 + kA >= pc.L) wA = 0u;
            if (key0 + kB >= pc.L) wB = 0u;
            if (key0 + kC >= pc.L) wC = 0u;
            if (key0 + kD >= pc.L) wD = 0u;
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
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int n = 0; n < NTW; ++n) mma_op<BF16>(o[w][2 * pl][n], a, pf[w][n][0], pf[w][n][1]);
          a[0] = byte_pair_to_half2<Cfg::KV>(ab23, false);
          a[1] = byte_pair_to_half2<Cfg::KV>(ab23, true);
          a[2] = byte_pair_to_half2<Cfg::KV>(cd23, false);
          a[3] = byte_pair_to_half2<Cfg::KV>(cd23, true);
#pragma unroll
          for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int n = 0; n < NTW; ++n) mma_op<BF16>(o[w][2 * pl + 1][n], a, pf[w][n][0], pf[w][n][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * stage);
    }
    q += pc.ntiles;

    // ---- end of the piece: row sums over the lanes of each row
#pragma unroll
    for (int n = 0; n < NTW; ++n)
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l_r[n][0] += __shfl_xor_sync(0xffffffffu, l_r[n][0], off);
        l_r[n][1] += __shfl_xor_sync(0xffffffffu, l_r[n][1], off);
      }
    // output dims of accumulator registers e = 0/1 and 2/3 of m-tile mtl
    auto dim0 = [&](int mtl) {
      const int mt = map * MTW + mtl;
      return BYTE ? (mt >> 1) * 32 + 4 * g + 2 * (mt & 1) : mt * 16 + g;
    };
    constexpr int kStep = BYTE ? 1 : 8;
    if (pc.npieces > 1) {
#pragma unroll
      for (int n = 0; n < NTW; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = (rg * NTW + n) * 8 + 2 * t4 + c;
          if (r >= pc.R) continue;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const long long prow = static_cast<long long>(pc.slot) * Cfg::RP + th * Cfg::RH + (map ^ w) * Cfg::RM + r;
            float* dst = p.ws_o + prow * D;
#pragma unroll
            for (int mtl = 0; mtl < MTW; ++mtl) {
              const int d0 = dim0(mtl);
              if constexpr (BYTE) {
                __stcg(reinterpret_cast<float2*>(dst + d0), make_float2(o[w][mtl][n][c], o[w][mtl][n][2 + c]));
              } else {
                __stcg(dst + d0, o[w][mtl][n][c]);
                __stcg(dst + d0 + 8, o[w][mtl][n][2 + c]);
              }
            }
            if (w == 0 && g == 0)
              __stcg(reinterpret_cast<float2*>(p.ws_ml + prow * 2), make_float2(m_r[n][c], l_r[n][c]));
          }
        }
      continue;
    }
    // ---- the whole unit: swap row sums, take the difference, normalise. A
    // piece with tiles had a barrier per tile after the last use of xend; one
    // without has all sums zero and swaps nothing.
    float lo_sum[NTW][2];  // the other map's row sums
#pragma unroll
    for (int n = 0; n < NTW; ++n) lo_sum[n][0] = lo_sum[n][1] = 0.f;
    if (pc.ntiles > 0) {
#pragma unroll
      for (int n = 0; n < NTW; ++n) xend[(map * NTW + n) * 32 + lane] = make_float4(l_r[n][0], l_r[n][1], 0.f, 0.f);
      named_bar_sync(2 + pair, 64);
#pragma unroll
      for (int n = 0; n < NTW; ++n) {
        const float4 w = xend[((map ^ 1) * NTW + n) * 32 + lane];
        lo_sum[n][0] = w.x;
        lo_sum[n][1] = w.y;
      }
    }
    float ss[NTW][2];
#pragma unroll
    for (int n = 0; n < NTW; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ss[n][c] = 0.f;
        const int r = (rg * NTW + n) * 8 + 2 * t4 + c;
        const float l1 = map == 0 ? l_r[n][c] : lo_sum[n][c], l2 = map == 0 ? lo_sum[n][c] : l_r[n][c];
        const float lam = r < pc.R ? __ldg(dp.lambda + (pc.kh + th) * p.G + r % p.G) : 0.f;
        const float inv1 = l1 > 0.f ? p.out_scale / l1 : 0.f;
        const float inv2 = l2 > 0.f ? p.out_scale / l2 * lam : 0.f;
#pragma unroll
        for (int mtl = 0; mtl < MTW; ++mtl)
#pragma unroll
          for (int e = c; e < 4; e += 2) {
            const float own = o[0][mtl][n][e], other = o[1][mtl][n][e];
            const float v = map == 0 ? diff_of(own, other, inv1, inv2) : diff_of(other, own, inv1, inv2);
            o[0][mtl][n][e] = v;
            ss[n][c] += v * v;
          }
      }
    float f[NTW][2];
#pragma unroll
    for (int n = 0; n < NTW; ++n) f[n][0] = f[n][1] = 1.f;
    if (dp.norm_weight != nullptr) {
#pragma unroll
      for (int n = 0; n < NTW; ++n)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          ss[n][0] += __shfl_xor_sync(0xffffffffu, ss[n][0], off);
          ss[n][1] += __shfl_xor_sync(0xffffffffu, ss[n][1], off);
        }
      if (pc.ntiles > 0) {
        named_bar_sync(2 + pair, 64);  // xend has been read
#pragma unroll
        for (int n = 0; n < NTW; ++n) xend[(map * NTW + n) * 32 + lane] = make_float4(ss[n][0], ss[n][1], 0.f, 0.f);
        named_bar_sync(2 + pair, 64);
#pragma unroll
        for (int n = 0; n < NTW; ++n) {
          const float4 w = xend[((map ^ 1) * NTW + n) * 32 + lane];
          ss[n][0] += w.x;
          ss[n][1] += w.y;
        }
      }
#pragma unroll
      for (int n = 0; n < NTW; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) f[n][c] = rsqrtf(ss[n][c] / static_cast<float>(D) + dp.norm_eps) * dp.norm_gain;
    }
#pragma unroll
    for (int mtl = 0; mtl < MTW; ++mtl) {
      const int d0 = dim0(mtl);
      float w0 = 1.f, w1 = 1.f;
      if (dp.norm_weight != nullptr) {
        w0 = norm_weight_at(dp, d0);
        w1 = norm_weight_at(dp, d0 + kStep);
      }
#pragma unroll
      for (int n = 0; n < NTW; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = (rg * NTW + n) * 8 + 2 * t4 + c;
          if (r >= pc.R) continue;
          uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) +
                          (static_cast<long long>(pc.q0 + r / p.G) * p.Hq + (pc.kh + th) * p.G + r % p.G) * D;
          // (a zero row with eps = 0: rsqrt is infinite, the row stays zero)
          const float a = o[0][mtl][n][c], b = o[0][mtl][n][2 + c];
          const uint32_t v = pack_out(p.out_bf16 != 0, a == 0.f ? 0.f : a * f[n][c] * w0, b == 0.f ? 0.f : b * f[n][c] * w1);
          if constexpr (BYTE) {
            *reinterpret_cast<uint32_t*>(dst + d0) = v;
          } else {
            dst[d0] = static_cast<uint16_t>(v & 0xffffu);
            dst[d0 + kStep] = static_cast<uint16_t>(v >> 16);
          }
        }
    }
  }
  if (!ok && lane == 0) raise_error(p.error_flag, kErrTimeout);
}

// ---------------------------------------------------------------------------
// Joins the partials of every split unit (unit_layout, merge_pieces), takes the
// difference of the two maps and, with a norm, normalises the row.
//   grid (units, row chunks, heads per tile), NT threads. A row's items are its
//   2 maps x D / 4 groups of four dims; RB rows are taken at a time with PG =
//   NT / (RB * items) threads per item, which share the item's pieces (pg, pg +
//   PG, ...) and are joined in pg order, so the result does not depend on
//   scheduling.
template <int D, int NB, int NT>
__global__ void __launch_bounds__(NT) diff_combine_kernel(const DiffParams dp, int RB) {
  const DecodeParams& p = dp.d;
  constexpr int S4 = D / 4, ITEMS = 2 * S4;
  __shared__ float s_m[NT], s_l[NT];
  __shared__ float4 s_o[NT];
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
  const int rbase = blockIdx.z * p.rows_head, rmap = p.rows_head / 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (P <= 1) return;
  const int live = p.G * qn;
  const int chunk = (live + gridDim.y - 1) / gridDim.y;
  const int r_begin = blockIdx.y * chunk, r_end = min(live, r_begin + chunk);
  const int t = threadIdx.x, width = RB * ITEMS, PG = NT / width;
  const int item = t % width, pg = t / width;
  const int j = item / ITEMS, map = (item / S4) & 1, c4 = item % S4;
  for (int r0 = r_begin; r0 < r_end; r0 += RB) {
    const int r = r0 + j;
    float m_run = -INFINITY, l_run = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < r_end && pg < PG)
      merge_pieces<D, NB>(p, P, slot0, slot_base, step, rbase, map * rmap + r, 4 * c4, pg, PG, m_run, l_run, acc);
    s_m[t] = m_run;
    s_l[t] = l_run;
    s_o[t] = acc;
    __syncthreads();
    // the threads of pg = 0 join the groups and leave out_scale O / l
    if (t < width && PG > 1) {
      float M = -INFINITY;
      for (int k = 0; k < PG; ++k) M = fmaxf(M, s_m[k * width + t]);
      l_run = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < PG; ++k) {
        const float mk = s_m[k * width + t];
        if (mk == -INFINITY) continue;
        const float w = ex2(mk - M);
        l_run += w * s_l[k * width + t];
        const float4 v = s_o[k * width + t];
        acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
      }
    }
    if (t < width) {
      const float lam = map == 0 || r >= r_end ? 1.f : __ldg(dp.lambda + kh * p.G + r % p.G);
      const float inv = l_run > 0.f ? p.out_scale / l_run * lam : 0.f;
      s_o[t] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
    __syncthreads();
    // thread (row jj, four dims)
    const int jj = t / S4, cc = t % S4, rr = r0 + jj;
    const bool on = jj < RB && rr < r_end;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
      const float4 a = s_o[jj * ITEMS + cc], c = s_o[jj * ITEMS + S4 + cc];
      v = make_float4(a.x - c.x, a.y - c.y, a.z - c.z, a.w - c.w);
    }
    if (dp.norm_weight != nullptr) {
      float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (S4 > 32) {  // a row spans two warps
        if ((t & 31) == 0) s_ss[t >> 5] = ss;
        __syncthreads();
        ss = s_ss[(t >> 5) & ~1] + s_ss[(t >> 5) | 1];
      }
      if (on) {
        const float f = rsqrtf(ss / static_cast<float>(D) + dp.norm_eps) * dp.norm_gain;
        v.x = v.x == 0.f ? 0.f : v.x * f * norm_weight_at(dp, 4 * cc);
        v.y = v.y == 0.f ? 0.f : v.y * f * norm_weight_at(dp, 4 * cc + 1);
        v.z = v.z == 0.f ? 0.f : v.z * f * norm_weight_at(dp, 4 * cc + 2);
        v.w = v.w == 0.f ? 0.f : v.w * f * norm_weight_at(dp, 4 * cc + 3);
      }
    }
    if (on) {
      uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) +
                      (static_cast<long long>(q0 + rr / p.G) * p.Hq + kh * p.G + rr % p.G) * D + 4 * cc;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_out(p.out_bf16 != 0, v.x, v.y), pack_out(p.out_bf16 != 0, v.z, v.w));
    }
    __syncthreads();  // s_o free again
  }
}

}  // namespace pd
