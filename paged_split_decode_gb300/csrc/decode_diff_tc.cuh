// decode_diff_tc.cuh -- differential decode for byte caches on the
// 5th-generation tensor cores (tcgen05, accumulators in tensor memory), for
// units with 9 or more query rows per map of a KV head (speculative verify).
//
// The formula and the work split are decode_diff.cuh's, the engine is the plain
// decode's tensor-memory kernel (decode_tci8.cuh), whose rings, barriers and
// widening it takes: 128-key blocks of eight tiles, two producer warps (K, V),
// one issuing thread, and softmax warps in NG groups of four, thread i of a
// group owning key i of a block (and output dims i, i + 128). What two maps
// change:
//  * A half of a K row meets one map only, so S^T of map m is the product of the
//    k-steps of half m: as many tcgen05.mma as one map over whole rows takes.
//    Both maps' weights stand side by side on the N side of O^T += V^T P^T, so V
//    is widened, read and multiplied once for both.
//  * Group g owns rows 8 g .. 8 g + 7 of both maps: one barrier decides for 16
//    rows whether a maximum is raised, and a thread holds the same dims of both
//    maps at the end, so their difference is its own.
//  * int8: codes are widened to fp16 exactly, as there (but K by widen_i8x16
//    too: the plain decode's offset would round in both maps). P^T is fp16, a
//    32-byte row per key and group, a 16-byte half per map (32-byte swizzle). (NG
//    = 4 at D = 256 does not fit beside the widened V and stays on
//    decode_diff.cuh.)
//  * e4m3: the products read the codes themselves (kind::f8f6f4), as in
//    decode_tc8.cuh: no widening at all. q is the sum of two (bfloat16) or three
//    (fp16) e4m3 terms, summed in the one accumulator of S^T. A weight is rounded
//    to fp16 and cut into three e5m2 terms, the second and third scaled by 2^4 and
//    2^8: every fp16 value in [0, 2^15] is the sum of its terms exactly, by bit
//    operations and subtractions alone (split_weight). The terms stand side by side
//    on the N side of P.V, their accumulators are added with their scales at a
//    piece's end.
//  * Weights are 2^15 where a score reaches its row's threshold, so that fp16 keeps
//    11 bits of them down to 2^-29 of that and the last down to 2^-39: a key of few
//    weights does not vanish beside a peak (it is what two maps leave of each other
//    once their peaks cancel). e4m3 terms reach 2^-22 of a peak, and in a map with one
//    key 16 nats above 32767 others a percent of it was lost.
//  * The row sums add the rounded weights. V rows of keys beyond the end are
//    zeros, so that stale NaN codes never meet a zero weight.
//  * S^T at NG = 3 also reads q rows 24 .. 31 of the operand, which belong to the
//    next term or slab: columns that nobody reads.
// Every wait is bounded as in decode_tc8.cuh.
#pragma once
#include "decode_diff.cuh"
#include "decode_tci8.cuh"

namespace pd {

template <int D_, int KV_, int NG_>
struct DiffTc {
  static constexpr int D = D_, KV = KV_, NG = NG_;
  static constexpr int kSlabs = D / 128;              // 128-byte slabs of a key row; 128-dim halves of O^T
  static constexpr int kBlkTiles = 8;                 // 16-key tiles per 128-key block
  static constexpr bool CODES = KV == kKvFp8;         // the products read the codes; else they are widened
  static constexpr int kTileBytes = kTileKeys * D;
  static constexpr int kBlkBytes = kBlkTiles * kTileBytes;
  // A block in a ring: [slab][128 keys][128 B], one TMA box per tile and slab,
  // where the products read it; [tile][slab][16 keys][128 B], one box per tile,
  // where it is widened.
  static constexpr int NBK = D == 256 ? 2 : 4;                        // stages of the K ring
  static constexpr int NBV = CODES ? (D == 256 ? 3 : 5) : NBK;        // of the V ring (CODES: until P.V is done)
  static constexpr int kSlabBlk = 128 * 128;
  static constexpr int kChunks = D / 16;              // 16-code chunks of a key row
  static constexpr int kV16Slab = 128 * 128;          // fp16 V, 64 dims of a block: [128 keys][128 B]
  static constexpr int kV16Bytes = CODES ? 0 : (D / 64) * kV16Slab;
  static constexpr int kRows = 8 * NG;                // rows per map
  static constexpr int kTerms = CODES ? 3 : 1;        // terms of a weight
  // e4m3: terms of q that stand side by side on the N side of S^T, two where the
  // tensor memory holds it (B = 8, L = 8192, qlen = 3: 16 products of one term
  // each take 1630 cycles a block to issue, 43.2 us; 8 of two take 1040, 37.7). A
  // third term then comes with a fourth of zeros in a second pass, added to the
  // first.
  static constexpr int kStack = CODES && 8 * kRows + kSlabs * 3 * 16 * NG <= 512 ? 2 : 1;
  static constexpr int kQTerms = !CODES ? 1 : kStack == 2 ? 4 : 3;
  static constexpr int kQTerm = kRows * 128;          // a term of q, 128 bytes of its dims: [rows][128 B]
  static constexpr int kQSlab = kQTerms * kQTerm;
  static constexpr int kQSlabs = CODES ? kSlabs : D / 64;
  static constexpr int kPtAtom = 128 * 32;            // 32 bytes of N of P^T: [128 keys][32 B]
  static constexpr int kPtBytes = (CODES ? (3 * NG + 1) / 2 : NG) * kPtAtom;
  static constexpr int kSoftThreads = 128 * NG;       // softmax warps 0 .. 4 NG - 1
  static constexpr int kThreads = kSoftThreads + 96;  // then the K and V producers and the MMA warp
  static constexpr int kProducerWarp = 4 * NG, kMmaWarp = 4 * NG + 2;
  static constexpr int kBarAll = NG + 1;              // named barrier of every softmax thread (1..NG: groups)
  static constexpr int kSN = (kStack * kRows + 15) / 16 * 16;  // N of S^T (a multiple of 16)
  static constexpr int kON = 16 * NG;                 // rows of O^T's N, per term: [group][map][8 rows]
  static constexpr int kColS = 0;                     // S^T, two buffers of [map][kSN]
  static constexpr int kColO = 4 * kSN;               // O^T, [slab][term] x kON
  static constexpr int kColK = kColO + kSlabs * kTerms * kON;  // fp16 K (A of S^T), two buffers of D / 2 columns
  static constexpr int kCols = kColK + (CODES ? 0 : D);
  static constexpr int kTmemCols = kCols <= 256 ? 256 : 512;
  static constexpr uint32_t kIdescS = CODES ? idesc_e4m3(128, kSN) : idesc_f16(128, kSN, false, false);
  static constexpr uint32_t kIdescO =
      CODES ? idesc_e4m3(128, kTerms * kON) | (1u << 10) /* B: e5m2 */ | (3u << 15) : idesc_f16(128, kON, true, true);
  // A running maximum is raised past a gap of kRaise (log2); weights are
  // 2^(x - m + kBias), at most 2^15. (A gap of 1 raises in most of the first blocks: 830 cycles a block for the
  // maxima, 300 with 3.)
  static constexpr float kRaise = CODES ? 3.f : 4.f;
  static constexpr float kBias = 15.f - kRaise;
  // The row state holds the threshold m + kRaise. Before the first visible key m is a
  // number below every score, so that nothing need be told apart: the exponential
  // of a masked score (-inf) against it is zero.
  static constexpr float kNone = -3e38f;
  // A piece's fixed cost in 16-key tiles (balanced split; 24 / 40 / 64: e4m3, 32
  // ragged sequences of up to 8192 keys, D = 256 72.3 / 63.2 / 64.9 us, 24 of 8 heads, D =
  // 128 76.3 / 64.0 / 61.5; int8, 24 / 32 / 40: 78.7 / 77.0 / 78.9, 79.9 / 73.1 / 72.2).
  static constexpr int kUnitCost = CODES ? 40 : 32;

  static constexpr int kOffV = NBK * kBlkBytes;
  static constexpr int kOffV16 = kOffV + NBV * kBlkBytes;
  static constexpr int kOffQ = kOffV16 + kV16Bytes;
  static constexpr int kOffPt = kOffQ + kQSlabs * kQSlab;
  static constexpr int kOffRed = kOffPt + kPtBytes;          // float [NG][4 warps][16]
  static constexpr int kOffRow = kOffRed + NG * 4 * 16 * 4;  // row state, [NG][map][8]: score factor,
  static constexpr int kFs = 0, kTh = kON, kAl = 2 * kON, kL = 3 * kON;  // threshold, rescale, sum;
  static constexpr int kLo = 4 * kON, kHi = kLo + kRows, kRow = kHi + kRows;  // [NG][8]: visible range,
  static constexpr int kLam = kRow + kRows, kFlag = kLam + kRows;  // output row (of Hq a token), lambda; a flag
  static constexpr int kOdd = kFlag + NG;  // a NaN code in V of a key that only some rows see
  // Cluster merge: each CTA stages its partial (m, l) here, [map][row], and its
  // partial O rows [map][row][D] at offset 0, over the K ring, idle by then.
  static constexpr int kOffStage = (kOffRow + (kOdd + 1) * 4 + 15) / 16 * 16;
  static constexpr int kOffBars = kOffStage + 2 * kRows * 8;
  // barriers: fullK, emptyK [NBK], fullV, emptyV [NBV], then these (kBarS2: S^T
  // read, CODES; else K widened)
  static constexpr int kBarSFull = 0, kBarS2 = 2, kBarPFull = 4, kBarPvDone = 5, kBarQFull = 6, kBarFinal = 7;
  static constexpr int kOffTmem = kOffBars + (2 * NBK + 2 * NBV + 8) * 8;
  static constexpr int kOffPre = kOffTmem + 16;
  static constexpr int kSmemBytes = kOffPre + (kMaxAutoB + 1) * 4 + 1024;  // + alignment slack
  static_assert(KV == kKvFp8 || KV == kKvInt8, "one-byte codes");
  static_assert(kOffQ % 1024 == 0 && kOffPt % 1024 == 0 && kQTerm % 1024 == 0 && kPtAtom % 1024 == 0,
                "tensor-core operands start on swizzle atoms");
  static_assert(kOffRow % 16 == 0, "row state read as float4");
  static_assert(kCols <= kTmemCols, "tensor-memory columns");
  static_assert(kSmemBytes <= 227 * 1024, "one CTA per SM");
  static_assert(2 * kRows * D * 4 <= kOffV, "the staged rows fit over the K ring");
};

// Four fp16 weights in [0, 2^15] (two pairs) to three words of e5m2 codes, w = t1 +
// t2 2^-4 + t3 2^-8 exactly. An e5m2 code is the upper byte of an fp16 value, the
// nearest one that of the bits plus half of the lower byte's range. What it leaves of a
// weight in [2^e, 2^(e+1)), a multiple of 2^(e-10), is at most 2^(e-3); 2^4 times that
// is rounded in turn and leaves at most 8 multiples of 2^(e-6), which 2^4 times are an
// e5m2 value. (Below 2^-14 the steps are those of e = -14.)
__device__ __forceinline__ void split_weight(uint32_t a, uint32_t b, uint32_t (&t)[3]) {
  const __half2 s16 = __float2half2_rn(16.f);
  auto near = [](uint32_t x) { return (x + 0x00800080u) & 0xff00ff00u; };
  auto codes = [](uint32_t x, uint32_t y) { return prmt(x, y, 0x7531u); };
  auto rest = [&](uint32_t x, uint32_t lead) {
    const __half2 r =
        __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&lead)), s16);
    return *reinterpret_cast<const uint32_t*>(&r);
  };
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint32_t na = near(a), nb = near(b);
    t[m] = codes(na, nb);
    a = rest(a, na), b = rest(b, nb);
  }
  t[2] = codes(a, b);
}

// 16 floats of shared memory (16-byte aligned).
__device__ __forceinline__ void load16(const float* src, float (&v)[16]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 f = reinterpret_cast<const float4*>(src)[k];
    v[4 * k] = f.x; v[4 * k + 1] = f.y; v[4 * k + 2] = f.z; v[4 * k + 3] = f.w;
  }
}

// One operand's producer warp: every block of the CTA's pieces, a box per lane
// (one lane that issues them all, as decode_diff.cuh's, took 54.8 us instead of 43.2
// at B = 8, L = 8192, qlen = 3, e4m3, 53.4 instead of 48.1 at int8); each lane
// translates its own of the next 32 tiles.
template <class T, int NB>
__device__ __forceinline__ void diff_tc_producer(const DecodeParams& p, const int* s_pre, WorkIter& it, Piece& pc,
                                                 const CUtensorMap* tm, uint32_t ring, uint32_t full, uint32_t empty) {
  const int lane = threadIdx.x & 31;
  constexpr int kBoxes = T::CODES ? T::kSlabs : 1;  // boxes of a tile
  const uint64_t pol = l2_policy_evict_first();
  uint32_t b = 0, posted = 0;  // blocks walked; blocks whose loads were issued
  bool ok = true;
  while (work_next(p, s_pre, it, pc)) {
    if (pc.ntiles == 0) continue;
    const int32_t* row = p.block_table + static_cast<long long>(pc.b) * p.max_blocks;
    auto load_group = [&](int t) -> int {
      return t + lane < pc.ntiles ? __ldg(row + (pc.first_tile + t + lane) / p.tiles_per_block) : 0;
    };
    int cur = load_group(0);
    for (int t = 0; t < pc.ntiles; t += 32) {
      const int nxt = t + 32 < pc.ntiles ? load_group(t + 32) : 0;
      if (cur < 0 || cur >= p.num_blocks) {
        raise_error(p.error_flag, kErrBlockId);
        cur = 0;
      }
      const int row0 = cur * p.block_size + ((pc.first_tile + t + lane) % p.tiles_per_block) * kTileKeys;
      for (int t0 = t; t0 < min(t + 32, pc.ntiles); t0 += T::kBlkTiles, ++b) {
        const uint32_t st = b % NB, fb = full + 8 * st;
        const int n = min(T::kBlkTiles, pc.ntiles - t0);
        if (lane == 0) {
          if (ok && b >= NB) ok = mbar_wait(empty + 8 * st, (b / NB - 1) & 1, p.timeout_ns);
          if (ok && p.inject == 1) ok = false;  // injected fault: the rings stay empty
          if (ok) {
            mbar_arrive_expect_tx(fb, n * T::kTileBytes);
            posted = b + 1;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        const uint32_t dst = ring + st * T::kBlkBytes;
        const int j = min(lane / kBoxes, T::kBlkTiles - 1), sl = lane % kBoxes;
        const int z = __shfl_sync(0xffffffffu, row0, t0 - t + j);
        if (ok && lane < kBoxes * n) {
          if constexpr (T::CODES)
            tma_load_3d(dst + sl * T::kSlabBlk + j * (kTileKeys * 128), tm, fb, sl * 128, pc.kh, z, pol);
          else
            tma_load_4d(dst + j * T::kTileBytes, tm, fb, 0, z, pc.kh, 0, pol);
        }
      }
      cur = nxt;
    }
  }
  if (lane == 0) {
    if (!ok) raise_error(p.error_flag, kErrTimeout);
    // every issued load lands before the CTA's shared memory is released
    for (uint32_t k = posted > NB ? posted - NB : 0; k < posted; ++k)
      if (!mbar_wait(full + 8 * (k % NB), (k / NB) & 1, kDrainLimitNs)) break;
  }
  __syncwarp();
}

// The softmax warps; int8: they also widen the codes, chunk c of a key row goes to
// group c % NG (K) and (kChunks + c) % NG (V).
template <class T>
__device__ __forceinline__ void diff_tc_softmax(const DiffParams& dp, const int* s_pre, WorkIter& it, Piece& pc,
                                                uint8_t* smem, uint32_t sbase, uint32_t tmem) {
  const DecodeParams& p = dp.d;
  constexpr int D = T::D, NBK = T::NBK, NBV = T::NBV, S = T::kSlabs, NG = T::NG, NCH = T::kChunks, PER = (NCH + NG - 1) / NG;
  constexpr int NST = T::kSoftThreads, NTM = T::kTerms;
  constexpr bool CODES = T::CODES;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = warp >> 2;      // row group
  const int key = tid & 127;    // TMEM lane of this thread
  const int swz = key & 7;      // 128-byte swizzle of this key's rows
  const int v_first = ((g - NCH) % NG + NG) % NG;
  const int bid = 1 + g;        // the group's named barrier
  float* rf = reinterpret_cast<float*>(smem + T::kOffRow);
  int* ri = reinterpret_cast<int*>(smem + T::kOffRow);
  float* red = reinterpret_cast<float*>(smem + T::kOffRed) + 64 * g;  // [4 warps][16]
  float *fs_row = rf + T::kFs + 16 * g, *th_row = rf + T::kTh + 16 * g, *al_row = rf + T::kAl + 16 * g,
        *l_row = rf + T::kL + 16 * g;
  const int *lo_row = ri + T::kLo + 8 * g, *hi_row = ri + T::kHi + 8 * g;
  const uint32_t fullk0 = sbase + T::kOffBars, emptyk0 = fullk0 + 8 * NBK;
  const uint32_t fullv0 = emptyk0 + 8 * NBK, emptyv0 = fullv0 + 8 * NBV, bx = emptyv0 + 8 * NBV;
  auto bar = [&](int i) -> uint32_t { return bx + 8 * i; };
  const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);  // this warp's TMEM lanes
  const uint32_t qs = sbase + T::kOffQ, v16 = sbase + T::kOffV16;
  const uint32_t key_off = (key >> 4) * T::kTileBytes + (key & 15) * 128;  // of this key's row in a ring stage
  // this key's row of the first 32 bytes of P^T's N; 16 bytes c of N are half c % 2
  // of it in atom c / 2, the halves swapped in rows 4 to 7 (32-byte swizzle)
  const uint32_t pt = sbase + T::kOffPt + (key >> 3) * 256 + swz * 32;
  auto pt_at = [&](int c) { return pt + (c >> 1) * T::kPtAtom + (((c & 1) ^ (swz >> 2)) << 4); };
  uint32_t bq = 0;
  bool ok = true;

  // K of block b into its tensor-memory buffer (last read by S^T of block b - 2,
  // which this warp has waited for); the ring stage is released.
  auto widen_k = [&](uint32_t b) {
    const int st = b % NBK;
    if (ok) ok = mbar_wait(fullk0 + 8 * st, (b / NBK) & 1, p.timeout_ns);
    ok = __all_sync(0xffffffffu, ok);  // tcgen05.st is warp-collective
    if (ok) {
      const uint32_t src = sbase + st * T::kBlkBytes + key_off;
      const uint32_t dst = tl + T::kColK + (b & 1) * (D / 2);
      uint4 w[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = min(g + NG * k, NCH - 1);
        w[k] = ld_shared_v4(src + (c >> 3) * 2048 + (((c & 7) ^ swz) << 4));
      }
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = g + NG * k;
        if (c < NCH) {  // warp-uniform
          uint32_t h[8];
          widen_i8x16(w[k], h);
          tmem_st8u(dst + 8 * c, h);
        }
      }
      tmem_wait_st();
    }
    tc_fence_before();
    __syncwarp();
    if (ok && lane == 0) {
      mbar_arrive(emptyk0 + 8 * st);
      mbar_arrive(bar(T::kBarS2 + (b & 1)));
    }
  };
  // V of block b into the fp16 buffer (last read by P.V of block b - 1, which has
  // completed), zeros for keys from lim on; the ring stage is released.
  auto widen_v = [&](uint32_t b, int lim) {
    const int st = b % NBV;
    if (ok) ok = mbar_wait(fullv0 + 8 * st, (b / NBV) & 1, p.timeout_ns);
    if (ok) {
      const uint32_t src = sbase + T::kOffV + st * T::kBlkBytes + key_off;
      uint4 w[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = min(v_first + NG * k, NCH - 1);
        w[k] = ld_shared_v4(src + (c >> 3) * 2048 + (((c & 7) ^ swz) << 4));
        if (key >= lim) w[k] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int c = v_first + NG * k;
        if (c < NCH) {
          uint32_t h[8];
          widen_i8x16(w[k], h);
          const uint32_t row = v16 + (c >> 2) * T::kV16Slab + key * 128;
          st_shared_v4(row + (((2 * (c & 3)) ^ swz) << 4), h[0], h[1], h[2], h[3]);
          st_shared_v4(row + (((2 * (c & 3) + 1) ^ swz) << 4), h[4], h[5], h[6], h[7]);
        }
      }
    }
    __syncwarp();
    if (ok && lane == 0) mbar_arrive(emptyv0 + 8 * st);
  };
  // A piece's q (B of S^T: K-major, 128-byte swizzle), score factors and visible
  // ranges. Item: row item / 8, dims [(item % 8) D / 8, + D / 8); the four items of
  // a half row scale it by the power of two that brings its largest |q| into
  // [2^14, 2^15) for fp16 operands (exact for an fp16 q; a bfloat16 q keeps its 8
  // bits), into [2^7, 2^8) for e4m3 terms (exact but where |q| is below 2^-6 of
  // the largest, fp16, 2^-9, bfloat16: there off by 2^-17 of the largest at most).
  auto q_setup = [&](const Piece& pq) {
    if (CODES && tid == 0) ri[T::kOdd] = 0;
    for (int item = tid; item < T::kRows * 8; item += NST) {
      const int r = item >> 3, part = item & 7;
      constexpr int NW = D / 64;  // 8-dim pieces per item
      const int row = (pq.q0 + r / p.G) * p.Hq + pq.kh * p.G + r % p.G;
      const __half* qrow = r < pq.R ? p.q + static_cast<long long>(row) * D : nullptr;
      uint4 qv[NW];
      float mx = 0.f;
      auto to_f = [&](uint32_t w) { return p.out_bf16 ? pair_to_float2<true>(w) : pair_to_float2<false>(w); };
#pragma unroll
      for (int c = 0; c < NW; ++c) {
        qv[c] = qrow ? __ldg(reinterpret_cast<const uint4*>(qrow + part * (D / 8) + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {qv[c].x, qv[c].y, qv[c].z, qv[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = to_f(w[k]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      constexpr int kTop = CODES ? 134 : 141;
      const int e = mx > 0.f ? max(-126, min(126, kTop - static_cast<int>((__float_as_uint(mx) >> 23) & 255u))) : 0;
      const float up = pow2f(e);
      uint32_t h[NW][4];
#pragma unroll
      for (int c = 0; c < NW; ++c) {
        const uint32_t w[4] = {qv[c].x, qv[c].y, qv[c].z, qv[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = to_f(w[k]);
          h[c][k] = pack_half2(f.x * up, f.y * up);
        }
      }
      if constexpr (CODES) {
#pragma unroll
        for (int c = 0; c < NW; c += 2) {
          const int d0 = part * (D / 8) + 8 * c;
          uint32_t tw[3][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t lo[3], hi[3];
            split3_e4m3(h[c + (k >> 1)][2 * (k & 1)], lo[0], lo[1], lo[2]);
            split3_e4m3(h[c + (k >> 1)][2 * (k & 1) + 1], hi[0], hi[1], hi[2]);
#pragma unroll
            for (int m = 0; m < 3; ++m) tw[m][k] = lo[m] | (hi[m] << 16);
          }
          const uint32_t at = qs + (d0 >> 7) * T::kQSlab + r * 128 + ((((d0 & 127) >> 4) ^ (r & 7)) << 4);
#pragma unroll
          for (int m = 0; m < 3; ++m) st_shared_v4(at + m * T::kQTerm, tw[m][0], tw[m][1], tw[m][2], tw[m][3]);
          if constexpr (T::kQTerms == 4) st_shared_v4(at + 3 * T::kQTerm, 0u, 0u, 0u, 0u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < NW; ++c) {
          const int d0 = part * (D / 8) + 8 * c;
          st_shared_v4(qs + (d0 >> 6) * T::kQSlab + r * 128 + ((((d0 & 63) >> 3) ^ (r & 7)) << 4), h[c][0], h[c][1],
                       h[c][2], h[c][3]);
        }
      }
      if ((part & 3) == 0) {
        const int at = 16 * (r >> 3) + 8 * (part >> 2) + (r & 7);
        // (an infinity has no e4m3 terms, and no key's score with it is a number)
        rf[T::kFs + at] = mx == INFINITY ? NAN : r < pq.R ? p.sl2 * pow2f(-e) : 0.f;
        rf[T::kTh + at] = T::kNone;
      }
      if (part == 0) {
        const int hi = r < pq.R ? pq.L - pq.qlen + r / p.G : -1;
        ri[T::kHi + r] = hi;
        ri[T::kLo + r] = p.window > 0 ? max(0, hi - p.window + 1) : 0;
        ri[T::kRow + r] = row;
        rf[T::kLam + r] = r < pq.R ? __ldg(dp.lambda + row % p.Hq) : 0.f;
      }
    }
    fence_proxy_async_smem();
  };

  while (tc_next_piece<T>(p, s_pre, it, pc)) {
    const int nblk = (pc.ntiles + T::kBlkTiles - 1) / T::kBlkTiles;
    q_setup(pc);
    named_bar_sync(T::kBarAll, NST);
    if (tid == 0) mbar_arrive(bar(T::kBarQFull));
    auto first_key = [&] { return p.window > 0 ? pc.tile_hi_all - p.window + 1 : 0; };  // that a row sees
    float lp[16];  // this key lane's share of each row's weight sum ([map][row])
#pragma unroll
    for (int r = 0; r < 16; ++r) lp[r] = 0.f;
    if constexpr (!CODES) widen_k(bq);

    for (int i = 0; i < nblk; ++i) {
      const uint32_t b = bq + i;
      const int sb = b & 1;
      const int key0 = (pc.first_tile + T::kBlkTiles * i) * kTileKeys;
      const int nvalid = min(128, kTileKeys * (pc.ntiles - T::kBlkTiles * i));  // keys loaded
      if constexpr (!CODES) {  // the next block's K, while S^T of this one is computed
        if (i + 1 < nblk) widen_k(b + 1);
      }
      // ---- this key's scores for the group's 8 rows of both maps
      float x[16], th[16];
      if (ok) ok = mbar_wait(bar(T::kBarSFull + sb), (b >> 1) & 1, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);  // tcgen05.ld is warp-collective
      tc_fence_after();
      if (ok) {
        float y[T::kStack][2][8];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int k = 0; k < T::kStack; ++k)
            tmem_ld8(tl + T::kColS + (2 * sb + m) * T::kSN + k * T::kRows + 8 * g, y[k][m]);
        tmem_wait_ld();
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          x[r] = y[0][r >> 3][r & 7];
          if constexpr (T::kStack == 2) x[r] += y[1][r >> 3][r & 7];
        }
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = 0.f;
      }
      if constexpr (CODES) {
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(T::kBarS2 + sb));
      }
      load16(fs_row, th);
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] *= th[r];
      const bool edge = nvalid < 128 || key0 < pc.tile_lo_all || key0 + 127 > pc.tile_hi_all;
      if (edge) {
        const int j = key0 + key;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (!(key < nvalid && j >= lo_row[r] && j <= hi_row[r])) x[r] = x[8 + r] = -INFINITY;
      }
      // ---- running maxima, raised where a block's maximum passes one by 2^kRaise
      load16(th_row, th);
      bool upd = false;
#pragma unroll
      for (int r = 0; r < 16; ++r) upd |= x[r] > th[r];
      bool rescale = false;
      if (bar_red_or(bid, 128, upd)) {
#pragma unroll
        for (int r = 0; r < 16; ++r) th[r] = x[r];
        const float m = warp_transpose_reduce<true, 16>(th, lane);
        if (lane < 16) red[(warp & 3) * 16 + lane] = m;
        named_bar_sync(bid, 128);
        if ((warp & 3) == 0) {
          const int l16 = lane & 15;
          const float mx = fmaxf(fmaxf(red[l16], red[16 + l16]), fmaxf(red[32 + l16], red[48 + l16]));
          const float th0 = th_row[l16];
          const bool up = mx > th0;
          const float al = up ? ex2(th0 - T::kRaise - mx) : 1.f;  // (0 from kNone)
          __syncwarp();
          if (lane < 16) {
            if (up) th_row[lane] = mx + T::kRaise;
            al_row[lane] = al;
          }
          const bool any = __any_sync(0xffffffffu, up);
          if (lane == 0) ri[T::kFlag + g] = any ? 1 : 0;
        }
        named_bar_sync(bid, 128);
        load16(th_row, th);
        rescale = ri[T::kFlag + g] != 0;
      }
      // ---- weights 2^(x - m + kBias) rounded to fp16; the sums add the rounded ones
      uint32_t pw[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        constexpr float kUp = T::kRaise + T::kBias;  // 15
        const float a = ex2(x[2 * k] - th[2 * k] + kUp), c = ex2(x[2 * k + 1] - th[2 * k + 1] + kUp);
        pw[k] = pack_half2(a, c);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&pw[k]));
        x[2 * k] = f.x;
        x[2 * k + 1] = f.y;
      }
      if (rescale) {
        load16(al_row, th);
#pragma unroll
        for (int r = 0; r < 16; ++r) lp[r] = lp[r] * th[r] + x[r];
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) lp[r] += x[r];
      }
      // ---- the P.V operands are free once the previous block's product is done
      if (ok && b >= 1) ok = mbar_wait(bar(T::kBarPvDone), (b - 1) & 1, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (rescale && i > 0 && ok) {
#pragma unroll 1
        for (int c = 0; c < S * NTM; ++c) {
          float o[16];
          tmem_ld16(tl + T::kColO + T::kON * c + 16 * g, o);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < 16; ++r) o[r] *= th[r];
          tmem_st16(tl + T::kColO + T::kON * c + 16 * g, o);
        }
        tmem_wait_st();
      }
      // ---- P^T: N runs over [group][map][8 rows] fp16, or [term][group][map][8 rows]
      // codes
      const int lim = min(nvalid, pc.L - key0);  // keys beyond are stale or not loaded
      if constexpr (CODES) {
        uint32_t tw[4][3];
#pragma unroll
        for (int k = 0; k < 4; ++k) split_weight(pw[2 * k], pw[2 * k + 1], tw[k]);
#pragma unroll
        for (int m = 0; m < 3; ++m) st_shared_v4(pt_at(m * NG + g), tw[0][m], tw[1][m], tw[2][m], tw[3][m]);
        if (g == 0 && edge) {
          const int st = b % NBV;
          const uint32_t vblk = sbase + T::kOffV + st * T::kBlkBytes;
          if (ok) ok = mbar_wait(fullv0 + 8 * st, (b / NBV) & 1, p.timeout_ns);
          if (ok && (key >= lim || key0 + key < first_key())) {  // V rows that no query row sees
#pragma unroll
            for (int c = 0; c < 8 * S; ++c)
              st_shared_v4(vblk + key * 128 + (c >> 3) * T::kSlabBlk + 16 * (c & 7), 0u, 0u, 0u, 0u);
          }
          // NaN codes of keys that only some of the rows see (several query tokens) become
          // zeros, lest they meet the others' zero weights; the piece's end puts them back
          const int lo0 = max(0, first_key() - key0), lo1 = min(lim, pc.tile_lo_all - key0);
          const int hi0 = max(max(lo0, lo1), pc.tile_hi_all + 1 - key0);
          const int nlo = max(0, lo1 - lo0), some = nlo + max(0, lim - hi0);
          for (int item = key; ok && item < some * 8 * S; item += 128) {
            const int r = item / (8 * S), c = item % (8 * S);
            const uint32_t at = vblk + (r < nlo ? lo0 + r : hi0 + r - nlo) * 128 + (c >> 3) * T::kSlabBlk + 16 * (c & 7);
            const uint4 v = ld_shared_v4(at);
            uint32_t w[4] = {v.x, v.y, v.z, v.w}, odd = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t nan = (((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
              w[k] &= ~(nan * 0xffu);
              odd |= nan;
            }
            if (odd) {
              st_shared_v4(at, w[0], w[1], w[2], w[3]);
              ri[T::kOdd] = 1;
            }
          }
        }
      } else {
        st_shared_v4(pt_at(2 * g), pw[0], pw[1], pw[2], pw[3]);
        st_shared_v4(pt_at(2 * g + 1), pw[4], pw[5], pw[6], pw[7]);
        widen_v(b, lim);
      }
      ok = __all_sync(0xffffffffu, ok);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar(T::kBarPFull));
    }
    bq += nblk;

    // does the piece hold keys that only some rows see? (the same for all threads; group
    // 0's note of a NaN among them reaches the others, who wait for its weights anyway)
    auto some_rows = [&] {
      return CODES && pc.qlen > 1 && (pc.first_tile * kTileKeys < pc.tile_lo_all ||
                                      min(pc.L, (pc.first_tile + pc.ntiles) * kTileKeys) - 1 > pc.tile_hi_all);
    };
    if (some_rows()) named_bar_sync(T::kBarAll, NST);
    float w[S];  // the norm's weights of this thread's dims, read before the waits
#pragma unroll
    for (int h = 0; h < S; ++h)
      w[h] = dp.norm_weight != nullptr && pc.npieces == 1 ? norm_weight_at(dp, 128 * h + key) : 0.f;
    // ---- the piece's end: O^T (this thread: dims key, key + 128) of the group's
    // rows of both maps, and the row sums
    if (ok) ok = mbar_wait(bar(T::kBarPvDone), (bq - 1) & 1, p.timeout_ns);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    float o[S][16];
#pragma unroll
    for (int h = 0; h < S; ++h) {
      if (ok) {
        const uint32_t at = tl + T::kColO + T::kON * NTM * h + 16 * g;
        tmem_ld16(at, o[h]);
        if constexpr (CODES) {  // the terms' scales
          float y[16];
          tmem_ld16(at + T::kON, y);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < 16; ++r) o[h][r] = fmaf(y[r], 0x1p-4f, o[h][r]);
          tmem_ld16(at + 2 * T::kON, y);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < 16; ++r) o[h][r] = fmaf(y[r], 0x1p-8f, o[h][r]);
        }
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) o[h][r] = 0.f;
      }
    }
    tc_fence_before();
    {
      const float sum = warp_transpose_reduce<false, 16>(lp, lane);
      if (lane < 16) red[(warp & 3) * 16 + lane] = sum;
    }
    named_bar_sync(bid, 128);
    if ((warp & 3) == 0 && lane < 16)
      l_row[lane] = (red[lane] + red[16 + lane]) + (red[32 + lane] + red[48 + lane]);
    named_bar_sync(bid, 128);
    if (pc.npieces == 1) {
      float ss[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float l1 = l_row[r], l2 = l_row[8 + r];
        const float lam = rf[T::kLam + 8 * g + r];
        const float i1 = l1 > 0.f ? p.out_scale / l1 : 0.f, i2 = l2 > 0.f ? p.out_scale / l2 * lam : 0.f;
        ss[r] = 0.f;
#pragma unroll
        for (int h = 0; h < S; ++h) {
          o[h][r] = map_out(l1, o[h][r]) * i1 - map_out(l2, o[h][8 + r]) * i2;
          ss[r] += o[h][r] * o[h][r];
        }
      }
      if (dp.norm_weight != nullptr) {
        const float sum = warp_transpose_reduce<false, 8>(ss, lane);
        if (lane < 8) red[(warp & 3) * 16 + lane] = sum;
        named_bar_sync(bid, 128);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float tot = (red[r] + red[16 + r]) + (red[32 + r] + red[48 + r]);
          const float f = norm_factor<D>(dp, tot);
#pragma unroll
          for (int h = 0; h < S; ++h) o[h][r] *= f * w[h];
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        if (8 * g + r >= pc.R) break;
        uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) + static_cast<long long>(ri[T::kRow + 8 * g + r]) * D;
#pragma unroll
        for (int h = 0; h < S; ++h)
          dst[128 * h + key] = static_cast<uint16_t>(pack_out(p.out_bf16 != 0, o[h][r], 0.f) & 0xffffu);
      }
    } else {
      // the partial rows: staged for a cluster merge, else the piece's slot
      float* part = p.cluster > 1 ? reinterpret_cast<float*>(smem)
                                  : p.ws_o + static_cast<long long>(pc.slot) * p.rows_padded * D;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (8 * g + r >= pc.R) break;
          float* dst = part + (m * T::kRows + 8 * g + r) * D + key;
#pragma unroll
          for (int h = 0; h < S; ++h) {
            if (p.cluster > 1) dst[128 * h] = o[h][8 * m + r];
            else __stcg(dst + 128 * h, o[h][8 * m + r]);
          }
        }
      }
      if (key < 16 && 8 * g + (key & 7) < pc.R) {
        const int row = (key >> 3) * T::kRows + 8 * g + (key & 7);
        const float th = th_row[key], l = l_row[key];  // (l = 0: no key was visible)
        const float2 ml = make_float2(l == 0.f ? -INFINITY : th - (T::kRaise + T::kBias), l);
        if (p.cluster > 1)
          reinterpret_cast<float2*>(smem + T::kOffStage)[row] = ml;
        else
          __stcg(reinterpret_cast<float2*>(p.ws_ml) + static_cast<long long>(pc.slot) * p.rows_padded + row, ml);
      }
    }
    if constexpr (CODES) {
      if (some_rows() && ri[T::kOdd] != 0) {
        // the outputs of rows that see a NaN are NaN (under a norm the whole row): each
        // thread writes over what it has written
        const int key_hi = min(pc.L, (pc.first_tile + pc.ntiles) * kTileKeys);
        float* part = p.cluster > 1 ? reinterpret_cast<float*>(smem)
                                    : p.ws_o + static_cast<long long>(pc.slot) * p.rows_padded * D;
#pragma unroll 1
        for (int j = max(first_key(), pc.first_tile * kTileKeys); j < key_hi; ++j) {
          if (j >= pc.tile_lo_all && j <= pc.tile_hi_all) {  // seen by all: in the products
            j = pc.tile_hi_all;
            continue;
          }
          const int blk = __ldg(p.block_table + static_cast<long long>(pc.b) * p.max_blocks + j / p.block_size);
          const long long slot = static_cast<long long>(blk >= 0 && blk < p.num_blocks ? blk : 0) * p.block_size + j % p.block_size;
          const uint8_t* v = static_cast<const uint8_t*>(dp.v_cache) + (slot * p.Hkv + pc.kh) * D;
          bool any = false;
#pragma unroll 1
          for (int d = 0; d < D && dp.norm_weight != nullptr; ++d) any |= (v[d] & 0x7fu) == 0x7fu;
#pragma unroll 1
          for (int i = 0; i < 8 * S; ++i) {
            const int r = i & 7, d = 128 * (i >> 3) + key;
            const bool nan = (v[d] & 0x7fu) == 0x7fu;
            if (8 * g + r >= pc.R || j < lo_row[r] || j > hi_row[r]) continue;
            if (pc.npieces == 1) {
              if ((nan || any) && (l_row[r] > 0.f || l_row[8 + r] > 0.f))
                reinterpret_cast<uint16_t*>(p.out)[static_cast<long long>(ri[T::kRow + 8 * g + r]) * D + d] = 0x7fffu;
            } else if (nan) {
              part[(8 * g + r) * D + d] = NAN;
              part[(T::kRows + 8 * g + r) * D + d] = NAN;
            }
          }
        }
      }
    }
    named_bar_sync(T::kBarAll, NST);  // the row state and red[] are rewritten by the next piece
  }
  if (!ok && lane == 0) raise_error(p.error_flag, kErrTimeout);
}

// Merge of a fixed split whose pieces are the CTAs of one cluster: a warp takes a
// row (both maps), CTA s the rows r with r % S == s, reads the S partials through
// distributed shared memory and finishes the row as diff_combine_kernel does. A
// CTA without a piece staged l = 0; a unit of one piece was finished by it.
template <class T>
__device__ __forceinline__ void diff_tc_merge(const DiffParams& dp, uint32_t sbase) {
  const DecodeParams& p = dp.d;
  constexpr int D = T::D, V4 = D / 128;
  const int S = p.cluster, rank = static_cast<int>(cluster_rank()), u = blockIdx.x / S;
  const int b = u / p.hgn, kh = u % p.hgn;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // what is no partial is read before the cluster's barrier
  int L, t0, n, q0, qn;
  seq_span(p, b, false, L, t0, n, q0, qn);
  const int R = n > (n + S - 1) / S ? p.G * qn : 0;  // (one piece or none: finished)
  float4 wt[V4];
  if (dp.norm_weight != nullptr) {
#pragma unroll
    for (int v = 0; v < V4; ++v) {
      const int d = 4 * (32 * v + lane);
      wt[v] = make_float4(norm_weight_at(dp, d), norm_weight_at(dp, d + 1), norm_weight_at(dp, d + 2),
                          norm_weight_at(dp, d + 3));
    }
  }
  int r = rank + S * warp;
  float lam = r < R ? __ldg(dp.lambda + kh * p.G + r % p.G) : 0.f;
  cluster_sync();  // every CTA of the cluster has staged its partial
  for (; r < R; r += S * (T::kThreads / 32)) {
    float4 y[V4];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int row = m * T::kRows + r;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < S) ml = ld_peer_f2(peer_smem(sbase + T::kOffStage + 8 * row, lane));
      float M = ml.x;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float w = ml.y == 0.f ? 0.f : ex2(ml.x - M);
      float l = w * ml.y;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const uint32_t live = __ballot_sync(0xffffffffu, ml.y != 0.f);
      float4 acc[V4];
#pragma unroll
      for (int v = 0; v < V4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int s = 0; s < S; ++s) {
        const float ws = __shfl_sync(0xffffffffu, w, s);
        if (!(live >> s & 1)) continue;
        const uint32_t at = peer_smem(sbase + row * D * 4, s);
#pragma unroll
        for (int v = 0; v < V4; ++v) {
          const float4 a = ld_peer_f4(at + 16 * (32 * v + lane));
          acc[v].x += ws * a.x; acc[v].y += ws * a.y; acc[v].z += ws * a.z; acc[v].w += ws * a.w;
        }
      }
      float inv = l > 0.f ? p.out_scale / l : 0.f;
      if (m == 1) inv *= -lam;
#pragma unroll
      for (int v = 0; v < V4; ++v) {
        acc[v] = make_float4(map_out(l, acc[v].x), map_out(l, acc[v].y), map_out(l, acc[v].z), map_out(l, acc[v].w));
        if (m == 0) y[v] = make_float4(acc[v].x * inv, acc[v].y * inv, acc[v].z * inv, acc[v].w * inv);
        else y[v] = make_float4(fmaf(acc[v].x, inv, y[v].x), fmaf(acc[v].y, inv, y[v].y), fmaf(acc[v].z, inv, y[v].z),
                                fmaf(acc[v].w, inv, y[v].w));
      }
    }
    if (dp.norm_weight != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V4; ++v) ss += y[v].x * y[v].x + y[v].y * y[v].y + y[v].z * y[v].z + y[v].w * y[v].w;
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float f = norm_factor<D>(dp, ss);
      auto normed = [&](float x, float w) { return x * (f * w); };
#pragma unroll
      for (int v = 0; v < V4; ++v)
        y[v] = make_float4(normed(y[v].x, wt[v].x), normed(y[v].y, wt[v].y), normed(y[v].z, wt[v].z),
                           normed(y[v].w, wt[v].w));
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(p.out) +
                    (static_cast<long long>(q0 + r / p.G) * p.Hq + kh * p.G + r % p.G) * D;
    const bool bf = p.out_bf16 != 0;
#pragma unroll
    for (int v = 0; v < V4; ++v)
      *reinterpret_cast<uint2*>(dst + 4 * (32 * v + lane)) =
          make_uint2(pack_out(bf, y[v].x, y[v].y), pack_out(bf, y[v].z, y[v].w));
    if (r + S * (T::kThreads / 32) < R) lam = __ldg(dp.lambda + kh * p.G + (r + S * (T::kThreads / 32)) % p.G);
  }
}

template <class T>
__global__ void __launch_bounds__(T::kThreads, 1)
    decode_diff_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                          const DiffParams dp) {
  const DecodeParams& p = dp.d;
  constexpr int D = T::D, NBK = T::NBK, NBV = T::NBV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t fullk0 = sbase + T::kOffBars, emptyk0 = fullk0 + 8 * NBK;
  const uint32_t fullv0 = emptyk0 + 8 * NBK, emptyv0 = fullv0 + 8 * NBV, bx = emptyv0 + 8 * NBV;
  auto bar = [&](int i) -> uint32_t { return bx + 8 * i; };
  int* s_pre = reinterpret_cast<int*>(smem + T::kOffPre);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + T::kOffTmem);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    constexpr int kRelease = T::CODES ? 1 : 4 * T::NG;  // the product's commit, or the widening warps
    for (int s = 0; s < NBK; ++s) {
      mbar_init(fullk0 + 8 * s, 1);
      mbar_init(emptyk0 + 8 * s, kRelease);
    }
    for (int s = 0; s < NBV; ++s) {
      mbar_init(fullv0 + 8 * s, 1);
      mbar_init(emptyv0 + 8 * s, kRelease);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(T::kBarSFull + s), 1);
      mbar_init(bar(T::kBarS2 + s), 4 * T::NG);
    }
    mbar_init(bar(T::kBarPFull), 4 * T::NG);
    mbar_init(bar(T::kBarPvDone), 1);
    mbar_init(bar(T::kBarQFull), 1);
    mbar_init(bar(T::kBarFinal), 1);
    fence_mbar_init();
  }
  if (warp == T::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), T::kTmemCols);
    tmem_relinquish();
  }
  if (warp == T::kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // a CTA of a cluster that gets no piece contributes nothing to the merge
  if (threadIdx.x < 2 * T::kRows)
    reinterpret_cast<float2*>(smem + T::kOffStage)[threadIdx.x] = make_float2(-INFINITY, 0.f);
  // nothing above touches global memory (programmatic dependent launch)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.num_splits == 0 && warp == 0) balanced_prefix(p, s_pre, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  WorkIter it;
  work_init(p, s_pre, it);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Piece pc;

  if (warp == T::kProducerWarp) {
    diff_tc_producer<T, NBK>(p, s_pre, it, pc, &tm_k, sbase, fullk0, emptyk0);
  } else if (warp == T::kProducerWarp + 1) {
    diff_tc_producer<T, NBV>(p, s_pre, it, pc, &tm_v, sbase + T::kOffV, fullv0, emptyv0);
  } else if (warp == T::kMmaWarp) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      uint32_t bq = 0, pq = 0;
      bool any = false, ok = true;
      // passes over q's terms: two hold a bfloat16's 8 bits
      [[maybe_unused]] const int passes = T::kStack == 2 ? (p.out_bf16 ? 1 : 2) : p.out_bf16 ? 2 : 3;
      // operand descriptors; an offset is added to their address field, in 16 bytes
      const uint64_t qd = sdesc_sw128(sbase + T::kOffQ), pd = sdesc_sw32_mn(sbase + T::kOffPt, T::kPtAtom);
      [[maybe_unused]] const uint64_t vd16 = sdesc_sw128_mn16(sbase + T::kOffV16, T::kV16Slab);
      while (work_next(p, s_pre, it, pc)) {
        if (pc.ntiles == 0) continue;
        const int nblk = (pc.ntiles + T::kBlkTiles - 1) / T::kBlkTiles;
        if (ok) ok = mbar_wait(bar(T::kBarQFull), pq & 1, p.timeout_ns);
        ++pq;
        tc_fence_after();
        for (int i = 0; i <= nblk; ++i) {
          if (i < nblk) {  // S^T of block i, map by map
            const uint32_t b = bq + i;
            const int sb = b & 1, sk = b % NBK;
            const uint32_t s = tmem + T::kColS + 2 * T::kSN * sb;
            if constexpr (T::CODES) {
              if (ok) ok = mbar_wait(fullk0 + 8 * sk, (b / NBK) & 1, p.timeout_ns);
              if (ok && b >= 2) ok = mbar_wait(bar(T::kBarS2 + sb), ((b >> 1) - 1) & 1, p.timeout_ns);
            } else {
              if (ok) ok = mbar_wait(bar(T::kBarS2 + sb), (b >> 1) & 1, p.timeout_ns);
            }
            tc_fence_after();
            if (ok) {
              if constexpr (T::CODES) {
                constexpr int KSW = D / 64;  // 32-code k-steps of a map
                const uint64_t kd = sdesc_sw128(sbase + sk * T::kBlkBytes);
#pragma unroll 1
                for (int m = 0; m < passes; ++m) {
                  const uint64_t qm = qd + static_cast<uint32_t>(m * T::kStack * T::kQTerm >> 4);
#pragma unroll
                  for (int ks = 0; ks < 2 * KSW; ++ks)
                    mma_e4m3(s + T::kSN * (ks / KSW), kd + (((ks >> 2) * T::kSlabBlk + (ks & 3) * 32) >> 4),
                             qm + (((ks >> 2) * T::kQSlab + (ks & 3) * 32) >> 4), T::kIdescS,
                             ks % KSW != 0 ? 1u : static_cast<uint32_t>(m));
                }
              } else {
                constexpr int KSW = D / 32;
#pragma unroll
                for (int ks = 0; ks < 2 * KSW; ++ks)
                  mma_f16_ts(s + T::kSN * (ks / KSW), tmem + T::kColK + sb * (D / 2) + 8 * ks,
                             qd + (((ks >> 2) * T::kQSlab + (ks & 3) * 32) >> 4), T::kIdescS,
                             ks % KSW != 0 ? 1u : 0u);
              }
              mma_commit(bar(T::kBarSFull + sb));
              if constexpr (T::CODES) mma_commit(emptyk0 + 8 * sk);
              any = true;
            }
          }
          if (i >= 1) {  // O^T += V^T P^T of block i - 1 (V MN-major), both maps
            const uint32_t b = bq + i - 1;
            const int sv = b % NBV;
            if (T::CODES && ok) ok = mbar_wait(fullv0 + 8 * sv, (b / NBV) & 1, p.timeout_ns);
            if (ok) ok = mbar_wait(bar(T::kBarPFull), b & 1, p.timeout_ns);
            tc_fence_after();
            if (ok) {
#pragma unroll
              for (int h = 0; h < T::kSlabs; ++h) {
                const uint32_t o = tmem + T::kColO + T::kTerms * T::kON * h;
                if constexpr (T::CODES) {
                  const uint64_t vd = sdesc_sw128_mn(sbase + T::kOffV + sv * T::kBlkBytes + h * T::kSlabBlk);
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    mma_e4m3(o, vd + (kk * 4096 >> 4), pd + (kk * 1024 >> 4), T::kIdescO, (i > 1 || kk > 0) ? 1u : 0u);
                } else {
#pragma unroll
                  for (int kk = 0; kk < 8; ++kk)
                    mma_f16_ss(o, vd16 + ((2 * h * T::kV16Slab + kk * 2048) >> 4), pd + (kk * 512 >> 4), T::kIdescO,
                               (i > 1 || kk > 0) ? 1u : 0u);
                }
              }
              mma_commit(bar(T::kBarPvDone));
              if constexpr (T::CODES) mma_commit(emptyv0 + 8 * sv);
              any = true;
            }
          }
        }
        bq += nblk;
      }
      if (!ok) raise_error(p.error_flag, kErrTimeout);
      // every issued product completes before the tensor memory is freed
      if (any) {
        mma_commit(bar(T::kBarFinal));
        mbar_wait(bar(T::kBarFinal), 0, kDrainLimitNs);
      }
    }
    __syncwarp();
  } else {
    diff_tc_softmax<T>(dp, s_pre, it, pc, smem, sbase, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (p.cluster > 1) {
    diff_tc_merge<T>(dp, sbase);
    cluster_sync();  // no CTA leaves while a peer still reads its shared memory
  }
  if (warp == T::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, T::kTmemCols);
  }
}

template <class T>
cudaError_t launch_diff_tc(const CUtensorMap& tk, const CUtensorMap& tv, const DiffParams& p, int grid,
                           cudaStream_t stream) {
  static unsigned long long attr_ctx[64] = {};
  const cudaError_t e =
      once_per_context(attr_ctx, [] { return set_kernel_attributes(decode_diff_tc_kernel<T>, T::kSmemBytes); });
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_diff_tc_kernel<T>, grid, T::kThreads, T::kSmemBytes, stream, p.d.cluster, tk, tv, p);
}

template <class T>
bool diff_tc_shape_of(KernelShape* out) {
  out->threads = T::kThreads;
  out->smem_bytes = T::kSmemBytes;
  out->rows_padded = 2 * T::kRows;
  out->ctas_per_sm = 1;
  out->heads = 1;
  out->unit_cost = T::kUnitCost;
  out->fixed_pieces = 1;
  out->step_tiles = out->key_groups = T::kBlkTiles;
  out->whole_tile = T::CODES ? 0 : 1;
  static unsigned long long ctx_done[64] = {};
  static int cache[64][kMaxCluster + 1] = {};
  max_active_clusters(decode_diff_tc_kernel<T>, T::kThreads, T::kSmemBytes, ctx_done, cache, out->max_clusters);
  return true;
}

}  // namespace pd
