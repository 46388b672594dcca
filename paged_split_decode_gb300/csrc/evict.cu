// evict.cu -- eviction from the paged caches by the attention weight that keys have
// collected (evict_kv_cache): each KV head of a long sequence keeps its first keys, its
// last ones and the heaviest of the rest, moved together in order.
//
// Launch 1, select_kernel: a cluster of one to eight CTAs for each (sequence, KV head), as many
// as the GPU holds (B = 1, eight heads, 32768 keys: one CTA each 38 us of the call's 47).
// Each CTA has a run of the keys. The weights, as integers
// that order as the numbers do, are held in shared memory (beyond its size they are
// read again); the m-th largest is found digit by digit (8 bits, most significant first)
// from histograms, added up over the cluster; then each warp counts what its run of keys keeps, a scan over the
// warps gives its place, and it writes where every kept key comes from and goes to, in
// order. Of the keys equal to the m-th largest the lowest indices are kept. Bound by
// latency: four loads of a thread are in flight at a time. (Three digits of 11 bits instead of four of 8
// save a pass but read 16 K counts of the peers' shared memory: B = 1 19.2 -> 30.2 us, single CTAs the same.)
//
// Launch 2, move_kernel: rows move to slots at or below their own. In place that is safe
// without a second buffer when a CTA takes its rows in order: it loads a batch of rows, waits for
// all its threads, and stores them; the next batch's sources are at or behind its own first slot,
// and no earlier store reaches that far. So a (sequence, head, array) is split over CTAs by the
// rows' columns only (32 bytes, HBM's sector, or more); copies to other blocks by rows
// as well. HBM-bound: 2 x the kept rows' bytes; a lane has four 16-byte pieces in flight.
//
// Launch 3, with a free list: the blocks behind the new ends are pushed.
//
// A launch's CTAs may be resident while the one before it still writes (programmatic dependent
// launch), so what another launch may have written (the weights, the table, the lists) is read from L2
// (__ldcg) behind the wait: the read-only path wants data that no one writes while the grid is resident.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "launch.h"
#include "pdecode.h"
#include "tc5.cuh"

namespace pd {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kLoads = 4;                        // a thread's loads in flight
constexpr int kMoveThreads = 256;
constexpr int kCachedKeys = 48 * 1024;           // weights in shared memory
constexpr int kMaxArrays = 5;

// n / d for n < 2^31 by a multiplication (Granlund and Montgomery's round-up method): with l =
// ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n) >> l. (One CTA divides for
// tens of thousands of keys: the GPU's own integer division was half of its time.)
struct FastDiv {
  uint32_t d, m, l;
  explicit FastDiv(uint32_t d_ = 1) : d(d_), l(0) {
    while ((1ull << l) < d) ++l;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(m, static_cast<uint32_t>(n)) + static_cast<uint32_t>(n)) >> l);
  }
  __device__ __forceinline__ int mod(int n) const { return n - div(n) * static_cast<int>(d); }
};

struct MoveArray {
  uint8_t* base;
  int row_bytes;   // of one key and head
  int vec;         // bytes a thread moves at once: 16, 8 or 4
  int keys_first;  // [num_blocks, block_size, Hkv, row], else [num_blocks, Hkv, block_size, row]
  int slices;      // CTAs that a row's columns are split over
};

struct EvictArgs {
  MoveArray arrays[kMaxArrays];
  int n_arrays, slices, parts;  // slices: of all arrays together; parts: CTAs that rows are split over (copies)
  const float* weights;
  const int32_t *table, *table_out, *lens;
  int32_t *lens_out, *free_blocks, *free_count;
  int4* moves;                  // workspace: [B, Hkv, most] (from, to) as slots, then as rows of [block, head, key]
  int32_t* kept;                // [B, Hkv, most]: a cut sequence's kept keys
  int32_t* old_lens;            // [B] (-1: a bad length)
  uint32_t* error_flag;
  int B, Hkv, block_size, num_blocks, max_blocks, max_blocks_out;
  FastDiv bs;                   // block_size
  int keep, trigger, first, recent;
  int most;                     // keys that a sequence can keep
  int in_place;
  int cluster;                  // CTAs of a (sequence, head) in the select
};

// The weight as an integer that orders as it does, NaN below all; zeros of either sign are equal.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_key[];            // the CTA's keys, kCachedKeys of them at most
  __shared__ uint32_t s_hist[2][256], s_sum[256], s_pick[2];
  __shared__ int s_count[2][32];
  __shared__ uint32_t s_total[2];                // the CTA's keys above and equal to the m-th largest
  const int C = a.cluster, rank = blockIdx.x % C, u = blockIdx.x / C;
  const int b = u / a.Hkv, h = u % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = __ldcg(a.lens + b);
  const bool bad = L < 0 || L > a.max_blocks * a.block_size;
  if (h == 0 && rank == 0 && threadIdx.x == 0) {
    a.old_lens[b] = bad ? -1 : L;
    if (bad && a.error_flag) atomicOr(a.error_flag, PD_DEVERR_SEQ_LEN);
  }
  const bool cut = L > a.trigger;
  if (bad || (a.in_place && !cut)) return;
  const int32_t* row = a.table + static_cast<long long>(b) * a.max_blocks;
  const int32_t* row_out = a.in_place ? row : a.table_out + static_cast<long long>(b) * a.max_blocks_out;
  int4* out = a.moves + (static_cast<long long>(b) * a.Hkv + h) * a.most;
  int32_t* kept = a.kept + (static_cast<long long>(b) * a.Hkv + h) * a.most;
  // where the n kept keys come from and go to
  const int thread = rank * kSelectThreads + threadIdx.x, threads = C * kSelectThreads;  // of the cluster
  auto list_moves = [&](int n) {
    for (int i0 = thread; i0 < n; i0 += threads * kLoads) {
      int j[kLoads], from[kLoads], to[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int i = i0 + k * threads;
        j[k] = i < n && cut ? __ldcg(kept + i) : i;
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int i = i0 + k * threads;
        from[k] = i < n ? __ldcg(row + a.bs.div(j[k])) : 0;
        to[k] = i < n ? __ldcg(row_out + a.bs.div(i)) : 0;
      }
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int i = i0 + k * threads;
        if (i >= n) continue;
        int4 m = make_int4(-1, -1, -1, -1);  // (not in the cache: not moved)
        if (from[k] >= 0 && from[k] < a.num_blocks && to[k] >= 0 && to[k] < a.num_blocks) {
          const int of = a.bs.mod(j[k]), ot = a.bs.mod(i);
          m = make_int4(from[k] * a.block_size + of, to[k] * a.block_size + ot, (from[k] * a.Hkv + h) * a.block_size + of,
                        (to[k] * a.Hkv + h) * a.block_size + ot);
        } else if (a.error_flag) {
          atomicOr(a.error_flag, PD_DEVERR_BLOCK_ID);
        }
        out[i] = m;
      }
    }
  };
  if (!cut) {
    list_moves(L);
    return;
  }
  const int lo = a.first, hi = L - a.recent;     // the keys that are chosen from
  auto weight = [&](int j, int blk) -> uint32_t {  // (a bad block counts as NaN; a move from it reports it)
    if (blk < 0 || blk >= a.num_blocks) return 0u;
    return order_of(__ldcg(a.weights + (static_cast<long long>(blk) * a.Hkv + h) * a.block_size + a.bs.mod(j)));
  };
  auto load = [&](int j) -> uint32_t { return weight(j, __ldcg(row + a.bs.div(j))); };
  const int all = hi - lo, share = (all + C - 1) / C;
  const int c0 = min(rank * share, all), n = min(c0 + share, all) - c0;  // this CTA's run: lo + c0 ..
  const int cached = min(n, kCachedKeys);
  for (int i0 = threadIdx.x; i0 < cached; i0 += kSelectThreads * kLoads) {
    int blk[kLoads];
    uint32_t u[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int i = i0 + k * kSelectThreads;
      blk[k] = i < cached ? __ldcg(row + a.bs.div(lo + c0 + i)) : -1;
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) u[k] = weight(lo + c0 + i0 + k * kSelectThreads, blk[k]);
#pragma unroll
    for (int k = 0; k < kLoads; ++k)
      if (i0 + k * kSelectThreads < cached) s_key[i0 + k * kSelectThreads] = u[k];
  }
  __syncthreads();
  auto key = [&](int i) -> uint32_t { return i < kCachedKeys ? s_key[i] : load(lo + c0 + i); };
  const int m = a.keep - a.first - a.recent;     // of all of them are kept: fewer than all, as L > trigger >= keep
  // the m-th largest, and how many equal to it are kept
  uint32_t pick = 0, mask = 0;
  uint32_t want = m;
  if (threadIdx.x < 512) s_hist[threadIdx.x >> 8][threadIdx.x & 255] = 0;
  __syncthreads();
  if (m > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      uint32_t* hist = s_hist[shift >> 3 & 1];
      for (int i = threadIdx.x; i < n; i += kSelectThreads) {
        const uint32_t u = key(i);
        if ((u & mask) == pick) atomicAdd(&hist[(u >> shift) & 255u], 1u);
      }
      if (C > 1) {
        cluster_sync();
        if (threadIdx.x < 256) {
          uint32_t c[8], sum = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            c[k] = k < C ? ld_peer_u32(peer_smem(static_cast<uint32_t>(__cvta_generic_to_shared(hist + threadIdx.x)), k)) : 0u;
#pragma unroll
          for (int k = 0; k < 8; ++k) sum += c[k];
          s_sum[threadIdx.x] = sum;
        }
      }
      __syncthreads();
      if (warp == 0) {  // lane: eight digits, the largest ones first
        const uint32_t* counts = C > 1 ? s_sum : hist;
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int d = 0; d < 8; ++d) sum += c[d] = counts[255 - (lane * 8 + d)];
        uint32_t above = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, above, o);
          if (lane >= o) above += y;
        }
        above -= sum;
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          if (above < want && want <= above + c[d]) {
            s_pick[0] = 255 - (lane * 8 + d);
            s_pick[1] = want - above;
          }
          above += c[d];
        }
      }
      // (the peers read this histogram; the one before, which the next pass fills, is read by nobody)
      if (warp == 1)
        for (int i = lane; i < 256; i += 32) s_hist[(shift >> 3 & 1) ^ 1][i] = 0;
      __syncthreads();
      pick |= s_pick[0] << shift;
      mask |= 255u << shift;
      want = s_pick[1];
    }
  }
  // a warp's run of keys; counts of those above and equal
  const int run = (n + 31) / 32, r0 = min(warp * run, n), r1 = min(r0 + run, n);
  int above = 0, equal = 0;
  if (m > 0) {
    for (int i = r0 + lane; i < r1; i += 32) {
      const uint32_t u = key(i);
      above += u > pick;
      equal += u == pick;
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    above += __shfl_xor_sync(0xffffffffu, above, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
  }
  if (lane == 0) {
    s_count[0][warp] = above;
    s_count[1][warp] = equal;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    int sum = 0;
    for (int w = 0; w < 32; ++w) sum += s_count[threadIdx.x][w];
    s_total[threadIdx.x] = static_cast<uint32_t>(sum);
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  int before = 0, ties = 0;                      // kept keys and ties of earlier runs
  for (int k = 0; k < rank; ++k) {
    const uint32_t peer = peer_smem(static_cast<uint32_t>(__cvta_generic_to_shared(s_total)), k);
    before += static_cast<int>(ld_peer_u32(peer));
    ties += static_cast<int>(ld_peer_u32(peer + 4));
  }
  for (int w = 0; w < warp; ++w) {
    before += s_count[0][w];
    ties += s_count[1][w];
  }
  const int quota = static_cast<int>(want);
  before += min(ties, quota);
  for (int i = thread; i < a.first; i += threads) __stcg(kept + i, i);
  for (int i = thread; i < a.recent; i += threads) __stcg(kept + a.keep - a.recent + i, hi + i);
  if (m > 0) {
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = r0; i0 < r1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t u = i < r1 ? key(i) : 0u;
      const bool tie = i < r1 && u == pick;
      const uint32_t tie_mask = __ballot_sync(0xffffffffu, tie);
      const bool keep = i < r1 && (u > pick || (tie && ties + __popc(tie_mask & below) < quota));
      const uint32_t keep_mask = __ballot_sync(0xffffffffu, keep);
      if (keep) __stcg(kept + a.first + before + __popc(keep_mask & below), lo + c0 + i);
      before += __popc(keep_mask);
      ties += __popc(tie_mask);
    }
  }
  if (C > 1) cluster_sync();  // (and no peer reads this CTA's shared memory any more)
  else __syncthreads();
  list_moves(a.keep);
}

template <class V>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const MoveArray& arr, int b, int h, int slice, int part, int n) {
  const int vecs = arr.row_bytes / static_cast<int>(sizeof(V));
  const int v0 = vecs * slice / arr.slices, width = vecs * (slice + 1) / arr.slices - v0;
  const int rows = kMoveThreads / width;         // rows side by side (threads beyond them idle)
  const int tv = threadIdx.x % width, tr = threadIdx.x / width;
  const int4* moves = a.moves + (static_cast<long long>(b) * a.Hkv + h) * a.most;
  // rows of this part (one part in place: its rows are taken in order)
  const int share = (n + a.parts - 1) / a.parts, j0 = part * share, j1 = min(j0 + share, n);
  const bool keys_first = arr.keys_first != 0;
  auto load = [&](int base, int2 (&m)[kLoads]) {  // where the thread's rows of a batch come from and go to
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int i = base + k * rows + tr;
      m[k] = make_int2(-1, -1);
      if (tr < rows && i < j1) m[k] = __ldcg(reinterpret_cast<const int2*>(moves + i) + (keys_first ? 0 : 1));
    }
  };
  auto at = [&](int row) -> V* {
    const long long r = keys_first ? static_cast<long long>(row) * a.Hkv + h : row;
    return reinterpret_cast<V*>(arr.base + r * arr.row_bytes) + v0 + tv;
  };
  int2 m[kLoads], next[kLoads];
  load(j0, m);
  for (int base = j0; base < j1; base += rows * kLoads) {
    V x[kLoads];
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (m[k].x < 0 || m[k].x == m[k].y) m[k].y = -1;  // (nothing to move)
      if (m[k].y >= 0) x[k] = *at(m[k].x);
    }
    load(base + rows * kLoads, next);
    if (a.in_place) __syncthreads();
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (m[k].y >= 0) *at(m[k].y) = x[k];
      m[k] = next[k];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const EvictArgs a) {
  // CTA: ((sequence, head), slice of an array, part of the rows)
  const int part = blockIdx.x % a.parts, s = blockIdx.x / a.parts % a.slices, u = blockIdx.x / a.parts / a.slices;
  const int b = u / a.Hkv, h = u % a.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = __ldcg(a.old_lens + b);
  const bool cut = L > a.trigger;
  const int n = cut ? a.keep : max(L, 0);
  if (h == 0 && s == 0 && part == 0 && threadIdx.x == 0) {
    if (L >= 0) a.lens_out[b] = n;
    else if (a.lens_out != a.lens) a.lens_out[b] = 0;
  }
  if (a.in_place && !cut) return;
  int i = 0, slice = s;
  while (slice >= a.arrays[i].slices) slice -= a.arrays[i++].slices;
  const MoveArray arr = a.arrays[i];
  if (arr.vec == 16) move_rows<uint4>(a, arr, b, h, slice, part, n);
  else if (arr.vec == 8) move_rows<uint2>(a, arr, b, h, slice, part, n);
  else move_rows<uint32_t>(a, arr, b, h, slice, part, n);
}

// One CTA: the blocks behind the cut sequences' new ends go to the free list.
__global__ void __launch_bounds__(1024) free_tail_kernel(const EvictArgs a) {
  __shared__ long long s_warp[32], s_off[1024];
  __shared__ int s_n[1024];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int bs = a.block_size, held = (a.keep + bs - 1) / bs;
  long long count = *a.free_count;
  bool full = false;
  if (count < 0 || count > a.num_blocks) {
    if (threadIdx.x == 0 && a.error_flag) atomicOr(a.error_flag, PD_DEVERR_FREE_LIST);
    return;
  }
  __syncthreads();  // (all have read the count)
  for (int b0 = 0; b0 < a.B; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    int v = 0;
    if (b < a.B) {
      const int L = __ldcg(a.old_lens + b);
      if (L > a.trigger) v = (L + bs - 1) / bs - held;
    }
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    s_off[threadIdx.x] = count + before + x - v;
    s_n[threadIdx.x] = v;
    __syncthreads();
    for (int i = warp; i < min(1024, a.B - b0); i += 32) {
      const int32_t* row = a.table + static_cast<long long>(b0 + i) * a.max_blocks + held;
      for (int k = lane; k < s_n[i]; k += 32) {
        const long long at = s_off[i] + k;
        int blk = __ldcg(row + k);
        if (blk < 0 || blk >= a.num_blocks) {
          if (a.error_flag) atomicOr(a.error_flag, PD_DEVERR_BLOCK_ID);
          blk = -1;
        }
        if (at < a.num_blocks) a.free_blocks[at] = blk;
        else full = true;
      }
    }
    count = min(count + total, static_cast<long long>(a.num_blocks));
    __syncthreads();
  }
  if (full && a.error_flag) atomicOr(a.error_flag, PD_DEVERR_FREE_LIST);
  if (threadIdx.x == 0) *a.free_count = static_cast<int32_t>(count);
}

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

pd_status check(const pd_dims* d, const pd_eviction* e) {
  if (!d || !e) return PD_ERR_NULL;
  if (d->B < 0 || d->Hkv < 1 || d->D < 16 || d->D % 16 != 0 || d->block_size < 1 || d->num_blocks < 0 ||
      d->max_blocks_per_seq < 0)
    return PD_ERR_SHAPE;
  if (d->kv_dtype < PD_KV_F16 || d->kv_dtype > PD_KV_FP4_BF16) return PD_ERR_DTYPE;
  if (e->keep < 1 || e->trigger < e->keep || e->first < 0 || e->recent < 0 ||
      static_cast<long long>(e->first) + e->recent > e->keep)
    return PD_ERR_SHAPE;
  const bool fp4 = d->kv_dtype == PD_KV_FP4 || d->kv_dtype == PD_KV_FP4_BF16;  // (block scales move four bytes at a time)
  if (d->D > 512 || (fp4 && d->D % 64 != 0) || static_cast<long long>(d->max_blocks_per_seq) * d->block_size > (1ll << 30) ||
      static_cast<long long>(d->num_blocks) * d->block_size * d->Hkv > 0x7fffffffll ||
      static_cast<long long>(d->B) * d->Hkv > (1 << 22))
    return PD_ERR_UNSUPPORTED;
  return PD_OK;
}

// Keys that a sequence can be left with in the workspace's lists.
long long most_kept(const pd_dims& d, const pd_eviction& e) {
  return std::min<long long>(e.trigger, static_cast<long long>(d.max_blocks_per_seq) * d.block_size);
}
size_t workspace_of(const pd_dims& d, const pd_eviction& e, size_t* off_lens) {
  const size_t moves = (static_cast<size_t>(d.B) * d.Hkv * most_kept(d, e) * 20 + 255) / 256 * 256;
  if (off_lens) *off_lens = moves;
  return moves + static_cast<size_t>(d.B) * 4;
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" size_t pd_evict_workspace_bytes(const pd_dims* dims, const pd_eviction* evict) {
  return check(dims, evict) == PD_OK ? workspace_of(*dims, *evict, nullptr) : 0;
}

extern "C" pd_status evict_kv_cache(void* k_cache, void* v_cache, void* k_block_scale, void* v_block_scale,
                                    float* key_weights, const int32_t* block_table, const int32_t* seq_lens,
                                    const pd_eviction* evict, const int32_t* block_table_out, int max_blocks_out,
                                    int32_t* seq_lens_out, int32_t* free_blocks, int32_t* free_count,
                                    const pd_dims* dims, void* workspace, size_t workspace_bytes,
                                    uint32_t* error_flag, void* stream) {
  const pd_status st = check(dims, evict);
  if (st != PD_OK) return st;
  const pd_dims& d = *dims;
  const pd_eviction& e = *evict;
  const bool fp4 = d.kv_dtype == PD_KV_FP4 || d.kv_dtype == PD_KV_FP4_BF16;
  const long long cap = static_cast<long long>(d.max_blocks_per_seq) * d.block_size;
  if (block_table_out != nullptr &&
      (max_blocks_out < 0 || static_cast<long long>(max_blocks_out) * d.block_size < most_kept(d, e)))
    return PD_ERR_SHAPE;
  if ((free_blocks != nullptr) != (free_count != nullptr)) return PD_ERR_NULL;
  if (free_blocks != nullptr && block_table_out != nullptr) return PD_ERR_SHAPE;
  if (d.B == 0) return PD_OK;
  if (!seq_lens || !seq_lens_out || !key_weights) return PD_ERR_NULL;
  if (cap > 0 && (!block_table || !k_cache || !v_cache || (fp4 && (!k_block_scale || !v_block_scale)))) return PD_ERR_NULL;
  if (misaligned(k_cache, 15) || misaligned(v_cache, 15) || misaligned(k_block_scale, 15) ||
      misaligned(v_block_scale, 15) || misaligned(key_weights, 3) || misaligned(block_table, 3) ||
      misaligned(seq_lens, 3) || misaligned(block_table_out, 3) || misaligned(seq_lens_out, 3) ||
      misaligned(free_blocks, 3) || misaligned(free_count, 3) || misaligned(error_flag, 3))
    return PD_ERR_ALIGN;
  size_t off_lens;
  const size_t need = workspace_of(d, e, &off_lens);
  if (!workspace || workspace_bytes < need) return PD_ERR_WORKSPACE;
  if (misaligned(workspace, 255)) return PD_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return PD_ERR_CUDA;

  EvictArgs a{};
  a.weights = key_weights;
  a.table = block_table;
  a.in_place = block_table_out == nullptr || block_table_out == block_table;
  a.table_out = block_table_out;
  a.lens = seq_lens;
  a.lens_out = seq_lens_out;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.moves = static_cast<int4*>(workspace);
  a.most = static_cast<int>(most_kept(d, e));
  a.kept = reinterpret_cast<int32_t*>(a.moves + static_cast<size_t>(d.B) * d.Hkv * a.most);
  a.old_lens = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + off_lens);
  a.error_flag = error_flag;
  a.B = d.B;
  a.Hkv = d.Hkv;
  a.block_size = d.block_size;
  a.bs = FastDiv(static_cast<uint32_t>(d.block_size));
  a.num_blocks = d.num_blocks;
  a.max_blocks = d.max_blocks_per_seq;
  a.max_blocks_out = max_blocks_out;
  a.keep = e.keep;
  a.trigger = e.trigger;
  a.first = e.first;
  a.recent = e.recent;

  const bool two_byte = d.kv_dtype == PD_KV_F16 || d.kv_dtype == PD_KV_BF16;
  const int row = fp4 ? d.D / 2 : two_byte ? 2 * d.D : d.D;
  auto add = [&](void* base, int bytes, bool keys_first) {
    const int vec = bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : 4;
    a.arrays[a.n_arrays++] = MoveArray{static_cast<uint8_t*>(base), bytes, vec, keys_first, 1};
  };
  add(k_cache, row, !fp4);
  add(v_cache, row, !fp4);
  if (fp4) {
    add(k_block_scale, d.D / 16, false);
    add(v_block_scale, d.D / 16, false);
  }
  add(key_weights, 4, false);
  // in place: columns of at least 32 bytes, while the CTAs are fewer than two per SM
  const long long units = static_cast<long long>(d.B) * d.Hkv;
  a.parts = 1;
  if (a.in_place) {
    for (int i = 0; i < 2; ++i) {
      int& s = a.arrays[i].slices;
      while (units * 2 * s < 2 * sms && row / (2 * s) >= 32) s *= 2;
    }
  } else {
    // up to four rounds of the resident CTAs (B = 32, fp16: one round 107.4 us, two 98.5, four 98.3), each with a
    // batch of its threads' loads at least (B = 1, 4-bit, 4096 keys kept: a batch 19.2 us, half of one 21.5, two 20.1)
    while (units * a.n_arrays * a.parts < 16 * sms &&
           static_cast<long long>(a.most) * (row / 16) / (2 * a.parts) >= kMoveThreads * kLoads)
      a.parts *= 2;
  }
  a.slices = 0;
  for (int i = 0; i < a.n_arrays; ++i) a.slices += a.arrays[i].slices;

  auto s = static_cast<cudaStream_t>(stream);
  static unsigned long long attr_ctx[64] = {};
  cudaError_t err = once_per_context(attr_ctx, [] {
    return cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCachedKeys * 4);
  });
  // as many CTAs a head as the GPU's SMs are, runs of 1024 keys and more
  a.cluster = 1;
  while (a.cluster < 8 && units * a.cluster * 2 <= sms && cap / (2 * a.cluster) >= 1024) a.cluster *= 2;
  const int smem = static_cast<int>(std::min<long long>((cap + a.cluster - 1) / a.cluster, kCachedKeys)) * 4;
  const long long ctas = units * a.slices * a.parts;
  if (ctas > 0x7fffffffll) return PD_ERR_UNSUPPORTED;
  const WorkspaceLock lock(workspace, true);
  if (err == cudaSuccess)
    err = launch_pdl(select_kernel, static_cast<int>(units * a.cluster), kSelectThreads, smem, s, a.cluster, a);
  if (err == cudaSuccess) err = launch_pdl(move_kernel, static_cast<int>(ctas), kMoveThreads, 0, s, 1, a);
  if (err == cudaSuccess && free_blocks != nullptr) err = launch_pdl(free_tail_kernel, 1, 1024, 0, s, 1, a);
  return err == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}
