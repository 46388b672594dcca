// evict.cu -- eviction from the paged caches by the attention weight that keys have
// collected (evict_kv_cache): each KV head of a long sequence keeps its first keys, its
// last ones and the heaviest of the rest, moved together in order.
//
// Launch 1, select_kernel: a CTA for each (sequence, KV head). The weights, as integers
// that order as the numbers do, are held in shared memory (beyond its size they are
// read again); the m-th largest is found digit by digit (8 bits, most significant first)
// from histograms; then each warp counts what its run of keys keeps, a scan over the
// warps gives its place, and it writes the kept keys' indices in order. Of the keys equal
// to the m-th largest the lowest indices are kept.
//
// Launch 2, move_kernel: rows move to slots at or below their own. In place that is safe
// without a second buffer when a CTA takes its rows in order: it loads R rows, waits for
// all its threads, and stores them; the next R rows' sources are at or behind the R-th
// slot from here, and no store comes before it. So a (sequence, head, array) is split over CTAs by the
// rows' columns only (pieces of 32 bytes, HBM's sector, or more); copies to other blocks by rows
// as well. HBM-bound: 2 x the kept rows' bytes.
//
// Launch 3, with a free list: the blocks behind the new ends are pushed.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "launch.h"
#include "pdecode.h"

namespace pd {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kMoveThreads = 512;
constexpr int kMoveRows = 4;                     // rows that a thread has in flight
constexpr int kCachedKeys = 48 * 1024;           // weights in shared memory
constexpr int kMaxArrays = 5;

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
  int32_t *kept, *old_lens;     // workspace: [B, Hkv, keep], [B] (-1: a bad length)
  uint32_t* error_flag;
  int B, Hkv, block_size, num_blocks, max_blocks, max_blocks_out;
  int keep, trigger, first, recent;
  int in_place;
};

// The weight as an integer that orders as it does, NaN below all.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w);
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t s_key[];            // [min(keys, kCachedKeys)]
  __shared__ uint32_t s_hist[256], s_pick[2];
  __shared__ int s_count[2][32];
  const int b = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = __ldg(a.lens + b);
  const bool bad = L < 0 || L > a.max_blocks * a.block_size;
  if (h == 0 && threadIdx.x == 0) {
    a.old_lens[b] = bad ? -1 : L;
    if (bad && a.error_flag) atomicOr(a.error_flag, PD_DEVERR_SEQ_LEN);
  }
  if (bad || L <= a.trigger) return;
  const int32_t* row = a.table + static_cast<long long>(b) * a.max_blocks;
  const int lo = a.first, hi = L - a.recent;     // the keys that are chosen from
  auto load = [&](int j) -> uint32_t {
    const int blk = __ldg(row + j / a.block_size);
    if (blk < 0 || blk >= a.num_blocks) return 0u;  // (the move reports it)
    return order_of(__ldg(a.weights + (static_cast<long long>(blk) * a.Hkv + h) * a.block_size + j % a.block_size));
  };
  const int cached = min(hi - lo, kCachedKeys);
  for (int i = threadIdx.x; i < cached; i += kSelectThreads) s_key[i] = load(lo + i);
  __syncthreads();
  auto key = [&](int i) -> uint32_t { return i < kCachedKeys ? s_key[i] : load(lo + i); };
  const int n = hi - lo;
  const int m = a.keep - a.first - a.recent;     // of them are kept: m < n, as L > trigger >= keep
  // the m-th largest, and how many equal to it are kept
  uint32_t pick = 0, mask = 0;
  uint32_t want = m;
  if (m > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (threadIdx.x < 256) s_hist[threadIdx.x] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kSelectThreads) {
        const uint32_t u = key(i);
        if ((u & mask) == pick) atomicAdd(&s_hist[(u >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {  // lane: eight digits, the largest ones first
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int d = 0; d < 8; ++d) sum += c[d] = s_hist[255 - (lane * 8 + d)];
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
  int before = 0, ties = 0;                      // kept keys and ties of earlier runs
  for (int w = 0; w < warp; ++w) {
    before += s_count[0][w];
    ties += s_count[1][w];
  }
  const int quota = static_cast<int>(want);
  before += min(ties, quota);
  int32_t* out = a.kept + (static_cast<long long>(b) * a.Hkv + h) * a.keep;
  for (int i = threadIdx.x; i < a.first; i += kSelectThreads) out[i] = i;
  for (int i = threadIdx.x; i < a.recent; i += kSelectThreads) out[a.keep - a.recent + i] = hi + i;
  if (m > 0) {
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = r0; i0 < r1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t u = i < r1 ? key(i) : 0u;
      const bool tie = i < r1 && u == pick;
      const uint32_t tie_mask = __ballot_sync(0xffffffffu, tie);
      const bool keep = i < r1 && (u > pick || (tie && ties + __popc(tie_mask & below) < quota));
      const uint32_t keep_mask = __ballot_sync(0xffffffffu, keep);
      if (keep) out[a.first + before + __popc(keep_mask & below)] = lo + i;
      before += __popc(keep_mask);
      ties += __popc(tie_mask);
    }
  }
}

template <class V>
__device__ __forceinline__ void move_rows(const EvictArgs& a, const MoveArray& arr, int b, int h, int slice, int part,
                                          int n, bool cut) {
  const int vecs = arr.row_bytes / static_cast<int>(sizeof(V));
  const int v0 = vecs * slice / arr.slices, v1 = vecs * (slice + 1) / arr.slices, width = v1 - v0;
  const int rows = kMoveThreads / width;         // rows side by side (threads beyond them idle)
  const int tv = threadIdx.x % width, tr = threadIdx.x / width;
  const int32_t* from = a.table + static_cast<long long>(b) * a.max_blocks;
  const int32_t* to = a.in_place ? from : a.table_out + static_cast<long long>(b) * a.max_blocks_out;
  const int32_t* kept = a.kept + (static_cast<long long>(b) * a.Hkv + h) * a.keep;
  auto at = [&](const int32_t* table, int j, bool report) -> V* {
    const int blk = __ldg(table + j / a.block_size), off = j % a.block_size;
    if (blk < 0 || blk >= a.num_blocks) {
      if (report && a.error_flag) atomicOr(a.error_flag, PD_DEVERR_BLOCK_ID);
      return nullptr;
    }
    const long long row = arr.keys_first ? (static_cast<long long>(blk) * a.block_size + off) * a.Hkv + h
                                         : (static_cast<long long>(blk) * a.Hkv + h) * a.block_size + off;
    return reinterpret_cast<V*>(arr.base + row * arr.row_bytes) + v0 + tv;
  };
  // rows of this part (one part in place: its rows are taken in order)
  const int share = (n + a.parts - 1) / a.parts, j0 = part * share, j1 = min(j0 + share, n);
  const bool live = tr < rows;
  for (int base = j0; base < j1; base += rows * kMoveRows) {
    V x[kMoveRows];
    V* dst[kMoveRows];
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k) {
      const int i = base + k * rows + tr;
      dst[k] = nullptr;
      if (live && i < j1) {
        const int j = cut ? __ldg(kept + i) : i;
        if (a.in_place && j == i) continue;
        const V* src = at(from, j, true);
        V* d = at(to, i, true);
        if (src != nullptr && d != nullptr) {
          x[k] = *src;
          dst[k] = d;
        }
      }
    }
    if (a.in_place) __syncthreads();
#pragma unroll
    for (int k = 0; k < kMoveRows; ++k)
      if (dst[k] != nullptr) *dst[k] = x[k];
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a) {
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
  if (arr.vec == 16) move_rows<uint4>(a, arr, b, h, slice, part, n, cut);
  else if (arr.vec == 8) move_rows<uint2>(a, arr, b, h, slice, part, n, cut);
  else move_rows<uint32_t>(a, arr, b, h, slice, part, n, cut);
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
        int blk = __ldg(row + k);
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
  if (d->D > 512 || static_cast<long long>(d->max_blocks_per_seq) * d->block_size > (1ll << 30) ||
      static_cast<long long>(d->num_blocks) * d->block_size > 0x7fffffffll ||
      static_cast<long long>(d->B) * d->Hkv > (1 << 22))
    return PD_ERR_UNSUPPORTED;
  return PD_OK;
}

size_t workspace_of(const pd_dims& d, const pd_eviction& e, size_t* off_lens) {
  // (a sequence that is cut has at least keep keys in its table)
  const size_t most = std::min<size_t>(e.keep, static_cast<size_t>(d.max_blocks_per_seq) * d.block_size);
  const size_t kept = (static_cast<size_t>(d.B) * d.Hkv * most * 4 + 255) / 256 * 256;
  if (off_lens) *off_lens = kept;
  return kept + static_cast<size_t>(d.B) * 4;
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
      (max_blocks_out < 0 || static_cast<long long>(max_blocks_out) * d.block_size <
                                 std::min<long long>(cap, std::max(e.keep, e.trigger))))
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
  a.kept = static_cast<int32_t*>(workspace);
  a.old_lens = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + off_lens);
  a.error_flag = error_flag;
  a.B = d.B;
  a.Hkv = d.Hkv;
  a.block_size = d.block_size;
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
    const int vec = bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : bytes % 4 == 0 ? 4 : 0;
    a.arrays[a.n_arrays++] = MoveArray{static_cast<uint8_t*>(base), bytes, vec, keys_first, 1};
    return vec != 0;
  };
  bool ok = add(k_cache, row, !fp4) && add(v_cache, row, !fp4);
  if (fp4) ok = ok && add(k_block_scale, d.D / 16, false) && add(v_block_scale, d.D / 16, false);
  ok = ok && add(key_weights, 4, false);
  if (!ok) return PD_ERR_UNSUPPORTED;
  // in place: columns of at least 32 bytes, while the CTAs are fewer than two per SM
  const long long units = static_cast<long long>(d.B) * d.Hkv;
  a.parts = 1;
  if (a.in_place) {
    for (int i = 0; i < 2; ++i) {
      int& s = a.arrays[i].slices;
      while (units * 2 * s < 2 * sms && row / (2 * s) >= 32) s *= 2;
    }
  } else {
    const long long rows = std::min<long long>(cap, std::max(e.keep, e.trigger));
    while (units * a.n_arrays * a.parts < 8 * sms && rows / (2 * a.parts) >= 32) a.parts *= 2;
  }
  a.slices = 0;
  for (int i = 0; i < a.n_arrays; ++i) a.slices += a.arrays[i].slices;

  auto s = static_cast<cudaStream_t>(stream);
  static unsigned long long attr_ctx[64] = {};
  cudaError_t err = once_per_context(attr_ctx, [] {
    return cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCachedKeys * 4);
  });
  const int smem = static_cast<int>(std::min<long long>(cap, kCachedKeys)) * 4;
  if (err == cudaSuccess) err = launch_pdl(select_kernel, static_cast<int>(units), kSelectThreads, smem, s, 1, a);
  const long long ctas = units * a.slices * a.parts;
  if (ctas > 0x7fffffffll) return PD_ERR_UNSUPPORTED;
  if (err == cudaSuccess) err = launch_pdl(move_kernel, static_cast<int>(ctas), kMoveThreads, 0, s, 1, a);
  if (err == cudaSuccess && free_blocks != nullptr) err = launch_pdl(free_tail_kernel, 1, 1024, 0, s, 1, a);
  return err == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}
