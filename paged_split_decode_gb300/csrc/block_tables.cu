// block_tables.cu -- block tables, slot maps and the free list, built on the
// GPU from the requests' lengths (build_block_tables, release_blocks): what a
// serving step needs before write_kv_cache and decode_paged_varlen, without a
// copy to the host.
//
// Mathematics, with bs keys per block (sequence b holds held_b blocks before
// the step and wants want_b after it):
//   held_b = ceil(context_b / bs), want_b = ceil((context_b + query_b) / bs),
//   start_b = sum_{a<b} query_a, off_b = sum_{a<b} (want_a - held_a);
//   block_table[b][held_b + i] = free[count - 1 - (off_b + i)]  (a stack: the
//   k-th block taken is the k-th from the top), count -= sum (want - held);
//   token t of sequence b (start_b <= t < start_b + query_b) has position
//   p = context_b + t - start_b and slot block_table[b][p / bs] * bs + p % bs.
// A release pushes the blocks of the marked sequences in sequence order.
//
// Latency-bound: a few bytes per sequence and 12 per token. One launch of one
// thread-block cluster: every CTA reads all lengths and scans them (each
// thread a run of consecutive sequences, then one block scan of one barrier),
// which costs less than a second launch; the cluster barrier then makes the in-place
// forms safe (seq_lens over context_lens, the count over itself), since no
// CTA writes before all have read. Tokens and blocks are dealt to the
// cluster's warps in contiguous shares: a lane finds its first item's sequence
// by a binary search in the prefix held in shared memory and the next ones
// from there, with eight items' loads in flight.
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"
#include "pdecode.h"

namespace pd {
namespace {

constexpr int kMaxTableB = 16384;  // three ints per sequence in shared memory
constexpr uint32_t kSatMax = 0x7fffffffu;

// Saturating sums of non-negative 31-bit values: associative, so a scan of
// them is well defined however the lengths overflow.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSatMax); }

// Exclusive scans over the block of K values per thread at once; `total` gets
// the sums. One barrier: every warp scans the warps' sums for itself.
template <int NT, int K>
__device__ __forceinline__ void block_scan(uint32_t (&v)[K], uint32_t (&s_warp)[K][32], uint32_t (&total)[K]) {
  constexpr int NW = NT / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    x[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] = sat_add(x[k], y);
    }
    if (lane == 31) s_warp[k][warp] = x[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    uint32_t w = lane < NW ? s_warp[k][lane] : 0u;
#pragma unroll
    for (int o = 1; o < NW; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = sat_add(w, y);
    }
    total[k] = __shfl_sync(0xffffffffu, w, NW - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    const uint32_t prev = __shfl_up_sync(0xffffffffu, x[k], 1);
    v[k] = sat_add(warp > 0 ? before : 0u, lane > 0 ? prev : 0u);
  }
}

// The sequence whose range holds x: the largest b with pre[b] <= x, given
// pre[0] = 0 <= x < pre[n] (empty ranges before it are passed over).
__device__ __forceinline__ int find_seq(const int* pre, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void raise_bits(uint32_t* flag, uint32_t bits) {
  if (flag && bits) atomicOr(flag, bits);
}

// The warps of the cluster take equal contiguous shares of n items, a lane
// every 32nd of its warp's: `item` is called with each k, in increasing order,
// kBatch of them between two calls of `flush`.
constexpr int kBatch = 8;
template <int NT, class Item, class Flush>
__device__ __forceinline__ void deal(int n, int rank, int ranks, Item item, Flush flush) {
  if (n <= ranks * NT) {  // one item a thread
    const int k = rank * NT + static_cast<int>(threadIdx.x);
    if (k < n) {
      item(k, 0);
      flush(k, 0);
    }
    return;
  }
  const int warps = ranks * (NT / 32), warp = rank * (NT / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int share = (n / warps + 32) / 32 * 32;
  const long long first = static_cast<long long>(warp) * share;
  const int end = static_cast<int>(min(static_cast<long long>(n), first + share));
  for (long long k0 = first + lane; k0 < end; k0 += 32 * kBatch) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long k = k0 + 32 * j;
      if (k < end) item(static_cast<int>(k), j);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long k = k0 + 32 * j;
      if (k < end) flush(static_cast<int>(k), j);
    }
  }
}

// find_seq for increasing x: from the last answer (-1: none yet) forwards.
__device__ __forceinline__ int next_seq(const int* pre, int n, int x, int last) {
  if (last < 0) return find_seq(pre, n, x);
  int b = last;
  for (int step = 0; step < 8; ++step) {
    if (b + 1 >= n || pre[b + 1] > x) return b;
    ++b;
  }
  return find_seq(pre, n, x);
}

struct TableArgs {
  const int32_t *context, *query;
  int32_t* table;
  const int32_t* free_blocks;
  const int32_t* count_in;
  int32_t* count_out;
  int32_t *seq_lens, *q_start;
  int64_t* slots;
  int32_t* positions;
  uint32_t* flag;
  int B, T, bs, num_blocks, max_blocks;
};

// Shared: s_start[B + 1], s_off[B + 1], s_ctx[B] (-1: the sequence is refused).
template <int NT>
__global__ void __launch_bounds__(NT, 1) build_tables_kernel(const TableArgs a) {
  extern __shared__ int s_dyn[];
  int* s_start = s_dyn;
  int* s_off = s_start + a.B + 1;
  int* s_ctx = s_off + a.B + 1;
  __shared__ uint32_t s_warp[2][32];
  __shared__ int s_taken;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
  const long long cap = static_cast<long long>(a.max_blocks) * a.bs;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, t * per), b1 = min(a.B, b0 + per);
  uint32_t bits = 0;
  int count = *a.count_in;
  if (count < 0 || count > a.num_blocks) {
    bits |= PD_DEVERR_FREE_LIST;
    count = count < 0 ? 0 : a.num_blocks;
  }
  if (t == 0) s_taken = 0;
  // lengths -> start and off
  uint32_t qs = 0, ns = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = a.context[b], q = a.query[b];
    const bool ok = c >= 0 && q >= 0 && static_cast<long long>(c) + q <= cap;
    if (!ok) bits |= PD_DEVERR_SEQ_LEN;
    const int need = ok ? (c + q + a.bs - 1) / a.bs - (c + a.bs - 1) / a.bs : 0;
    s_ctx[b] = ok ? c : -1;
    s_start[b] = q > 0 ? q : 0;
    s_off[b] = need;
    qs = sat_add(qs, q > 0 ? q : 0);
    ns = sat_add(ns, need);
  }
  uint32_t run[2] = {qs, ns}, total[2];
  block_scan<NT, 2>(run, s_warp, total);
  uint32_t q_run = run[0], n_run = run[1];
  int taken = 0;
  for (int b = b0; b < b1; ++b) {
    const uint32_t q = s_start[b], need = s_off[b];
    s_start[b] = static_cast<int>(q_run);
    s_off[b] = static_cast<int>(n_run);
    const uint32_t qe = sat_add(q_run, q), ne = sat_add(n_run, need);
    // a sequence is served whole or not at all; those that need blocks fail
    // from the first that does not fit, so the blocks taken are the list's top
    if (q > 0 && qe > static_cast<uint32_t>(a.T)) {
      bits |= PD_DEVERR_QUERY_START;
      s_ctx[b] = -1;
    }
    if (need > 0 && ne > static_cast<uint32_t>(count)) {
      bits |= PD_DEVERR_FREE_LIST;
      s_ctx[b] = -1;
    }
    if (need > 0 && s_ctx[b] >= 0) taken = static_cast<int>(ne);
    q_run = qe;
    n_run = ne;
  }
  if (t == 0) {
    s_start[a.B] = static_cast<int>(total[0]);
    s_off[a.B] = static_cast<int>(total[1]);
  }
  if (taken) atomicMax(&s_taken, taken);
  cluster_sync();  // (and a block barrier) every CTA has read its inputs
  taken = s_taken;

  const int nt = ranks * NT, me = rank * NT + t;
  for (int b = me; b <= a.B; b += nt) {
    a.q_start[b] = s_start[b];
    if (b < a.B) {
      const int c = s_ctx[b];
      // query_b = start_{b+1} - start_b (exact while the sums do not saturate,
      // and a sequence behind a saturated sum is refused). In place, a refused
      // sequence keeps its context: nothing else knows the blocks that it holds.
      if (c >= 0) a.seq_lens[b] = c + (s_start[b + 1] - s_start[b]);
      else if (a.seq_lens != a.context) a.seq_lens[b] = 0;
    }
  }
  if (me == 0) *a.count_out = count - taken;
  {
    int b = -1, blk[kBatch];
    long long at[kBatch];
    deal<NT>(taken, rank, ranks,
         [&](int k, int j) {
           b = next_seq(s_off, a.B, k, b);
           blk[j] = a.free_blocks[count - 1 - k];
           const int held = (s_ctx[b] + a.bs - 1) / a.bs;
           at[j] = static_cast<long long>(b) * a.max_blocks + held + (k - s_off[b]);
         },
         [&](int, int j) {
           if (blk[j] < 0 || blk[j] >= a.num_blocks) bits |= PD_DEVERR_BLOCK_ID;
           a.table[at[j]] = blk[j];
         });
  }
  const int live = min(s_start[a.B], a.T);
  {
    int b = -1, blk[kBatch], pos[kBatch];
    deal<NT>(a.T, rank, ranks,
         [&](int k, int j) {
           pos[j] = -1;
           if (k >= live) return;
           b = next_seq(s_start, a.B, k, b);
           const int c = s_ctx[b];
           if (c < 0) return;
           pos[j] = c + (k - s_start[b]);
           const int n = pos[j] / a.bs, held = (c + a.bs - 1) / a.bs;
           blk[j] = n < held ? a.table[static_cast<long long>(b) * a.max_blocks + n]
                             : a.free_blocks[count - 1 - (s_off[b] + n - held)];
         },
         [&](int k, int j) {
           long long slot = -1;
           if (pos[j] >= 0) {
             if (blk[j] < 0 || blk[j] >= a.num_blocks) bits |= PD_DEVERR_BLOCK_ID;
             else slot = static_cast<long long>(blk[j]) * a.bs + pos[j] % a.bs;
           }
           a.slots[k] = slot;
           if (a.positions) a.positions[k] = max(pos[j], 0);
         });
  }
  raise_bits(a.flag, bits);
}

struct ReleaseArgs {
  const int32_t* table;
  const int32_t* lens;
  const uint8_t* released;
  int32_t* free_blocks;
  const int32_t* count_in;
  int32_t* count_out;
  int32_t* lens_out;
  uint32_t* flag;
  int B, bs, num_blocks, max_blocks;
};

// Shared: s_off[B + 1], s_len[B] (the length to write).
template <int NT>
__global__ void __launch_bounds__(NT, 1) release_kernel(const ReleaseArgs a) {
  extern __shared__ int s_dyn[];
  int* s_off = s_dyn;
  int* s_len = s_off + a.B + 1;
  __shared__ uint32_t s_warp[1][32];
  __shared__ int s_given;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
  const long long cap = static_cast<long long>(a.max_blocks) * a.bs;
  const int per = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, t * per), b1 = min(a.B, b0 + per);
  uint32_t bits = 0;
  int count = *a.count_in;
  if (count < 0 || count > a.num_blocks) {
    bits |= PD_DEVERR_FREE_LIST;
    count = count < 0 ? 0 : a.num_blocks;
  }
  if (t == 0) s_given = 0;
  uint32_t ns = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = a.lens[b];
    int n = 0;
    if (a.released[b]) {
      if (len < 0 || len > cap) bits |= PD_DEVERR_SEQ_LEN;
      else n = (len + a.bs - 1) / a.bs;
    }
    s_len[b] = len;
    s_off[b] = n;
    ns = sat_add(ns, n);
  }
  uint32_t run[1] = {ns}, total[1];
  block_scan<NT, 1>(run, s_warp, total);
  uint32_t n_run = run[0];
  int given = 0;
  for (int b = b0; b < b1; ++b) {
    const uint32_t n = s_off[b], ne = sat_add(n_run, n);
    s_off[b] = static_cast<int>(n_run);
    if (n > 0) {
      if (ne > static_cast<uint32_t>(a.num_blocks - count)) bits |= PD_DEVERR_FREE_LIST;
      else {
        s_len[b] = 0;
        given = static_cast<int>(ne);
      }
    }
    n_run = ne;
  }
  if (t == 0) s_off[a.B] = static_cast<int>(total[0]);
  if (given) atomicMax(&s_given, given);
  cluster_sync();
  given = s_given;
  const int nt = ranks * NT, me = rank * NT + t;
  for (int b = me; b < a.B; b += nt) a.lens_out[b] = s_len[b];
  if (me == 0) *a.count_out = count + given;
  int b = -1, blk[kBatch];
  deal<NT>(given, rank, ranks,
       [&](int k, int j) {
         b = next_seq(s_off, a.B, k, b);
         blk[j] = a.table[static_cast<long long>(b) * a.max_blocks + (k - s_off[b])];
       },
       [&](int k, int j) {
         if (blk[j] < 0 || blk[j] >= a.num_blocks) {
           bits |= PD_DEVERR_BLOCK_ID;
           blk[j] = -1;
         }
         a.free_blocks[count + k] = blk[j];
       });
  raise_bits(a.flag, bits);
}

pd_status check_table_dims(const pd_dims* d) {
  if (!d) return PD_ERR_NULL;
  if (d->B < 0 || d->block_size < 1 || d->num_blocks < 0 || d->max_blocks_per_seq < 0) return PD_ERR_SHAPE;
  // lengths and slots of one sequence fit 31 bits
  if (static_cast<long long>(d->max_blocks_per_seq) * d->block_size > (1ll << 30)) return PD_ERR_UNSUPPORTED;
  if (d->B > kMaxTableB) return PD_ERR_UNSUPPORTED;
  return PD_OK;
}

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// One cluster of `ctas` CTAs of NT threads: 1, 8 (the portable size) or, where
// the device runs such a cluster, 16.
template <int NT, class Kern, class Args>
pd_status launch_cluster(Kern kernel, int ctas, size_t smem, cudaStream_t s, const Args& args) {
  static unsigned long long done[64] = {}, done_occ[64] = {};
  static int cache[64][kMaxCluster + 1] = {};
  const int most = (3 * kMaxTableB + 2) * 4;
  if (once_per_context(done, [&] { return set_kernel_attributes(kernel, most); }) != cudaSuccess) return PD_ERR_CUDA;
  if (ctas > 8) {
    int counts[kMaxCluster + 1];
    max_active_clusters(kernel, NT, most, done_occ, cache, counts);
    if (counts[ctas] < 1) ctas = 8;
  }
  return launch_pdl(kernel, ctas, NT, static_cast<int>(smem), s, ctas, args) == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

// At most 256 sequences and items (one a thread): one CTA of 256 threads, whose
// launch and barriers are shorter (32 sequences of one token 3.6 -> 3.2 us; with
// several items a thread it loses: 1000 tokens 4.2 -> 6.5). Else CTAs of 1024
// for the `items` dealt out to the threads: more than one costs a cluster launch
// and barrier, more than eight a place for 16 CTAs (32768 tokens 7.3 -> 5.9 us,
// 262144 released blocks 12.2 -> 8.7 against eight; other boxes 6.5 and 9.2).
bool few_items(int B, long long items) { return B <= 256 && items <= 256; }
int table_ctas(long long items) { return items <= 1024 ? 1 : items <= 8 * 1024 ? 8 : 16; }

template <class Args>
pd_status launch_build(const Args& a, size_t smem, cudaStream_t s) {
  if (few_items(a.B, a.T)) return launch_cluster<256>(build_tables_kernel<256>, 1, smem, s, a);
  return launch_cluster<1024>(build_tables_kernel<1024>, table_ctas(a.T), smem, s, a);
}
template <class Args>
pd_status launch_release(const Args& a, long long blocks, size_t smem, cudaStream_t s) {
  if (few_items(a.B, blocks)) return launch_cluster<256>(release_kernel<256>, 1, smem, s, a);
  return launch_cluster<1024>(release_kernel<1024>, table_ctas(blocks), smem, s, a);
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" pd_status build_block_tables(const int32_t* context_lens, const int32_t* query_lens, int num_tokens,
                                        int32_t* block_table, const int32_t* free_blocks, const int32_t* free_count,
                                        int32_t* free_count_out, int32_t* seq_lens, int32_t* query_start_loc,
                                        int64_t* slot_mapping, int32_t* positions, const pd_dims* dims,
                                        uint32_t* error_flag, void* stream) {
  const pd_status st = check_table_dims(dims);
  if (st != PD_OK) return st;
  if (num_tokens < 0) return PD_ERR_SHAPE;
  const pd_dims& d = *dims;
  if (!free_count || !free_count_out || !query_start_loc) return PD_ERR_NULL;
  if (d.B > 0 && (!context_lens || !query_lens || !seq_lens)) return PD_ERR_NULL;
  if (d.B > 0 && d.max_blocks_per_seq > 0 && !block_table) return PD_ERR_NULL;
  if (d.num_blocks > 0 && !free_blocks) return PD_ERR_NULL;
  if (num_tokens > 0 && !slot_mapping) return PD_ERR_NULL;
  if (misaligned(context_lens, 3) || misaligned(query_lens, 3) || misaligned(block_table, 3) ||
      misaligned(free_blocks, 3) || misaligned(free_count, 3) || misaligned(free_count_out, 3) ||
      misaligned(seq_lens, 3) || misaligned(query_start_loc, 3) || misaligned(slot_mapping, 7) ||
      misaligned(positions, 3) || misaligned(error_flag, 3))
    return PD_ERR_ALIGN;
  TableArgs a{context_lens, query_lens, block_table, free_blocks, free_count, free_count_out, seq_lens,
              query_start_loc, slot_mapping, positions, error_flag, d.B, num_tokens, d.block_size, d.num_blocks,
              d.max_blocks_per_seq};
  return launch_build(a, (3 * static_cast<size_t>(d.B) + 2) * 4, static_cast<cudaStream_t>(stream));
}

extern "C" pd_status release_blocks(const int32_t* block_table, const int32_t* seq_lens, const uint8_t* released,
                                    int32_t* free_blocks, const int32_t* free_count, int32_t* free_count_out,
                                    int32_t* seq_lens_out, const pd_dims* dims, uint32_t* error_flag, void* stream) {
  const pd_status st = check_table_dims(dims);
  if (st != PD_OK) return st;
  const pd_dims& d = *dims;
  if (!free_count || !free_count_out) return PD_ERR_NULL;
  if (d.B > 0 && (!seq_lens || !released || !seq_lens_out)) return PD_ERR_NULL;
  if (d.B > 0 && d.max_blocks_per_seq > 0 && !block_table) return PD_ERR_NULL;
  if (d.num_blocks > 0 && !free_blocks) return PD_ERR_NULL;
  if (misaligned(block_table, 3) || misaligned(seq_lens, 3) || misaligned(free_blocks, 3) ||
      misaligned(free_count, 3) || misaligned(free_count_out, 3) || misaligned(seq_lens_out, 3) ||
      misaligned(error_flag, 3))
    return PD_ERR_ALIGN;
  ReleaseArgs a{block_table, seq_lens, released, free_blocks, free_count, free_count_out, seq_lens_out, error_flag,
                d.B, d.block_size, d.num_blocks, d.max_blocks_per_seq};
  const long long blocks = static_cast<long long>(d.B) * d.max_blocks_per_seq;
  return launch_release(a, blocks, (2 * static_cast<size_t>(d.B) + 1) * 4, static_cast<cudaStream_t>(stream));
}
