// pdecode_api.cu -- host side of libpdecode: argument validation, the split
// plan, TMA descriptors for the paged caches, and launches on the caller's
// stream. The C ABI is declared in include/pdecode.h.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <atomic>
#include <mutex>

#include "diff_launch.h"
#include "launch.h"
#include "pdecode.h"
#include "scored_launch.h"

namespace pd {

bool kernel_shape(int D, int kv, int nt, int grouped, KernelShape* out) {
  if (kv == kKvBf16)
    return D == 128 ? shape_bf16_d128(nt, grouped, out)
                    : D == 256 && shape_bf16_d256(nt, grouped, out);
  if (kv == kKvFp8Bq)
    return D == 128 ? shape_fp8q_d128(nt, grouped, out) : D == 256 && shape_fp8q_d256(nt, grouped, out);
  if (kv == kKvInt8Bq)
    return D == 128 ? shape_i8q_d128(nt, grouped, out) : D == 256 && shape_i8q_d256(nt, grouped, out);
  if (D == 128)
    return kv == kKvFp8 ? shape_fp8_d128(nt, grouped, out) : kv == kKvInt8 ? shape_i8_d128(nt, grouped, out)
                                                                      : shape_f16_d128(nt, grouped, out);
  if (D == 256)
    return kv == kKvFp8 ? shape_fp8_d256(nt, grouped, out) : kv == kKvInt8 ? shape_i8_d256(nt, grouped, out)
                                                                      : shape_f16_d256(nt, grouped, out);
  return false;
}

cudaError_t launch_decode(int D, int kv, int nt, int grouped, const CUtensorMap& tk,
                          const CUtensorMap& tv, const DecodeParams& p, int grid, cudaStream_t s) {
  if (kv == kKvBf16)
    return D == 128 ? launch_bf16_d128(nt, grouped, tk, tv, p, grid, s)
                    : launch_bf16_d256(nt, grouped, tk, tv, p, grid, s);
  if (kv == kKvFp8Bq)
    return D == 128 ? launch_fp8q_d128(nt, grouped, tk, tv, p, grid, s)
                    : launch_fp8q_d256(nt, grouped, tk, tv, p, grid, s);
  if (kv == kKvInt8Bq)
    return D == 128 ? launch_i8q_d128(nt, grouped, tk, tv, p, grid, s)
                    : launch_i8q_d256(nt, grouped, tk, tv, p, grid, s);
  if (D == 128)
    return kv == kKvFp8 ? launch_fp8_d128(nt, grouped, tk, tv, p, grid, s)
           : kv == kKvInt8 ? launch_i8_d128(nt, grouped, tk, tv, p, grid, s)
                           : launch_f16_d128(nt, grouped, tk, tv, p, grid, s);
  return kv == kKvFp8 ? launch_fp8_d256(nt, grouped, tk, tv, p, grid, s)
         : kv == kKvInt8 ? launch_i8_d256(nt, grouped, tk, tv, p, grid, s)
                         : launch_f16_d256(nt, grouped, tk, tv, p, grid, s);
}

std::mutex& workspace_mutex(const void* workspace) {
  static std::mutex locks[61];
  return locks[(reinterpret_cast<uintptr_t>(workspace) >> 8) % 61];
}

namespace {

constexpr unsigned long long kTimeoutNs = 2000000000ull;  // 2 s per pipeline wait (default)
std::atomic<unsigned long long> g_wait_limit_ns{kTimeoutNs};
std::atomic<int> g_inject{0};

// Which decode a plan is for: their kernels' shapes differ.
enum class Op { kPlain, kDiff, kScored };

// Resolved work decomposition of one call.
struct Plan {
  int splits;       // 0 = balanced, >= 1 fixed
  int grid;         // CTAs launched
  int nt;           // row tiles per head
  int hg;           // KV heads per tile
  long long slots;  // partial slots in the workspace
  long long n_merge; // units the split combine visits
  long long units;  // B * Hkv / hg work units
  int rows_padded;
  int unit_cost;    // balanced split: virtual tiles per unit start
  bool whole_tile;  // a TMA box is a tile of all slabs
  int cluster;      // > 1: the fixed split's pieces of a unit form a cluster that merges them
  int sms;          // SMs of the device the plan was made for
  int head_tiles;   // row tiles of a head in a partial
  int least;        // scored decode: tiles of a fixed split's piece at least
  size_t off_ml, off_o, bytes;  // workspace layout
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Caches of one-byte codes (e4m3fn or int8, with an fp16 or a bfloat16 q).
bool byte_kind(int kv) {
  return kv == PD_KV_FP8_E4M3 || kv == PD_KV_INT8 || kv == PD_KV_FP8_E4M3_BF16 || kv == PD_KV_INT8_BF16;
}
bool fp4_kind(int kv) { return kv == PD_KV_FP4 || kv == PD_KV_FP4_BF16; }
// q and out (and a writer's new tokens) in bfloat16.
bool bf16_io(int kv) {
  return kv == PD_KV_BF16 || kv == PD_KV_FP8_E4M3_BF16 || kv == PD_KV_INT8_BF16 || kv == PD_KV_FP4_BF16;
}

pd_status check_dims(const pd_dims* d, int qlen, Op op = Op::kPlain) {
  if (!d) return PD_ERR_NULL;
  if (d->B < 0 || d->Hq < 1 || d->Hkv < 1 || d->D < 1 || d->block_size < 1 || d->num_blocks < 0 ||
      d->max_blocks_per_seq < 0 || qlen < 1)
    return PD_ERR_SHAPE;
  if (d->Hq % d->Hkv != 0) return PD_ERR_SHAPE;
  const bool fp4 = op == Op::kScored && fp4_kind(d->kv_dtype);
  if (d->kv_dtype != PD_KV_F16 && d->kv_dtype != PD_KV_BF16 && !byte_kind(d->kv_dtype) && !fp4)
    return PD_ERR_DTYPE;
  if ((byte_kind(d->kv_dtype) || fp4) && (!std::isfinite(d->k_scale) || !std::isfinite(d->v_scale)))
    return PD_ERR_SHAPE;
  if (d->D != 128 && d->D != 256) return PD_ERR_UNSUPPORTED;
  if (d->block_size % kTileKeys != 0) return PD_ERR_UNSUPPORTED;
  if (qlen > 8) return PD_ERR_UNSUPPORTED;
  const int R = d->Hq / d->Hkv * qlen;
  if (R > 32) return PD_ERR_UNSUPPORTED;
  // 32-bit index headroom: tiles, keys and cache rows
  const long long cap_keys = static_cast<long long>(d->max_blocks_per_seq) * d->block_size;
  if (cap_keys > (1ll << 30)) return PD_ERR_UNSUPPORTED;
  if (static_cast<long long>(d->B) * d->Hkv * (cap_keys / kTileKeys + 1 + 64) > (1ll << 31) - 1)
    return PD_ERR_UNSUPPORTED;
  if (static_cast<long long>(d->num_blocks) * d->block_size > (1ll << 31) - 1) return PD_ERR_UNSUPPORTED;
  if (fp4 && static_cast<long long>(d->num_blocks) * d->block_size * d->Hkv > (1ll << 31) - 1)
    return PD_ERR_UNSUPPORTED;  // its rows are (key, head) pairs
  if (static_cast<long long>(d->B) * qlen * d->Hq > (1ll << 31) - 1) return PD_ERR_UNSUPPORTED;
  return PD_OK;
}

int device_sm_count(int sm_count) {
  if (sm_count > 0) return sm_count;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

// Automatic split (num_splits = 0): balanced over every resident CTA slot,
// except when the units are few (<= a quarter of the CTA slots) and either
// their work is small (at most 24 visible tiles per CTA slot, from the table
// capacity and the window: latency-bound, where each piece's fixed cost and
// the combine's fan-in dominate) or the kernel's pieces carry a large fixed
// cost (the tensor-memory kernels, KernelShape::fixed_pieces): then a fixed
// split of each unit into
// floor(0.84 CTA slots / units) chunks, one per CTA, which leaves about a
// sixth of the SMs idle but gives every CTA one piece. Measured on GB300
// (D=256 GQA 6:1, L=4096): B = 1 / 2 / 3 12.9 / 16.1 / 19.2 -> 12.0 / 15.0 /
// 18.0 us; windowed L=32768 B = 1 / 2 12.8 / 15.8 -> 12.0 / 14.9 us; qlen=3
// e4m3 verify B=8 39.8 -> 36.0 us; shapes with more work per CTA (B >= 8 at
// L=4096, L=32768 without a window) stay balanced: there the two splits are
// within ~2 % or the fixed one loses (B=16: +1.0 us, 2 x 2048 tiles: +0.5). The
// workspace is sized for the balanced split in either case (the fixed split
// needs fewer slots), so pd_workspace_bytes does not depend on the window.
// The differential decode's kernels hold two maps' rows. How many keys `prefixes` add to a
// window is known on the device alone: a fixed split then has as many pieces as
// the table's capacity could need, and the device makes pieces of Plan::least tiles or more of
// the keys that there are. (24 x 4 heads, D = 256, B = 1, L = 8192; planned by the window alone -> so:
// window 16, prefix 8000, fp16 / 4-bit / e4m3 with qlen = 3 343 / 91 / 84 -> 12.4 / 11.6 / 15.4 us; window
// 256, prefix 4, a table of 131072 keys 11.1 / 8.3 / 12.1 -> 11.7 / 9.0 / 13.5; window 4096, prefix 128,
// 4-bit, B = 4 13.9 both ways.)
pd_status make_plan(const pd_dims* d, int qlen, int num_splits, int sm_count, Plan* pl, int window = 0,
                    Op op = Op::kPlain, bool prefixes = false) {
  const bool diff = op == Op::kDiff;
  pd_status st = check_dims(d, qlen, op);
  if (st != PD_OK) return st;
  if (num_splits < 0) return PD_ERR_SHAPE;
  const int sms = device_sm_count(sm_count);
  if (sms <= 0) return PD_ERR_CUDA;
  pl->sms = sms;
  const int R = d->Hq / d->Hkv * qlen;
  pl->nt = (R + 7) / 8;
  KernelShape ks;
  // tiles of several KV heads read the cache contiguously; they serve the
  // single-row-tile shapes whose head count is a multiple of four (the
  // instantiation chooses how many heads a tile holds: 2 or 4)
  const bool grouped = pl->nt == 1 && d->Hkv % 4 == 0;
  const auto shape = diff ? diff_kernel_shape : op == Op::kScored ? scored_kernel_shape : kernel_shape;
  if (!(grouped && shape(d->D, d->kv_dtype, pl->nt, 1, &ks)) && !shape(d->D, d->kv_dtype, pl->nt, 0, &ks))
    return PD_ERR_UNSUPPORTED;
  pl->hg = ks.heads;
  pl->rows_padded = ks.rows_padded;
  pl->head_tiles = ks.rows_padded / ks.heads / 8;
  pl->unit_cost = ks.unit_cost;
  pl->whole_tile = ks.whole_tile != 0;
  pl->units = static_cast<long long>(d->B) * (d->Hkv / pl->hg);
  int splits = num_splits;
  if (splits == 0 && d->B > kMaxAutoB) splits = 1;  // plenty of units: one piece each
  const int ctas = sms * ks.ctas_per_sm;  // persistent grid: every resident CTA slot
  const bool automatic = splits == 0;
  const long long cap_keys = static_cast<long long>(d->max_blocks_per_seq) * d->block_size;
  const long long vis_keys = window > 0 ? std::min<long long>(cap_keys, 0ll + window + qlen + kTileKeys) : cap_keys;
  // Short tables: whole units, one per CTA, walk (waves - units / ctas) * tiles more
  // than the balanced split does, but launch no join and end no pieces inside a
  // unit, which costs four steps of the CTA and up to twice that where every CTA
  // has such ends. Balanced -> whole: fp16 D = 256, 48 units, 1 / 4 / 8 tiles 9.2 /
  // 12.2 / 13.5 -> 6.9 / 9.1 / 12.4 us; three key groups, 2 units, 8 / 16 tiles 8.3 /
  // 8.3 -> 7.2 / 8.7; tensor-memory engine (steps of 8 tiles), 4 / 64 / 384 units, 16
  // tiles 12.6 / 18.5 / 44.4 -> 11.3 / 11.8 / 33.3, 64 tiles 16.1 / 25.6 / 72.6 ->
  // 19.1 / 19.6 / 59.5. Eight steps at most: a batch with one long sequence then
  // waits four steps longer. Where pieces merge inside a cluster, as many of two steps
  // or more as the CTAs hold are better still (4 / 32 / 64 units, 48 tiles 16.7 / 16.8
  // / 17.1 -> 13.4 / 13.8 / 15.4). A step is as many tiles as the CTA takes at once,
  // two per key group where a warp takes two (D = 128, 32 x 8 heads, B = 76, 12 / 16 tiles
  // balanced 25.9 / 28.6 -> 18.1 / 20.9, three row tiles, B = 38, 24 / 32 tiles 26.5 / 29.6
  // -> 21.7 / 24.7); for few units, whose other plan is the fixed split below with pieces
  // that end early, one per key group (B = 1, 12 tiles 11.8, whole 14.2).
  if (automatic && diff && pl->units > 0) {
    const long long waves = (pl->units + ctas - 1) / ctas;
    const long long tiles = (vis_keys + kTileKeys - 1) / kTileKeys;
    const int step = pl->units <= ctas / 4 ? ks.key_groups : ks.step_tiles;
    const long long room = std::min<long long>({ctas / pl->units, tiles / (2 * step), kMaxCluster});
    if (tiles <= 8 * step) {
      if (room >= 2 && ks.max_clusters[room] >= pl->units)
        splits = static_cast<int>(room);
      else if (tiles * (waves * ctas - pl->units) <= 4ll * step * (ctas + pl->units))
        splits = 1;
    }
  }
  pl->least = 1;
  if (splits == 0 && pl->units > 0 && pl->units <= ctas / 4) {
    const long long tiles = pl->units * (vis_keys / kTileKeys + 1);
    if (tiles <= 24ll * ctas || ks.fixed_pieces)
      splits = static_cast<int>(std::max<long long>(1, (ctas * 27 / 32) / pl->units));
    // the differential decode's join reads two maps' partials: pieces of at least four tiles (B = 1, L
    // = 4096, fp16 / e4m3: 13.9 / 13.6 -> 12.4 / 12.3 us; eight tiles 13.3 / 13.9), of
    // two steps on the tensor-memory engine (qlen = 3, e4m3, L = 1024 / 2048: 16.1 /
    // 15.5 -> 13.2 / 14.0). The scored decode's too (B = 1, L = 4096, 24 x 4 heads, D = 256 11.2 -> 10.1 us,
    // 8 x 1 heads, D = 128 11.0 -> 8.8; L = 1024 8.8 -> 9.3 and 8.6 -> 8.3), there of a block of eight
    // (qlen = 3, e4m3, L = 1024 14.9 -> 12.4, 8 x 1 heads, D = 128, L = 4096 15.8 -> 11.2; two blocks 12.3 and 12.2)
    const long long piece = !ks.fixed_pieces ? 4 : diff ? 2 * ks.step_tiles : 8;
    const long long most = ((prefixes ? cap_keys : vis_keys) / kTileKeys + piece - 1) / piece;
    if (op != Op::kPlain && splits > 1) splits = static_cast<int>(std::max<long long>(1, std::min<long long>(splits, most)));
    if (prefixes && vis_keys < cap_keys) pl->least = static_cast<int>(piece);
  }
  pl->splits = splits;
  if (splits == 0) {
    pl->grid = ctas;
    pl->slots = 2ll * ctas;  // a CTA's range holds at most two split pieces
    pl->n_merge = pl->units;
  } else {
    const long long pieces = pl->units * splits;
    pl->grid = static_cast<int>(pieces < ctas ? (pieces > 0 ? pieces : 1) : ctas);
    pl->slots = splits > 1 ? pieces : 0;
    pl->n_merge = splits > 1 ? pl->units : 0;
  }
  // an automatic plan sizes its workspace for the balanced split, whichever
  // split it chose (so the size does not depend on the window)
  const long long ws_slots = automatic && d->B <= kMaxAutoB ? 2ll * ctas : pl->slots;
  if (pl->slots == 0 && ws_slots == 0) {
    pl->off_ml = pl->off_o = pl->bytes = 0;
  } else {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t ml = up(static_cast<size_t>(ws_slots) * pl->rows_padded * 2 * 4);
    const size_t o = static_cast<size_t>(ws_slots) * pl->rows_padded * d->D * 4;
    pl->off_ml = 0;
    pl->off_o = ml;
    pl->bytes = ml + o;
  }
  // A fixed split of at most kMaxCluster pieces per unit, one CTA each, on a kernel
  // that merges a unit's pieces inside its thread-block cluster (distributed
  // shared memory), when the device runs every unit's cluster at once: no
  // split-combine launch. (The workspace keeps the size computed above, so it
  // does not depend on the device's cluster occupancy.)
  pl->cluster = 0;
  if (splits >= 2 && splits <= kMaxCluster && pl->units * splits == pl->grid &&
      ks.max_clusters[splits] >= pl->units) {
    pl->cluster = splits;
    pl->n_merge = 0;
  }
  return PD_OK;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

}  // namespace

// cuCtxGetCurrent and cuCtxGetId through the runtime's driver entry points.
unsigned long long current_context_id() {
  static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
  });
  if (!get_current || !get_id) return 0;
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (get_current(&ctx) != CUDA_SUCCESS || ctx == nullptr) return 0;
  if (get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

namespace {

// Map over a paged cache viewed as [num_blocks*block_size][Hkv][D], 128-byte
// swizzled. The decode's is 3-D, a box being 128 bytes of D x hg heads x 16
// keys; the differential decode's 4-D: 128 bytes x 16 keys x hg heads x all
// D * elem / 128 slabs, a whole tile in one box.
bool encode_cache_map(CUtensorMap* m, const void* base, const pd_dims* d, int hg, bool whole_tile) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool byte = byte_kind(d->kv_dtype);
  const cuuint64_t elem = byte ? 1 : 2;
  const cuuint64_t rows = static_cast<cuuint64_t>(d->num_blocks) * d->block_size;
  const cuuint64_t keys = rows > 0 ? rows : 1, heads = static_cast<cuuint64_t>(d->Hkv);
  const cuuint64_t slab = 128 / elem, slabs = d->D / slab;
  const cuuint64_t head_bytes = d->D * elem, key_bytes = heads * head_bytes;
  const cuuint32_t tk = static_cast<cuuint32_t>(kTileKeys), th = static_cast<cuuint32_t>(hg);
  cuuint64_t dims3[3] = {static_cast<cuuint64_t>(d->D), heads, keys}, strides3[2] = {head_bytes, key_bytes};
  cuuint32_t box3[3] = {static_cast<cuuint32_t>(slab), th, tk};
  cuuint64_t dims4[4] = {slab, keys, heads, slabs}, strides4[3] = {key_bytes, head_bytes, 128};
  cuuint32_t box4[4] = {static_cast<cuuint32_t>(slab), tk, th, static_cast<cuuint32_t>(slabs)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = byte ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : d->kv_dtype == PD_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  CUresult r = fn(m, type, whole_tile ? 4 : 3, const_cast<void*>(base), whole_tile ? dims4 : dims3,
                  whole_tile ? strides4 : strides3, whole_tile ? box4 : box3, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" {

void pd_set_wait_limit_ns(unsigned long long ns) {
  g_wait_limit_ns.store(ns ? ns : kTimeoutNs, std::memory_order_relaxed);
}

void pd_set_fault_injection(int mode) { g_inject.store(mode == 1 ? 1 : 0, std::memory_order_relaxed); }

const char* pd_status_str(pd_status s) {
  switch (s) {
    case PD_OK: return "ok";
    case PD_ERR_NULL: return "a required pointer is NULL";
    case PD_ERR_SHAPE: return "inconsistent or out-of-range sizes";
    case PD_ERR_DTYPE: return "unknown KV dtype";
    case PD_ERR_UNSUPPORTED: return "shape not implemented by these kernels";
    case PD_ERR_ALIGN: return "pointer not 16-byte aligned";
    case PD_ERR_WORKSPACE: return "workspace missing or too small";
    case PD_ERR_CUDA: return "CUDA runtime error";
  }
  return "unknown status";
}

size_t pd_workspace_bytes(const pd_dims* dims, int qlen, int num_splits, int sm_count) {
  Plan pl;
  if (make_plan(dims, qlen, num_splits, sm_count, &pl) != PD_OK) return 0;
  return pl.bytes;
}

size_t pd_diff_workspace_bytes(const pd_dims* dims, int qlen, int num_splits, int sm_count) {
  Plan pl;
  if (make_plan(dims, qlen, num_splits, sm_count, &pl, 0, Op::kDiff) != PD_OK) return 0;
  return pl.bytes;
}

int pd_grid_ctas(const pd_dims* dims, int qlen, int num_splits, int sm_count) {
  Plan pl;
  if (make_plan(dims, qlen, num_splits, sm_count, &pl) != PD_OK) return 0;
  return pl.grid;
}

}  // extern "C"

namespace {

// What every decode call checks and fills in: the plan, the caches' maps and
// the kernel's parameters. `ready` is
// false when there is nothing to launch. prefixes: keys beside the window's may be visible. q_start null means B sequences of qlen
// query tokens each (total_q = B * qlen); otherwise sequence b owns rows
// [q_start[b], q_start[b+1]) of q and out, at most qlen of them.
pd_status prepare_decode(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_start,
                         int total_q, float scale, int window, int qlen, int num_splits, void* out,
                         const pd_dims* dims, void* workspace, size_t workspace_bytes,
                         uint32_t* error_flag, Op op, bool prefixes, Plan& pl, CUtensorMap& tk, CUtensorMap& tv,
                         DecodeParams& p, bool& ready) {
  ready = false;
  pd_status st = check_dims(dims, qlen, op);
  if (st != PD_OK) return st;
  if (num_splits < 0 || !std::isfinite(scale)) return PD_ERR_SHAPE;
  if (total_q < 0 || static_cast<long long>(total_q) * dims->Hq > (1ll << 31) - 1)
    return q_start ? PD_ERR_SHAPE : PD_ERR_UNSUPPORTED;
  if (dims->B == 0 || total_q == 0) return PD_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out) return PD_ERR_NULL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(block_table) & 3u) || (reinterpret_cast<uintptr_t>(seq_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(q_start) & 3u) || (reinterpret_cast<uintptr_t>(error_flag) & 3u))
    return PD_ERR_ALIGN;
  if (dims->num_blocks == 0) return PD_ERR_SHAPE;
  st = make_plan(dims, qlen, num_splits, 0, &pl, window, op, prefixes);
  if (st != PD_OK) return st;
  if (pl.bytes > 0) {
    if (!workspace || workspace_bytes < pl.bytes) return PD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PD_ERR_ALIGN;
  }

  const bool fp4 = fp4_kind(dims->kv_dtype);
  if (fp4) {
    tk = tv = CUtensorMap{};  // its kernels copy without maps
  } else if (!encode_cache_map(&tk, k_cache, dims, pl.hg, pl.whole_tile) ||
             !encode_cache_map(&tv, v_cache, dims, pl.hg, pl.whole_tile)) {
    return PD_ERR_CUDA;
  }

  const bool fp8 = byte_kind(dims->kv_dtype) || fp4;  // scaled codes
  p.q = static_cast<const __half*>(q);
  p.out = static_cast<__half*>(out);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.q_start = q_start;
  p.total_q = total_q;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.n_merge = static_cast<int>(pl.n_merge);
  p.decode_grid = pl.grid;
  p.rows_padded = pl.rows_padded;
  p.ws_ml = pl.bytes ? reinterpret_cast<float*>(ws + pl.off_ml) : nullptr;
  p.ws_o = pl.bytes ? reinterpret_cast<float*>(ws + pl.off_o) : nullptr;
  p.error_flag = error_flag;
  p.B = dims->B;
  p.qlen = qlen;
  p.Hq = dims->Hq;
  p.Hkv = dims->Hkv;
  p.G = dims->Hq / dims->Hkv;
  p.R = p.G * qlen;
  p.hg = pl.hg;
  p.hgn = dims->Hkv / pl.hg;
  p.rows_head = pl.rows_padded / pl.hg;
  p.max_blocks = dims->max_blocks_per_seq;
  p.block_size = dims->block_size;
  p.num_blocks = dims->num_blocks;
  p.tiles_per_block = dims->block_size / kTileKeys;
  // a window that no sequence can fill is none (and positions less a window stay in 32 bits)
  const long long cap_keys = static_cast<long long>(dims->max_blocks_per_seq) * dims->block_size;
  p.window = window > 0 && window < cap_keys ? window : 0;
  p.num_splits = pl.splits;
  p.unit_cost = pl.unit_cost;
  const double ks = fp8 ? static_cast<double>(dims->k_scale) : 1.0;
  p.sl2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634 * ks);
  p.out_scale = fp8 ? dims->v_scale : 1.0f;
  p.out_bf16 = bf16_io(dims->kv_dtype) ? 1 : 0;
  p.timeout_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.inject = g_inject.load(std::memory_order_relaxed);
  p.cluster = pl.cluster;

  ready = true;
  return PD_OK;
}

// How a split combine is launched: CTAs that a unit head's dims are spread over, pieces loaded
// at a time, threads.
struct CombineShape {
  int chunks, batch, threads;
};
CombineShape combine_shape(const Plan& pl, int D, int R) {
  // pieces per split unit: about grid / units + 1 (balanced) or S (fixed);
  // many pieces -> spread a unit's dims over CTAs so threads can share pieces,
  // but keep the combine grid within one CTA per SM: those CTAs are resident
  // beside the decode grid and do their pre-wait work (the unit's piece
  // layout) while it runs, where CTAs beyond that start only as decode CTAs
  // exit and add that work to the tail (measured on GB300, D=256 GQA 6:1:
  // B = 2 / 3 / 8 15.0 / 17.6 / 28.9 -> 13.9 / 16.7 / 28.6 us, e4m3 B = 32
  // 54.1 -> 52.5, L = 32768 B = 2 47.2 -> 45.8, windowed B = 2 14.7 ->
  // 13.7; D=128 (28,4) ragged 86.5 -> 87.0; B = 1 and B = 32 unchanged)
  const long long per_unit = pl.splits == 0 ? pl.grid / (pl.units > 0 ? pl.units : 1) + 1 : pl.splits;
  int chunks = per_unit >= 16 ? D / 8 : per_unit >= 4 ? D / 32 : 1;
  while (chunks > 1 && pl.n_merge * chunks * pl.hg > pl.sms) chunks >>= 1;
  // units of more than four pieces: the combine that loads eight pieces'
  // partials at a time (one L2 round trip for up to eight), else the one
  // of four, which needs fewer registers (measured on GB300, D=256 GQA 6:1:
  // e4m3 B = 32 52.3 -> 50.8 us, B = 8 28.2 -> 27.9, B = 3 16.6 -> 16.4 with
  // eight; the headline's ~3.4 pieces per unit 0.3 us slower with eight)
  const int batch = per_unit > 4 ? 8 : 4;
  // a CTA's items (row, 4 dims) beyond 256: the batch-8 kernel's 512-thread
  // form gives each thread one item (e4m3 / int8 B = 32: 384 items)
  const long long items = static_cast<long long>(R) * (D / chunks / 4);
  const int threads = items > 256 ? 512 : 256;
  return {chunks, batch, threads};
}

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// Workspace of a scored decode that sums its keys' weights: the split partials, the rows' (m, l), and
// the scores of every key of the table (16 keys x 8 rows for each tile and row tile).
struct ScoredLayout {
  size_t off_ml, off_scores, bytes;
};
ScoredLayout scored_layout(const pd_dims& d, const Plan& pl, int qlen) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  ScoredLayout l;
  l.off_ml = up(pl.bytes);
  l.off_scores = l.off_ml + up(static_cast<size_t>(d.B) * qlen * d.Hq * 8);
  const size_t tiles = static_cast<size_t>(d.max_blocks_per_seq) * (d.block_size / kTileKeys);
  l.bytes = l.off_scores + static_cast<size_t>(d.B) * d.Hkv * tiles * pl.head_tiles * 512;
  return l;
}

pd_status decode_impl(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_start,
                      int total_q, float scale, int window, int qlen, int num_splits, void* out,
                      const pd_dims* dims, void* workspace, size_t workspace_bytes,
                      uint32_t* error_flag, void* stream) {
  Plan pl;
  CUtensorMap tk, tv;
  DecodeParams p;
  bool ready;
  const pd_status st = prepare_decode(q, k_cache, v_cache, block_table, seq_lens, q_start, total_q, scale, window, qlen,
                                      num_splits, out, dims, workspace, workspace_bytes, error_flag, Op::kPlain,
                                      false, pl, tk, tv, p, ready);
  if (st != PD_OK || !ready) return st;
  const WorkspaceLock lock(workspace, pl.n_merge > 0);
  cudaError_t e = launch_decode(dims->D, dims->kv_dtype, pl.nt, pl.hg > 1 ? 1 : 0, tk, tv, p, pl.grid,
                                static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess && pl.n_merge > 0) {
    const CombineShape c = combine_shape(pl, dims->D, p.R);
    e = launch_split_combine(dims->D, p, static_cast<int>(pl.n_merge), c.chunks, c.batch, c.threads,
                             static_cast<cudaStream_t>(stream));
  }
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // namespace

extern "C" {

pd_status decode_paged(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* seq_lens, float scale,
                       int window, int qlen, int num_splits, void* out, const pd_dims* dims,
                       void* workspace, size_t workspace_bytes, uint32_t* error_flag,
                       void* stream) {
  if (!dims) return PD_ERR_NULL;
  const long long total = static_cast<long long>(dims->B) * (qlen > 0 ? qlen : 0);
  if (total > (1ll << 31) - 1) return PD_ERR_UNSUPPORTED;
  return decode_impl(q, k_cache, v_cache, block_table, seq_lens, nullptr, static_cast<int>(total),
                     scale, window, qlen, num_splits, out, dims, workspace, workspace_bytes,
                     error_flag, stream);
}

pd_status decode_paged_varlen(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, const int32_t* seq_lens,
                              const int32_t* query_start_loc, int num_query_tokens, int max_qlen,
                              float scale, int window, int num_splits, void* out,
                              const pd_dims* dims, void* workspace, size_t workspace_bytes,
                              uint32_t* error_flag, void* stream) {
  if (!dims) return PD_ERR_NULL;
  if (dims->B > 0 && num_query_tokens > 0 && !query_start_loc) return PD_ERR_NULL;
  return decode_impl(q, k_cache, v_cache, block_table, seq_lens, query_start_loc,
                     num_query_tokens, scale, window, max_qlen, num_splits, out, dims, workspace,
                     workspace_bytes, error_flag, stream);
}

pd_status decode_paged_diff(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                            const int32_t* seq_lens, const int32_t* query_start_loc, int num_query_tokens,
                            const float* lambda, float scale, int window, int qlen, int num_splits,
                            const void* norm_weight, int norm_weight_f32, float norm_eps, float norm_gain, void* out,
                            const pd_dims* dims, void* workspace, size_t workspace_bytes, uint32_t* error_flag,
                            void* stream) {
  if (!dims) return PD_ERR_NULL;
  long long total = num_query_tokens;
  if (!query_start_loc) {
    total = static_cast<long long>(dims->B) * (qlen > 0 ? qlen : 0);
    if (total > (1ll << 31) - 1) return PD_ERR_UNSUPPORTED;
  }
  if (norm_weight && (!(norm_eps >= 0.f) || !std::isfinite(norm_eps) || !std::isfinite(norm_gain))) return PD_ERR_SHAPE;
  if (dims->B > 0 && total > 0) {
    if (!lambda) return PD_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(lambda) & 3u) ||
        (reinterpret_cast<uintptr_t>(norm_weight) & (norm_weight_f32 ? 3u : 1u)))
      return PD_ERR_ALIGN;
  }
  Plan pl;
  CUtensorMap tk, tv;
  DiffParams p;
  bool ready;
  const pd_status st = prepare_decode(q, k_cache, v_cache, block_table, seq_lens, query_start_loc,
                                      static_cast<int>(total), scale, window, qlen, num_splits, out, dims, workspace,
                                      workspace_bytes, error_flag, Op::kDiff, false, pl, tk, tv, p.d, ready);
  if (st != PD_OK || !ready) return st;
  p.v_cache = v_cache;
  p.lambda = lambda;
  p.norm_weight = norm_weight;
  p.norm_f32 = norm_weight_f32 ? 1 : 0;
  p.norm_eps = norm_eps;
  p.norm_gain = norm_gain;
  auto s = static_cast<cudaStream_t>(stream);
  const WorkspaceLock lock(workspace, pl.n_merge > 0);
  cudaError_t e = launch_diff(dims->D, dims->kv_dtype, pl.nt, pl.hg > 1 ? 1 : 0, tk, tv, p, pl.grid, s);
  if (e == cudaSuccess && pl.n_merge > 0) {
    // rows of a unit's head spread over CTAs while the grid stays within one
    // CTA per SM. A CTA takes all its rows at once where its threads suffice;
    // what is left of them share a row's pieces. Units of many pieces (few
    // units: SMs stand free) take the join of 1024 threads.
    const long long per_unit = pl.splits == 0 ? pl.grid / (pl.units > 0 ? pl.units : 1) + 1 : pl.splits;
    int chunks = p.d.R;
    while (chunks > 1 && pl.n_merge * chunks * pl.hg > pl.sms) chunks = (chunks + 1) / 2;
    const bool many = per_unit > 12;
    const int slots = (many ? kJoinThreadsMany : kJoinThreads) / (dims->D / 4);  // (row, piece group) places
    const int rows = std::min((p.d.R + chunks - 1) / chunks, slots);
    const int groups = static_cast<int>(std::min<long long>(slots / rows, per_unit));
    e = launch_diff_combine(dims->D, p, static_cast<int>(pl.n_merge), chunks, rows, groups, many, s);
  }
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

size_t pd_scored_workspace_bytes(const pd_dims* dims, int qlen, int num_splits, int key_weights, int sm_count) {
  Plan pl;
  if (make_plan(dims, qlen, num_splits, sm_count, &pl, 0, Op::kScored) != PD_OK) return 0;
  return key_weights ? scored_layout(*dims, pl, qlen).bytes : pl.bytes;
}

pd_status decode_paged_scored(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                              const int32_t* seq_lens, const int32_t* query_start_loc, int num_query_tokens, float scale,
                              int window, int qlen, int num_splits, const pd_score* score, void* out,
                              const pd_dims* dims, void* workspace, size_t workspace_bytes, uint32_t* error_flag,
                              void* stream) {
  if (!dims || !score) return PD_ERR_NULL;
  long long total = num_query_tokens;
  if (!query_start_loc) {
    total = static_cast<long long>(dims->B) * (qlen > 0 ? qlen : 0);
    if (total > (1ll << 31) - 1) return PD_ERR_UNSUPPORTED;
  }
  const pd_score& sc = *score;
  const bool fp4 = fp4_kind(dims->kv_dtype), weights = sc.key_weights_out != nullptr;
  if (!(sc.cap == 0.f || (sc.cap >= 1e-30f && sc.cap <= 1e30f))) return PD_ERR_SHAPE;
  if (misaligned(sc.alibi_slopes, 3) || misaligned(sc.prefix_lens, 3) || misaligned(sc.lse, 3) ||
      misaligned(sc.key_weights, 3) || misaligned(sc.key_weights_out, 3) || misaligned(sc.k_block_scale, 15) ||
      misaligned(sc.v_block_scale, 15))
    return PD_ERR_ALIGN;
  Plan pl;
  CUtensorMap tk, tv;
  Fp4Params p;
  bool ready;
  const pd_status st = prepare_decode(q, k_cache, v_cache, block_table, seq_lens, query_start_loc,
                                      static_cast<int>(total), scale, window, qlen, num_splits, out, dims, workspace,
                                      workspace_bytes, error_flag, Op::kScored, sc.prefix_lens != nullptr, pl, tk, tv, p,
                                      ready);
  if (st != PD_OK || !ready) return st;
  if (fp4 && (!sc.k_block_scale || !sc.v_block_scale)) return PD_ERR_NULL;
  if (weights && !sc.key_weights) return PD_ERR_NULL;
  p.cap_u = sc.cap > 0.f ? static_cast<float>(0.6931471805599453 / sc.cap) : 0.f;
  p.cap_out = sc.cap > 0.f ? static_cast<float>(sc.cap * 1.4426950408889634) : 0.f;
  p.slopes = sc.alibi_slopes;
  p.prefix_lens = sc.prefix_lens;
  p.least_tiles = pl.least;
  p.lse = sc.lse;
  p.row_ml = nullptr;
  p.scores = nullptr;
  p.k_codes = static_cast<const uint8_t*>(k_cache);
  p.v_codes = static_cast<const uint8_t*>(v_cache);
  p.k_sf = static_cast<const uint8_t*>(sc.k_block_scale);
  p.v_sf = static_cast<const uint8_t*>(sc.v_block_scale);
  if (weights) {
    const ScoredLayout lay = scored_layout(*dims, pl, qlen);
    if (!workspace || workspace_bytes < lay.bytes) return PD_ERR_WORKSPACE;
    if (misaligned(workspace, 255)) return PD_ERR_ALIGN;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.row_ml = reinterpret_cast<float2*>(ws + lay.off_ml);
    p.scores = reinterpret_cast<float*>(ws + lay.off_scores);
  }
  auto s = static_cast<cudaStream_t>(stream);
  const WorkspaceLock lock(workspace, pl.n_merge > 0 || weights);
  cudaError_t e = launch_scored(dims->D, dims->kv_dtype, pl.nt, pl.hg > 1 ? 1 : 0, tk, tv, p, pl.grid, s);
  if (e == cudaSuccess && pl.n_merge > 0) {
    const CombineShape c = combine_shape(pl, dims->D, p.R);
    e = launch_scored_combine(dims->D, p, static_cast<int>(pl.n_merge), c.chunks, c.batch, c.threads, s);
  }
  if (e == cudaSuccess && weights) {
    KeyWeightParams kw;
    kw.d = p;
    kw.in = sc.key_weights;
    kw.out = sc.key_weights_out;
    kw.row_tiles = pl.head_tiles;
    e = launch_key_weights(kw, pl.sms, s);
  }
  return e == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}

}  // extern "C"
