/*
 * pdecode.h -- C ABI of libpdecode: paged split-K decode attention on one
 * NVIDIA GB300 (sm_103a).
 *
 * What the library computes follows opengfx1030/vllm-rdna pull request #33
 * ("Paged split-K decode"):
 *   - "Purpose": a per-head decode over a paged KV cache -- page lookups
 *     through a block table, scores scale * q . k, online softmax, P.V, and
 *     split-K partials merged by a combine; fp16, fp8 and int8 KV share the body;
 *     every launch runs on the caller's current stream;
 *   - "What changed vs the old #33 diff": an empty key range never enters the
 *     P.V loop (empty rows are zero);
 *   - "Test Plan" step 2: the decode cells -- writer layout, empty rows are
 *     zero, a custom scale written into a caller-owned `out`, a paged sliding
 *     window, multi-token (speculative verify) queries, split decode;
 *   - "Test Result": the split-K schedule must agree with a one-shot fp64
 *     reference.
 *
 * Readings where the page is silent:
 *   - seq_lens[b] counts every cached key of sequence b, including its qlen
 *     query tokens; query token i sits at position p = seq_lens[b] - qlen + i
 *     and sees keys j <= p (causal among the query tokens);
 *   - window W > 0 keeps keys p - W + 1 <= j <= p; W <= 0 disables it;
 *   - query head h reads KV head h / (Hq / Hkv);
 *   - a row with no visible key is written as zeros.
 *
 * Conventions shared by every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller, contiguous
 *     and row-major, on the device that is current when the call is made. The
 *     library never allocates, frees or synchronises; it launches on `stream`
 *     (a cudaStream_t; NULL = the legacy default stream) and returns at once.
 *   - Host-checkable problems are reported through the return value before
 *     anything is launched. PD_ERR_CUDA means a launch or runtime call failed;
 *     the library only peeks at the runtime's last error, so the caller's
 *     cudaGetLastError() still returns the CUDA error.
 *   - Data errors that only the device can see (a block id outside
 *     [0, num_blocks), a seq_len outside [0, max_blocks_per_seq*block_size],
 *     a pipeline wait that ran past its time limit) never trap: the kernel
 *     sets a bit of *error_flag (if error_flag is not NULL) with atomicOr and
 *     carries on; the affected rows are then unspecified. The caller clears
 *     the flag.
 *   - There is no CPU fallback and no alternative back end: shapes the
 *     kernels do not implement return PD_ERR_UNSUPPORTED.
 */
#ifndef PDECODE_H
#define PDECODE_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PD_API __attribute__((visibility("default")))
#else
#define PD_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PD_OK = 0,
  PD_ERR_NULL = 1,        /* a required pointer is NULL */
  PD_ERR_SHAPE = 2,       /* sizes are inconsistent or out of range */
  PD_ERR_DTYPE = 3,       /* unknown KV dtype */
  PD_ERR_UNSUPPORTED = 4, /* legal, but no kernel here implements it */
  PD_ERR_ALIGN = 5,       /* a pointer is not 16-byte aligned */
  PD_ERR_WORKSPACE = 6,   /* workspace missing or smaller than pd_workspace_bytes */
  PD_ERR_CUDA = 7         /* a CUDA runtime call or launch failed */
} pd_status;

typedef enum {
  PD_KV_F16 = 0,       /* K and V caches hold IEEE binary16 */
  PD_KV_FP8_E4M3 = 1,  /* K and V caches hold OCP e4m3fn codes; value = decode(code) * scale */
  PD_KV_INT8 = 2,      /* K and V caches hold int8 two's-complement codes; value = code * scale */
  PD_KV_BF16 = 3,      /* K and V caches, q and out hold bfloat16 (scales ignored); the products
                          run on bfloat16 tensor-core operands (P rounded to bfloat16) */
  PD_KV_FP8_E4M3_BF16 = 4, /* e4m3fn caches as PD_KV_FP8_E4M3, q and out (and the writer's new
                              tokens) in bfloat16: each q row is scaled by a power of two into
                              fp16 exactly and the products run as for an fp16 q */
  PD_KV_INT8_BF16 = 5  /* int8 caches as PD_KV_INT8, q and out (and new tokens) in bfloat16 */
} pd_kv_dtype;

/* Bits written into *error_flag by the device. */
#define PD_DEVERR_BLOCK_ID 1u /* a block_table entry used by the call is outside [0, num_blocks) */
#define PD_DEVERR_SEQ_LEN 2u  /* a seq_len is negative or above max_blocks_per_seq*block_size */
#define PD_DEVERR_TIMEOUT 4u  /* a pipeline wait ran past its limit; the call gave up */
#define PD_DEVERR_SLOT 8u     /* write_kv_cache: a slot at or beyond num_blocks*block_size */
#define PD_DEVERR_QUERY_START 16u /* decode_paged_varlen: a sequence's query range is malformed */
#define PD_DEVERR_FREE_LIST 32u /* the free list has too few blocks, would overflow, or its count is bad */

/* Shapes of one call.
 *   B                  number of sequences (rows of block_table / seq_lens)
 *   Hq, Hkv            query and KV heads; Hq % Hkv == 0
 *   D                  head size; the kernels implement 128 and 256
 *   block_size         keys per cache block; a multiple of 16
 *   num_blocks         blocks in each of the K and V caches
 *   max_blocks_per_seq columns of block_table
 *   kv_dtype           pd_kv_dtype
 *   k_scale, v_scale   fp8 / int8 (either q type): per-cache dequantisation scales
 *                      (ignored for fp16 and bfloat16 caches) */
typedef struct {
  int32_t B, Hq, Hkv, D;
  int32_t block_size, num_blocks, max_blocks_per_seq;
  int32_t kv_dtype;
  float k_scale, v_scale;
} pd_dims;

/* Workspace bytes that decode_paged needs for these shapes, qlen and
 * num_splits (0 = balanced automatic split) on a device with sm_count SMs
 * (sm_count <= 0: the current device's). 0 means no workspace is needed (the
 * pointer may then be NULL). Layout: the fp32 split partials (m and l of
 * every partial row, then its O row); a split unit's pieces and their slots
 * follow from the sequence lengths, so nothing else is stored. Every
 * call writes what it later reads, so the buffer needs no initialisation and
 * one buffer serves any sequence of calls on one stream, from any threads (a
 * call's launches stay together); calls that may run at the same time on the
 * GPU must not share a workspace. Returns 0 for invalid dims. */
PD_API size_t pd_workspace_bytes(const pd_dims* dims, int qlen, int num_splits, int sm_count);

/* Number of CTAs decode_paged launches for these arguments (persistent grid),
 * or 0 for invalid dims. Host-only; no device work. */
PD_API int pd_grid_ctas(const pd_dims* dims, int qlen, int num_splits, int sm_count);

/* Paged decode attention, split-K over keys, GQA heads packed per CTA.
 * With a split (num_splits != 1) the call is two launches on `stream`: the
 * decode kernel, then a split-combine kernel launched with programmatic
 * dependent launch that merges the partials of units cut into pieces; a
 * fixed split of 2 to 16 pieces per unit whose pieces get one CTA each is
 * instead one launch of thread-block clusters (one per unit) that merge the
 * pieces themselves, when the device runs all those clusters at once.
 *
 *   q            fp16 [B*qlen, Hq, D] (bfloat16 for PD_KV_BF16, PD_KV_FP8_E4M3_BF16 and
 *                PD_KV_INT8_BF16); row b*qlen + i is query token i of sequence b
 *   k_cache      [num_blocks, block_size, Hkv, D] fp16, bfloat16, e4m3fn or int8
 *                (dims->kv_dtype)
 *   v_cache      same layout and dtype as k_cache
 *   block_table  int32 [B, max_blocks_per_seq]; entry [b][n] is the physical
 *                block holding keys n*block_size .. n*block_size+block_size-1 of
 *                sequence b. Only the entries of blocks holding visible keys are read.
 *   seq_lens     int32 [B]; keys cached for each sequence, query tokens included
 *   scale        multiplies q . k (e.g. 1/sqrt(D))
 *   window       sliding window in keys (<= 0: none)
 *   qlen         query tokens per sequence, 1..8; Hq/Hkv*qlen must be <= 32
 *   num_splits   0: balanced split of all visible key tiles over the SMs;
 *                >= 1: each sequence's visible tiles cut into num_splits
 *                contiguous chunks (1 = no split)
 *   out          q's type, [B*qlen, Hq, D], written in full (rows without a visible
 *                key are zeros); must not overlap the inputs
 *   workspace    device buffer of >= pd_workspace_bytes(...) bytes (contents need
 *                no initialisation; see pd_workspace_bytes)
 *   error_flag   device uint32 or NULL (see PD_DEVERR_*)
 *   stream       cudaStream_t to launch on
 * All pointers must be 16-byte aligned. */
PD_API pd_status decode_paged(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* seq_lens, float scale,
                       int window, int qlen, int num_splits, void* out, const pd_dims* dims,
                       void* workspace, size_t workspace_bytes, uint32_t* error_flag,
                       void* stream);

/* decode_paged with a different number of query tokens per sequence (the
 * multi-token verify cell of "Test Plan" generalised: a batch mixing plain
 * decode with speculative verify of varying depth).
 *   query_start_loc  device int32 [B+1], non-decreasing: sequence b owns rows
 *                    query_start_loc[b] .. query_start_loc[b+1]-1 of q and
 *                    out, its qlen_b = query_start_loc[b+1] - query_start_loc[b]
 *                    tokens at positions seq_lens[b] - qlen_b + i (i < qlen_b)
 *   num_query_tokens rows of q and out (total over the batch)
 *   max_qlen         an upper bound of every qlen_b, 1..8; it sizes the
 *                    kernel (G * max_qlen <= 32) and the workspace:
 *                    pd_workspace_bytes(dims, max_qlen, num_splits, 0)
 * Every other argument is decode_paged's. A sequence with qlen_b = 0 writes
 * nothing; rows of out outside [query_start_loc[0], query_start_loc[B]) are
 * not written. A range that decreases, exceeds max_qlen or leaves
 * [0, num_query_tokens) sets PD_DEVERR_QUERY_START and that sequence is
 * skipped. */
PD_API pd_status decode_paged_varlen(const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* block_table, const int32_t* seq_lens,
                                     const int32_t* query_start_loc, int num_query_tokens,
                                     int max_qlen, float scale, int window, int num_splits,
                                     void* out, const pd_dims* dims, void* workspace,
                                     size_t workspace_bytes, uint32_t* error_flag, void* stream);

/* Split-K combine on its own (the combine step of "Purpose" and of the
 * schedule model in "Test Result"). For each of `rows` rows and S partials:
 *   part_m  fp32 [rows, S]     largest score of the chunk, natural-log units
 *                              (-inf for an empty chunk)
 *   part_l  fp32 [rows, S]     sum over the chunk of exp(s_j - m)
 *   part_o  fp32 [rows, S, D]  sum over the chunk of exp(s_j - m) * V_j
 *   out     fp16 [rows, D]     sum_s w_s O_s / sum_s w_s l_s with
 *                              w_s = exp(m_s - max_s m_s); zeros when every
 *                              chunk is empty
 * D is 1..1024 and a multiple of 8. */
PD_API pd_status decode_paged_combine(const float* part_m, const float* part_l, const float* part_o,
                               int rows, int num_splits, int D, void* out, void* stream);

/* Paged KV-cache writer: stores the K and V rows of new tokens where the
 * decode reads them (opengfx1030/vllm-rdna pull request #33, "Test Plan": the
 * decode is checked against the paged writer's layout).
 *   k_new, v_new  fp16 [num_tokens, Hkv, D] (bfloat16 for PD_KV_BF16, PD_KV_FP8_E4M3_BF16
 *                 and PD_KV_INT8_BF16), 16-byte aligned
 *   slot_mapping  int64 [num_tokens], device; token t goes to block
 *                 slot / block_size, offset slot % block_size of both caches;
 *                 a negative slot is a padding token and writes nothing
 *   k_cache,      [num_blocks, block_size, Hkv, D] of dims->kv_dtype (16-byte
 *   v_cache       aligned for 16-bit kinds, 8-byte for one-byte codes), updated in place
 *   dims          Hkv, D (a multiple of 8), block_size, num_blocks, kv_dtype,
 *                 k_scale, v_scale are read; B, Hq, max_blocks_per_seq are not
 *   error_flag    device uint32 or NULL
 * fp16 and bfloat16 caches receive the input bits unchanged. fp8 / int8 caches receive the
 * code nearest to the IEEE fp32 quotient x / k_scale (V: v_scale): e4m3fn
 * with ties to even, saturating at +-448, NaN -> 0x7F; int8 with ties to even,
 * clamped to [-127, 127], NaN -> 0. A slot at or beyond num_blocks*block_size
 * writes nothing and sets PD_DEVERR_SLOT. Two tokens with the same slot race
 * (one of them wins). One launch on `stream`; nothing is allocated. */
PD_API pd_status write_kv_cache(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                                int num_tokens, void* k_cache, void* v_cache, const pd_dims* dims,
                                uint32_t* error_flag, void* stream);

/* Differential decode over the paged caches: decode_paged with two softmax
 * maps per head and their difference weighted by a learned factor. The head
 * size D of dims (128 or 256) is that of the cache rows and of V; each q row
 * and each K row is two halves of D / 2, one per map:
 *   out[h] = softmax(scale * q[h][:D/2] . K[:][:D/2]) V
 *          - lambda[h] * softmax(scale * q[h][D/2:] . K[:][D/2:]) V
 * over the keys that decode_paged's masks leave (causal, window), followed,
 * where norm_weight is given, by the head's own root-mean-square norm:
 *   out[h] = out[h] * rsqrt(mean(out[h]^2) + norm_eps) * norm_weight * norm_gain.
 * The caches, their writer (write_kv_cache), block_table, seq_lens, the
 * splits, the workspace rules and the errors are decode_paged's. Both maps of
 * a head are computed from one reading of its K and V.
 *   lambda          device fp32 [Hq]
 *   query_start_loc NULL: qlen query tokens for each sequence (num_query_tokens
 *                   is then ignored); else int32 [B+1] as in
 *                   decode_paged_varlen, and qlen is the bound of every count
 *   norm_weight     [D] of q's type (norm_weight_f32 = 0) or fp32 (1), or NULL
 *   norm_eps        >= 0; norm_gain multiplies the result (ignored without a
 *                   norm_weight)
 *   workspace       pd_diff_workspace_bytes(dims, qlen, num_splits, 0) bytes
 * A map contributes zeros to a row that has no visible key, or where a visible
 * score is NaN or +infinity (a NaN in that half of q or K). NaN and infinities
 * of V rows show, as NaN or infinity, in the output rows that see the key and in no other
 * (several query tokens, windows). Softmax weights are computed in fp32 and
 * enter the product with V as two 16-bit operands over 16-bit caches with
 * Hq/Hkv*qlen <= 16, else rounded once to 16 bits (bfloat16 for bfloat16 caches,
 * fp16 for all others); every sum is fp32. Hq/Hkv*qlen must be <= 32. */
PD_API size_t pd_diff_workspace_bytes(const pd_dims* dims, int qlen, int num_splits, int sm_count);
PD_API pd_status decode_paged_diff(const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_table, const int32_t* seq_lens,
                                   const int32_t* query_start_loc, int num_query_tokens,
                                   const float* lambda, float scale, int window, int qlen,
                                   int num_splits, const void* norm_weight, int norm_weight_f32,
                                   float norm_eps, float norm_gain, void* out, const pd_dims* dims,
                                   void* workspace, size_t workspace_bytes, uint32_t* error_flag,
                                   void* stream);

/* Block tables and slot maps of one serving step, built on the GPU from the
 * requests' lengths, for write_kv_cache and decode_paged_varlen. Sequence b
 * has context_lens[b] keys in the cache and brings query_lens[b] new tokens;
 * it holds the first ceil(context_lens[b] / block_size) entries of its
 * block_table row and is given what it lacks from the top of the free list.
 *   context_lens    int32 [B]
 *   query_lens      int32 [B]; 0 for a sequence that rests (or a padding row)
 *   num_tokens      entries of slot_mapping and positions: at least the sum of
 *                   query_lens, more for a padded batch
 *   block_table     int32 [B, max_blocks_per_seq], new entries written
 *   free_blocks     int32 [num_blocks], of which the first free_count[0] are
 *                   the free blocks' ids; the last of them is taken first,
 *                   sequences in order
 *   free_count      int32 [1]; free_count_out [1] gets what is left (may be
 *                   free_count itself)
 *   seq_lens        int32 [B]: context + query (may be context_lens itself)
 *   query_start_loc int32 [B+1]: exclusive prefix sums of query_lens
 *   slot_mapping    int64 [num_tokens]: the tokens' slots, -1 behind the last
 *   positions       int32 [num_tokens] or NULL: the tokens' positions in their
 *                   sequences, 0 behind the last
 *   dims            B (at most 16384), block_size, num_blocks and
 *                   max_blocks_per_seq are read
 * A sequence is served whole or not at all: one with a bad length
 * (PD_DEVERR_SEQ_LEN), whose tokens pass num_tokens (PD_DEVERR_QUERY_START) or
 * for which the free list has too few blocks (PD_DEVERR_FREE_LIST; every later
 * sequence that needs a block is refused too) takes no block and its slots are
 * -1. Its seq_lens entry is 0 where seq_lens is a buffer of its own (a decode
 * then writes zeros for it); where seq_lens is context_lens itself the entry
 * stays as it was, so that the sequence keeps its blocks, can be served in a
 * later step and released (a decode of the refused step then gives its rows
 * the keys that it has: results to be ignored, as its slots say). An id outside
 * [0, num_blocks) among those used sets PD_DEVERR_BLOCK_ID and gives slot -1.
 * One launch on `stream`. */
PD_API pd_status build_block_tables(const int32_t* context_lens, const int32_t* query_lens,
                                    int num_tokens, int32_t* block_table,
                                    const int32_t* free_blocks, const int32_t* free_count,
                                    int32_t* free_count_out, int32_t* seq_lens,
                                    int32_t* query_start_loc, int64_t* slot_mapping,
                                    int32_t* positions, const pd_dims* dims,
                                    uint32_t* error_flag, void* stream);

/* Returns the blocks of finished sequences to the free list: for every b with
 * released[b] != 0 (one byte each), in order, the first
 * ceil(seq_lens[b] / block_size) entries of its block_table row are appended.
 *   free_count      int32 [1]; free_count_out [1] gets the new count (may be
 *                   free_count itself)
 *   seq_lens_out    int32 [B]: seq_lens, 0 for a released sequence (may be
 *                   seq_lens itself)
 * The table's entries stay. A marked sequence with a bad length
 * (PD_DEVERR_SEQ_LEN), or whose blocks would make the list longer than
 * num_blocks (PD_DEVERR_FREE_LIST), is not released. An entry outside
 * [0, num_blocks) sets PD_DEVERR_BLOCK_ID and is appended as -1. One launch on
 * `stream`. */
PD_API pd_status release_blocks(const int32_t* block_table, const int32_t* seq_lens,
                                const uint8_t* released, int32_t* free_blocks,
                                const int32_t* free_count, int32_t* free_count_out,
                                int32_t* seq_lens_out, const pd_dims* dims,
                                uint32_t* error_flag, void* stream);

typedef enum {
  PD_NORM_SAME = 0, /* x's type */
  PD_NORM_E4M3 = 1, /* OCP e4m3fn codes; value = decode(code) * scale */
  PD_NORM_INT8 = 2  /* int8 codes in [-127, 127]; value = code * scale */
} pd_norm_out;

/* Shapes of one rms_norm call.
 *   rows, N     x is [rows, N]; N is at most 32768
 *   norm_size   values normalised together, a divisor of N (N: the whole row;
 *               D: every head of a decode's output on its own)
 *   scale_size  8-bit outputs: values that share a scale, a divisor of N
 *   x_bf16      x, residual (and out, for PD_NORM_SAME) are bfloat16, else fp16
 *   weight_f32  weight is fp32, else of x's type
 *   out_kind    pd_norm_out */
typedef struct {
  int64_t rows;
  int32_t N, norm_size, scale_size;
  int32_t x_bf16, weight_f32, out_kind;
} pd_norm_dims;

/* Root-mean-square norm of rows with the residual's addition and an 8-bit
 * output: in fp32, h = x + residual; y = h * rsqrt(mean(h^2) + eps) * weight *
 * gain, the mean over each norm_size values.
 *   x            [rows, N]
 *   residual     [rows, N] of x's type, or NULL (h = x)
 *   weight       [norm_size]
 *   residual_out [rows, N] of x's type or NULL: gets h rounded (may be
 *                residual or x)
 *   out          [rows, N]: y in x's type (may be x or, without a
 *                residual_out, residual), or one byte codes of y / s rounded
 *                to the nearest, ties to even, NaN as write_kv_cache's
 *   out_scale    8-bit outputs: fp32 [rows, N / scale_size], s = max(max |y| / Q,
 *                2^-100), Q = 448 (e4m3fn) or 127 (int8), NaN left out of the
 *                maximum
 * Otherwise no output may overlap an input or another output (PD_ERR_SHAPE). One
 * launch on `stream`. */
PD_API pd_status rms_norm(const void* x, const void* residual, const void* weight, float eps,
                          float gain, void* residual_out, void* out, float* out_scale,
                          const pd_norm_dims* dims, void* stream);

/* Failure-detection controls (process-wide, read at each launch; for tests of
 * the error path, not for production use).
 *   pd_set_wait_limit_ns: wall-time limit of every pipeline wait inside the
 *     decode kernel (0 restores the default, 2 s). A wait that runs past it
 *     sets PD_DEVERR_TIMEOUT; the kernel then skips its remaining waits and
 *     work, keeps its barrier sequence, lets every issued copy land and exits,
 *     so the CUDA context stays usable.
 *   pd_set_fault_injection: 1 makes the decode kernel's producer issue no
 *     loads, so the consumers' waits can only run out (a wait that nothing
 *     completes); 0 turns it off. The outputs of such calls are unspecified. */
PD_API void pd_set_wait_limit_ns(unsigned long long ns);
PD_API void pd_set_fault_injection(int mode);

/* Size of the scratch array built into the library for
 * decode_paged_static_scratch (32 MiB). Every GPU on which that entry point
 * has been called keeps this much device memory until the process exits. */
#define PD_STATIC_SCRATCH_BYTES (32u << 20)

/* decode_paged for callers that cannot allocate device memory (no counterpart
 * in the pages: it exists for this library's users). Some callers cannot call
 * cudaMalloc -- code running inside an allocator's own callbacks, a plugin
 * host that hands out no device buffers, a process whose device footprint is
 * fixed after start-up -- so they cannot provide decode_paged's workspace.
 * This entry point takes the same arguments minus the workspace and uses a
 * scratch array of PD_STATIC_SCRATCH_BYTES compiled into the library.
 *   - It allocates nothing: no cudaMalloc, no cudaFree, no allocating
 *     library routine. The caller still owns q, the caches, the tables,
 *     out and error_flag.
 *   - Calls whose workspace (pd_workspace_bytes) exceeds
 *     PD_STATIC_SCRATCH_BYTES return PD_ERR_WORKSPACE before anything runs.
 *   - Each call launches exactly as decode_paged does, on `stream`.
 *   - The first call on a device looks up the scratch's device address on
 *     that device (cudaGetSymbolAddress, the device being current). Under
 *     CUDA's lazy module loading (the default) that lookup is also when the
 *     driver loads the module holding the array and takes its
 *     PD_STATIC_SCRATCH_BYTES of device memory. So make the first call on
 *     each device at start-up: outside any allocator callback, while the
 *     process may still grow its footprint, and before any stream capture.
 *     Later calls take no device memory.
 *   - After a cudaDeviceReset the next call on that device is a first call
 *     again (the address is looked up in the new context).
 *   - All calls on a device share the one scratch array, which keeps the
 *     last call's contents: calls that may overlap on the GPU (different
 *     streams without ordering between them) race and give wrong results. */
PD_API pd_status decode_paged_static_scratch(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_table, const int32_t* seq_lens, float scale,
                       int window, int qlen, int num_splits, void* out, const pd_dims* dims,
                       uint32_t* error_flag, void* stream);

/* Human-readable name of a status. */
PD_API const char* pd_status_str(pd_status status);

#ifdef __cplusplus
}
#endif

#endif /* PDECODE_H */
