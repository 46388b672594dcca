// key_weights.cu -- the attention weight that keys collect, behind a scored decode.
//
//   out[key, kv head] = in[key, kv head] + sum over query tokens i and heads h of
//   the group of 2^(x_ih - m_ih) / l_ih
// over the scores x (log2 units, -inf where masked) that the decode left in the
// workspace, and the rows' (m, l), final only when all of a row's pieces are
// joined: hence a launch of its own behind them. Keys of the call's own query
// tokens start from zero, keys that no row sees keep their sum.
//
// Bytes: 32 a key, head and row tile of eight rows, written by the decode and
// read here, and 8 for the sums; against 512 to 2048 for the key's K and V. A thread
// takes two keys: each one's eight rows are two 16-byte loads, the rows' (m, 1 / l) come
// from shared memory. Bound by the latency of two dependent loads: the table and the old
// sums are read before the decode's end is waited for, and a CTA has 256 keys only, so
// that long sequences of a ragged batch spread over the SMs (32 sequences of up to 16384
// keys, eight heads of four rows, 4-bit: the call takes 100.1 us with CTAs of 128 threads
// and two keys a thread, 113.0 with four, 119.6 with eight; 115.6 with one key of 256
// threads and every load behind the wait; without this launch 86.8).
#include <algorithm>

#include "scored_launch.h"

namespace pd {
namespace {

constexpr int kThreads = 128;
constexpr int kKeys = 2;  // keys of a thread, in flight together

__global__ void __launch_bounds__(kThreads) key_weights_kernel(const KeyWeightParams kp) {
  const ScoredParams& p = kp.d;
  __shared__ float2 s_row[32];  // (m, 1 / l); 0 for l where the row gives nothing
  const int u = blockIdx.x / kp.chunks, c = blockIdx.x % kp.chunks;  // unit, share of its keys
  const int b = u / p.Hkv, kh = u % p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // lengths, table and the old sums are not the decode's: they are read before its end
  int L, t0, n, q0, qn;
  seq_span(p, b, false, L, t0, n, q0, qn);
  const int R = p.G * qn;
  // visible tiles: [0, np) and [first, ...)
  const int first = p.window > 0 ? max(0, L - qn - p.window + 1) / kTileKeys : 0;
  const int np = (prefix_of(p, b, L) + kTileKeys - 1) / kTileKeys;
  const int stride = kp.row_tiles * 128;  // floats of a tile
  const float* scores = p.scores + static_cast<long long>(u) * p.max_blocks * p.tiles_per_block * stride;
  const int32_t* row = p.block_table + static_cast<long long>(b) * p.max_blocks;
  bool ready = false;
  for (int j0 = c * kThreads * kKeys; j0 < L; j0 += kp.chunks * kThreads * kKeys) {
    long long at[kKeys];
    float old[kKeys], sum[kKeys];
    const float* src[kKeys];  // null: no row sees the key
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      const int j = j0 + k * kThreads + threadIdx.x;
      const int blk = j < L ? __ldg(row + j / p.block_size) : -1;
      // (a bad block: the decode reported it, where it is visible)
      at[k] = blk < 0 || blk >= p.num_blocks
                  ? -1 : (static_cast<long long>(blk) * p.Hkv + kh) * p.block_size + j % p.block_size;
    }
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      const int j = j0 + k * kThreads + threadIdx.x, tile = j / kTileKeys;
      old[k] = at[k] >= 0 && j < L - qn ? kp.in[at[k]] : 0.f;
      sum[k] = 0.f;
      src[k] = at[k] >= 0 && (tile < np || tile >= first)
                   ? scores + static_cast<long long>(tile) * stride + (j % kTileKeys) * 8 : nullptr;
    }
    if (!ready) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      if (threadIdx.x < 32) {
        float2 v = make_float2(0.f, 0.f);
        if (static_cast<int>(threadIdx.x) < R) {
          v = __ldcg(p.row_ml + (static_cast<long long>(b) * p.qlen + threadIdx.x / p.G) * p.Hq + kh * p.G +
                     threadIdx.x % p.G);
          v.y = v.y == 0.f ? 0.f : 1.f / v.y;
        }
        s_row[threadIdx.x] = v;
      }
    }
    for (int r = 0; r < R; r += 8) {
      float4 x[kKeys][2];
#pragma unroll
      for (int k = 0; k < kKeys; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[k][h] = src[k] ? __ldcg(reinterpret_cast<const float4*>(src[k] + r * 16) + h)
                           : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (!ready) __syncthreads();
      ready = true;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 ml = s_row[r + e];
        if (r + e >= R) break;
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
          const float4 v = x[k][e >> 2];
          const float y = (e & 3) == 0 ? v.x : (e & 3) == 1 ? v.y : (e & 3) == 2 ? v.z : v.w;
          if (y != -INFINITY) sum[k] += ex2(y - ml.x) * ml.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kKeys; ++k)
      if (at[k] >= 0) kp.out[at[k]] = old[k] + sum[k];
  }
  // (CTAs without keys leave at once; one must stay, so that this grid does not end before the decode)
  if (blockIdx.x == 0 && !ready) asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

cudaError_t launch_key_weights(KeyWeightParams p, int sms, cudaStream_t stream) {
  // CTAs for a table's every key, at most eight rounds of the SMs' resident ones
  const long long units = static_cast<long long>(p.d.B) * p.d.Hkv;
  const long long keys = static_cast<long long>(p.d.max_blocks) * p.d.block_size;
  const long long most = std::max<long long>(1, 64ll * sms / units);
  p.chunks = static_cast<int>(std::max<long long>(1, std::min((keys + kThreads * kKeys - 1) / (kThreads * kKeys), most)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * p.chunks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, key_weights_kernel, p);
  return e != cudaSuccess ? e : cudaPeekAtLastError();
}

}  // namespace pd
