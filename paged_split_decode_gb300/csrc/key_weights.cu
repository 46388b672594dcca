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
// read here mostly from L2 (B = 32, L = 4096, four heads: 17 MB), and 8 for the
// sums; against 512 to 2048 for the key's K and V. A thread a key: its eight rows
// are two 16-byte loads, the rows' (m, 1 / l) come from shared memory.
#include <algorithm>

#include "scored_launch.h"

namespace pd {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) key_weights_kernel(const KeyWeightParams kp) {
  const ScoredParams& p = kp.d;
  __shared__ float2 s_row[32];  // (m, 1 / l); 0 for l where the row gives nothing
  const int u = blockIdx.x / kp.chunks, c = blockIdx.x % kp.chunks;  // unit, share of its keys
  const int b = u / p.Hkv, kh = u % p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int L, t0, n, q0, qn;
  seq_span(p, b, false, L, t0, n, q0, qn);
  if (c * kThreads >= L) return;
  const int R = p.G * qn;
  if (threadIdx.x < 32) {
    float2 v = make_float2(0.f, 0.f);
    if (static_cast<int>(threadIdx.x) < R) {
      v = __ldcg(p.row_ml + (static_cast<long long>(b) * p.qlen + threadIdx.x / p.G) * p.Hq + kh * p.G + threadIdx.x % p.G);
      v.y = v.y == 0.f ? 0.f : 1.f / v.y;
    }
    s_row[threadIdx.x] = v;
  }
  __syncthreads();
  // visible tiles: [0, np) and [first, ...)
  const int first = p.window > 0 ? max(0, L - qn - p.window + 1) / kTileKeys : 0;
  const int np = (prefix_of(p, b, L) + kTileKeys - 1) / kTileKeys;
  const float* scores = p.scores + static_cast<long long>(u) * p.max_blocks * p.tiles_per_block * (kp.row_tiles * 128);
  const int32_t* row = p.block_table + static_cast<long long>(b) * p.max_blocks;
  for (int j = c * kThreads + threadIdx.x; j < L; j += kp.chunks * kThreads) {
    const int blk = __ldg(row + j / p.block_size);
    if (blk < 0 || blk >= p.num_blocks) continue;  // (the decode reported it, where it is visible)
    const long long at = (static_cast<long long>(blk) * p.Hkv + kh) * p.block_size + j % p.block_size;
    const float old = j < L - qn ? kp.in[at] : 0.f;
    const int tile = j / kTileKeys;
    float sum = 0.f;
    if (tile < np || tile >= first) {
      const float* src = scores + static_cast<long long>(tile) * (kp.row_tiles * 128) + (j % kTileKeys) * 8;
      for (int r = 0; r < R; r += 8) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(src + r * 16));
        const float4 c = __ldcg(reinterpret_cast<const float4*>(src + r * 16 + 4));
        const float x[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 ml = s_row[r + e];
          if (r + e < R && x[e] != -INFINITY) sum += ex2(x[e] - ml.x) * ml.y;
        }
      }
    }
    kp.out[at] = old + sum;
  }
}

}  // namespace

cudaError_t launch_key_weights(KeyWeightParams p, int sms, cudaStream_t stream) {
  // CTAs for a table's every key, at most eight rounds of the SMs' resident ones
  const long long units = static_cast<long long>(p.d.B) * p.d.Hkv;
  const long long keys = static_cast<long long>(p.d.max_blocks) * p.d.block_size;
  const long long most = std::max<long long>(1, 64ll * sms / units);
  p.chunks = static_cast<int>(std::max<long long>(1, std::min((keys + kThreads - 1) / kThreads, most)));
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
