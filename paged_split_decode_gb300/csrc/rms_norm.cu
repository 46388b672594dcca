// rms_norm.cu -- the root-mean-square norm of rows, with an optional residual
// added first and an optional 8-bit output with scales (rms_norm): per row
//   h = x + residual (residual_out gets h rounded to x's type),
//   y = h * rsqrt(mean of h^2 over each norm_size values + eps) * w * gain,
// and either y rounded to x's type, or, per scale_size values,
//   s = max(max |y| / Q, 2^-100), code = round(y / s)   (Q = 448 e4m3fn, 127 int8).
// The sum h is normalised as it is in fp32, not as rounded to x's type: one
// rounding per output.
//
// Memory-bound: x and the residual are read once and h and the output written
// once. The rows lie end to end, so the work is cut into chunks of whole rows
// (several where a row is short); a CTA holds a chunk in registers as fp32, up
// to eight vectors of 8 values a thread, so that nothing is read twice and
// a thread's loads are all in flight at once. The two reductions (squares per
// norm group, largest |y| per scale group) run by the group's size in vectors:
// the whole CTA; within a warp's lanes, for 1 to 32 vectors in a power of two;
// else through shared memory, a warp per group. Rows whose sizes or addresses
// do not allow 16-byte vectors take a plainer kernel. Measured: 32768 x 4096,
// fp16, residual, fp16 output 154 us (7.0 TB/s; the plainer kernel 867 us); 8192
// x 6144, bfloat16, residual, e4m3 with a scale for every 128 values 53.7 us (6.6
// TB/s; with divisions by the scale 63.5).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "launch.h"
#include "pdecode.h"

namespace pd {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxNormN = 32768;
constexpr float kMinScale = 0x1p-100f;

struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *out;
  float* out_scale;
  long long rows;
  int N, norm_size, scale_size;
  float eps, gain;
  int w_f32;
};

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

template <int OUT>
__device__ __forceinline__ uint8_t code_of(float t) {
  if constexpr (OUT == PD_NORM_E4M3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(t));
    return static_cast<uint8_t>(r & 0xffu);
  } else {
    uint32_t r;
    asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(r) : "f"(t));  // NaN -> 0
    return static_cast<uint8_t>(r & 0xffu);
  }
}

// ---- vectorised path ----------------------------------------------------------
// Threads a kernel of V vectors per thread may run: bounded by its registers.
constexpr int max_threads(int V) { return V <= 2 ? 1024 : 512; }

template <class T>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2 && std::is_same_v<T, __half>) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <class T>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same_v<T, __half>) w[i] = pack_half2(f[2 * i], f[2 * i + 1]);
    else w[i] = pack_bf162(f[2 * i], f[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int OUT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if constexpr (OUT == PD_NORM_E4M3) {
    uint16_t lo, hi;  // the first source lands in the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    return code_of<OUT>(a) | (code_of<OUT>(b) << 8) | (code_of<OUT>(c) << 16) |
           (static_cast<uint32_t>(code_of<OUT>(d)) << 24);
  }
}

// How a reduction over groups of `vecs` vectors runs.
enum Reach { kReachCta, kReachLanes, kReachShared };
struct Groups {
  int vecs;      // vectors of a group
  int reach;     // Reach
  uint32_t mul;  // ceil(2^32 / vecs) (vecs > 1): i / vecs = the product's high word, as i and vecs
                 // are at most 4096, so that i (mul vecs - 2^32) < 2^32
  __device__ __forceinline__ int of(int i) const {
    return vecs > 1 ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), mul)) : i;
  }
  __device__ __forceinline__ int within(int i) const { return i - of(i) * vecs; }
};

// Quotients of many numbers by one, rounded as y / s is, in three operations each:
// Markstein's correction (IBM Journal of Research and Development 34 (1990)). r is 1
// / s, the hardware's approximation and a step of Newton's iteration; t = y r is
// within a last place or two of y / s; the rest y - t s comes from one fused operation
// (below 2^-102 of |y| its last bits fall under fp32's range), and t + rest r is y / s
// rounded to the nearest. An infinite s gives y 0: zero, or NaN for an infinite y, as
// the division does.
struct Divider {
  float s, r;
  __device__ __forceinline__ explicit Divider(float x) : s(x < INFINITY ? x : 0.f) {
    float r0;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(x));
    r = fmaf(r0, fmaf(-s, r0, 1.f), r0);
  }
  __device__ __forceinline__ float operator()(float y) const {
    const float t = y * r;
    return fmaf(fmaf(-t, s, y), r, t);
  }
  // Two at once, in packed operations (8192 x 6144 without a residual to e4m3: 37 us
  // for y r alone, 52 with divisions, 41.4 one by one, 39.6 so; int8's conversions
  // take the values one by one, 44.4 against 47.4 packed).
  __device__ __forceinline__ void operator()(float& a, float& b) const {
    uint64_t y, rr, ss, t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(rr) : "f"(r));
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(-s));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(y), "l"(rr));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(y) : "l"(t), "l"(ss));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(y), "l"(rr), "l"(t));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(y));
  }
};

struct Plus {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Most {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// v[j] (one value per vector, vector j * threads + thread of the chunk's nv)
// becomes the op over the vector's group. s_part: a float per vector of the
// chunk; s_warp: one per warp. Values of vectors past nv are ignored (0 is
// neutral for both ops: squares and magnitudes).
template <int V, class Op>
__device__ __forceinline__ void group_reduce(float (&v)[V], int nv, const Groups& g, float* s_part, float* s_warp, Op op) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x >> 5;
  if (g.reach == kReachCta) {
    float x = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) x = op(x, v[j]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (lane == 0) s_warp[warp] = x;
    __syncthreads();
    x = lane < warps ? s_warp[lane] : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = x;
  } else if (g.reach == kReachLanes) {
    for (int o = 1; o < g.vecs; o <<= 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = op(v[j], __shfl_xor_sync(0xffffffffu, v[j], o));
    }
  } else {
    const int groups = g.of(nv);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = j * blockDim.x + t;
      if (i < nv) s_part[i] = v[j];
    }
    __syncthreads();
    // a group's result is left in its first place: by one thread (a group of at
    // most 32 vectors), else by a warp, which reads the group before
    if (g.vecs <= 32) {
      for (int q = t; q < groups; q += blockDim.x) {
        float x = s_part[q * g.vecs];
        for (int i = 1; i < g.vecs; ++i) x = op(x, s_part[q * g.vecs + i]);
        s_part[q * g.vecs] = x;
      }
    } else {
      for (int q = warp; q < groups; q += warps) {
        float x = 0.f;
        for (int i = lane; i < g.vecs; i += 32) x = op(x, s_part[q * g.vecs + i]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (lane == 0) s_part[q * g.vecs] = x;
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = j * blockDim.x + t;
      if (i < nv) v[j] = s_part[g.of(i) * g.vecs];
    }
  }
}

struct VecArgs {
  NormArgs n;
  long long vecs;   // of all rows
  int chunk;        // vectors of a chunk (whole rows)
  Groups norm, scale;
};

template <class T, int OUT, int V>
__global__ void __launch_bounds__(max_threads(V)) rms_norm_vec_kernel(const VecArgs a) {
  extern __shared__ float s_part[];  // chunk floats where a reduction needs them, twice
  __shared__ float s_warp[2][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long base = static_cast<long long>(blockIdx.x) * a.chunk;
  const int nv = static_cast<int>(min(static_cast<long long>(a.chunk), a.vecs - base));
  const int t = threadIdx.x, nt = blockDim.x;
  const uint4* x = static_cast<const uint4*>(a.n.x) + base;
  const uint4* r = a.n.residual ? static_cast<const uint4*>(a.n.residual) + base : nullptr;
  uint4* ro = a.n.residual_out ? static_cast<uint4*>(a.n.residual_out) + base : nullptr;
  uint4 xv[V], rv[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * nt + t;
    xv[j] = rv[j] = make_uint4(0u, 0u, 0u, 0u);
    if (i < nv) xv[j] = x[i];
    if (r && i < nv) rv[j] = r[i];
  }
  float h[V][8], ss[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * nt + t;
    widen8<T>(xv[j], h[j]);
    if (r) {
      float f[8];
      widen8<T>(rv[j], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[j][e] += f[e];
    }
    if (ro && i < nv) ro[i] = narrow8<T>(h[j]);
    ss[j] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss[j] += h[j][e] * h[j][e];
  }
  group_reduce(ss, nv, a.norm, s_part, s_warp[0], Plus());
  const float inv_n = 1.f / static_cast<float>(a.n.norm_size);
  float m[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = j * nt + t;
    const float inv = rsqrtf(ss[j] * inv_n + a.n.eps) * a.n.gain;
    const int wi = a.norm.reach == kReachCta ? min(i, nv - 1) : a.norm.within(i);
    float w[8];
    if (a.n.w_f32) {
      const float4* wp = static_cast<const float4*>(a.n.weight) + 2 * wi;
      const float4 w0 = __ldg(wp), w1 = __ldg(wp + 1);
      w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
      w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
    } else {
      widen8<T>(__ldg(static_cast<const uint4*>(a.n.weight) + wi), w);
    }
    m[j] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[j][e] = h[j][e] * inv * w[e];
      m[j] = fmaxf(m[j], fabsf(h[j][e]));
    }
  }
  if constexpr (OUT == PD_NORM_SAME) {
    uint4* out = static_cast<uint4*>(a.n.out) + base;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = j * nt + t;
      if (i < nv) out[i] = narrow8<T>(h[j]);
    }
  } else {
    constexpr float Q = OUT == PD_NORM_E4M3 ? 448.f : 127.f;
    const Divider by_q(Q);
    const long long scale0 = static_cast<long long>(blockIdx.x) * a.scale.of(a.chunk);
    group_reduce(m, nv, a.scale, s_part + a.chunk, s_warp[1], Most());
    uint2* out = static_cast<uint2*>(a.n.out) + base;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = j * nt + t;
      if (i >= nv) continue;
      const float s = fmaxf(m[j] < INFINITY ? by_q(m[j]) : m[j], kMinScale);
      if (a.scale.within(i) == 0) a.n.out_scale[scale0 + a.scale.of(i)] = s;
      const Divider by(s);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if constexpr (OUT == PD_NORM_E4M3) by(h[j][e], h[j][e + 1]);
        else h[j][e] = by(h[j][e]), h[j][e + 1] = by(h[j][e + 1]);
      }
      out[i] = make_uint2(codes4<OUT>(h[j][0], h[j][1], h[j][2], h[j][3]), codes4<OUT>(h[j][4], h[j][5], h[j][6], h[j][7]));
    }
  }
}

Groups groups_of(int vecs, int chunk) {
  const bool pow2 = (vecs & (vecs - 1)) == 0;
  const uint32_t mul = vecs > 1 ? static_cast<uint32_t>(((1ull << 32) + vecs - 1) / vecs) : 0u;
  return {vecs, vecs == chunk ? kReachCta : pow2 && vecs <= 32 ? kReachLanes : kReachShared, mul};
}

template <class T, int OUT, int V>
pd_status launch_vec(const VecArgs& a, int threads, cudaStream_t s) {
  static unsigned long long done[64] = {};
  if (once_per_context(done, [] {
        return set_kernel_attributes(rms_norm_vec_kernel<T, OUT, V>, 2 * kMaxNormN / 8 * 4);
      }) != cudaSuccess)
    return PD_ERR_CUDA;
  const int smem = a.norm.reach == kReachShared || (OUT != PD_NORM_SAME && a.scale.reach == kReachShared) ? 2 * a.chunk * 4 : 0;
  const long long chunks = (a.vecs + a.chunk - 1) / a.chunk;
  return launch_pdl(rms_norm_vec_kernel<T, OUT, V>, static_cast<int>(chunks), threads, smem, s, 1, a) == cudaSuccess
             ? PD_OK
             : PD_ERR_CUDA;
}

// Whether the vectorised path takes the call; its chunks, threads and vectors
// per thread. Short rows are joined to chunks of about 256 vectors. With
// fewer chunks than SMs a thread takes as few vectors as 1024 threads allow
// (latency), else four (8192 x 6144 to e4m3, residual: 54 us, with one / two /
// three vectors 112 / 59 / 54; 32768 x 6144 without one 125 us, three / eight
// 134 / 186); the widest rows take eight.
bool vec_plan(const NormArgs& n, int out_kind, int sms, VecArgs* a, int* threads, int* per) {
  auto off = [](const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
  const bool codes = out_kind != PD_NORM_SAME;
  if (n.N % 8 || n.norm_size % 8 || (codes && n.scale_size % 8)) return false;
  if (off(n.x, 15) || off(n.residual, 15) || off(n.residual_out, 15) || off(n.weight, 15) || off(n.out, codes ? 7 : 15))
    return false;
  const int row = n.N / 8;
  a->n = n;
  a->vecs = n.rows * row;
  const long long join = std::max<long long>(1, std::min<long long>(n.rows, 256 / row));
  a->chunk = static_cast<int>(join) * row;
  const long long chunks = (a->vecs + a->chunk - 1) / a->chunk;
  if (chunks > 0x7fffffffll) return false;
  *per = chunks <= sms ? 1 : 4;
  while (a->chunk > max_threads(*per) * *per) *per *= 2;
  *threads = ((a->chunk + *per - 1) / *per + 31) / 32 * 32;
  a->norm = groups_of(n.norm_size / 8, a->chunk);
  a->scale = codes ? groups_of(n.scale_size / 8, a->chunk) : Groups{1, kReachLanes, 0};
  return true;
}

// ---- any sizes and alignments: one CTA per row, the row in shared memory; each
// warp takes whole norm groups, then whole scale groups
template <class T, int OUT>
__global__ void __launch_bounds__(kNormThreads) rms_norm_kernel(const NormArgs a) {
  extern __shared__ float s_h[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr int NW = kNormThreads / 32;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.N;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * a.N : nullptr;
    T* ro = a.residual_out ? static_cast<T*>(a.residual_out) + row * a.N : nullptr;
    for (int i = t; i < a.N; i += kNormThreads) {
      float h = to_f<T>(x[i]);
      if (r) h += to_f<T>(r[i]);
      if (ro) ro[i] = from_f<T>(h);
      s_h[i] = h;
    }
    __syncthreads();
    for (int g = warp; g < a.N / a.norm_size; g += NW) {
      float* h = s_h + g * a.norm_size;
      float ss = 0.f;
      for (int i = lane; i < a.norm_size; i += 32) ss += h[i] * h[i];
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(ss / static_cast<float>(a.norm_size) + a.eps) * a.gain;
      for (int i = lane; i < a.norm_size; i += 32) {
        const float w = a.w_f32 ? static_cast<const float*>(a.weight)[i] : to_f<T>(static_cast<const T*>(a.weight)[i]);
        h[i] = h[i] * inv * w;
      }
    }
    __syncthreads();
    if constexpr (OUT == PD_NORM_SAME) {
      T* out = static_cast<T*>(a.out) + row * a.N;
      for (int i = t; i < a.N; i += kNormThreads) out[i] = from_f<T>(s_h[i]);
    } else {
      constexpr float Q = OUT == PD_NORM_E4M3 ? 448.f : 127.f;
      uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.N;
      const int groups = a.N / a.scale_size;
      for (int g = warp; g < groups; g += NW) {
        const float* y = s_h + g * a.scale_size;
        float m = 0.f;
        for (int i = lane; i < a.scale_size; i += 32) m = fmaxf(m, fabsf(y[i]));
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float s = fmaxf(m / Q, kMinScale);
        if (lane == 0) a.out_scale[row * groups + g] = s;
        for (int i = lane; i < a.scale_size; i += 32) out[g * a.scale_size + i] = code_of<OUT>(y[i] / s);
      }
    }
    __syncthreads();
  }
}

template <class T, int OUT>
pd_status launch_norm(const NormArgs& a, int sms, cudaStream_t s) {
  VecArgs v;
  int threads, per;
  if (vec_plan(a, OUT, sms, &v, &threads, &per)) {
    if (per == 1) return launch_vec<T, OUT, 1>(v, threads, s);
    if (per == 2) return launch_vec<T, OUT, 2>(v, threads, s);
    if (per == 4) return launch_vec<T, OUT, 4>(v, threads, s);
    return launch_vec<T, OUT, 8>(v, threads, s);
  }
  static unsigned long long done[64] = {};
  if (once_per_context(done, [] { return set_kernel_attributes(rms_norm_kernel<T, OUT>, kMaxNormN * 4); }) !=
      cudaSuccess)
    return PD_ERR_CUDA;
  const long long cap = static_cast<long long>(sms) * 8;
  const int grid = static_cast<int>(a.rows < cap ? a.rows : cap);
  return launch_pdl(rms_norm_kernel<T, OUT>, grid, kNormThreads, a.N * 4, s, 1, a) == cudaSuccess ? PD_OK
                                                                                                 : PD_ERR_CUDA;
}

template <class T>
pd_status launch_out(const NormArgs& a, int out_kind, int sms, cudaStream_t s) {
  if (out_kind == PD_NORM_SAME) return launch_norm<T, PD_NORM_SAME>(a, sms, s);
  if (out_kind == PD_NORM_E4M3) return launch_norm<T, PD_NORM_E4M3>(a, sms, s);
  return launch_norm<T, PD_NORM_INT8>(a, sms, s);
}

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" pd_status rms_norm(const void* x, const void* residual, const void* weight, float eps, float gain,
                              void* residual_out, void* out, float* out_scale, const pd_norm_dims* dims,
                              void* stream) {
  if (!dims) return PD_ERR_NULL;
  const pd_norm_dims& d = *dims;
  if (d.rows < 0 || d.N < 1 || d.norm_size < 1 || d.N % d.norm_size != 0) return PD_ERR_SHAPE;
  if (d.out_kind != PD_NORM_SAME && d.out_kind != PD_NORM_E4M3 && d.out_kind != PD_NORM_INT8) return PD_ERR_DTYPE;
  if (d.out_kind != PD_NORM_SAME && (d.scale_size < 1 || d.N % d.scale_size != 0)) return PD_ERR_SHAPE;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(gain)) return PD_ERR_SHAPE;
  if (d.N > kMaxNormN) return PD_ERR_UNSUPPORTED;
  if (d.rows == 0) return PD_OK;
  if (!x || !weight || !out) return PD_ERR_NULL;
  if (d.out_kind != PD_NORM_SAME && !out_scale) return PD_ERR_NULL;
  auto bad = [](const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
  if (bad(x, 1) || bad(residual, 1) || bad(residual_out, 1) || bad(weight, d.weight_f32 ? 3 : 1) ||
      bad(out, d.out_kind == PD_NORM_SAME ? 1 : 0) || bad(out_scale, 3))
    return PD_ERR_ALIGN;
  // outputs over inputs or each other, but for h over x or the residual and y over x or
  // a residual that h does not replace: those a thread reads before it writes them
  const int64_t n = d.rows * d.N, code = d.out_kind == PD_NORM_SAME ? 2 : 1;
  const int64_t scales = d.out_kind == PD_NORM_SAME ? 0 : d.rows * (d.N / d.scale_size) * 4;
  const int64_t weights = static_cast<int64_t>(d.norm_size) * (d.weight_f32 ? 4 : 2);
  auto over = [](const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return p && q && p < q + static_cast<uintptr_t>(nb) && q < p + static_cast<uintptr_t>(na);
  };
  const bool same = d.out_kind == PD_NORM_SAME;
  if ((residual_out != x && over(residual_out, 2 * n, x, 2 * n)) ||
      (residual_out != residual && over(residual_out, 2 * n, residual, 2 * n)) ||
      over(residual_out, 2 * n, weight, weights) || over(residual_out, 2 * n, out, code * n) ||
      over(residual_out, 2 * n, out_scale, scales) || (!(same && out == x) && over(out, code * n, x, 2 * n)) ||
      (!(same && out == residual) && over(out, code * n, residual, 2 * n)) || over(out, code * n, weight, weights) ||
      over(out, code * n, out_scale, scales) || over(out_scale, scales, x, 2 * n) ||
      over(out_scale, scales, residual, 2 * n) || over(out_scale, scales, weight, weights))
    return PD_ERR_SHAPE;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return PD_ERR_CUDA;
  NormArgs a{x, residual, weight, residual_out, out, out_scale, d.rows, d.N, d.norm_size, d.scale_size, eps, gain,
             d.weight_f32 ? 1 : 0};
  auto s = static_cast<cudaStream_t>(stream);
  return d.x_bf16 ? launch_out<__nv_bfloat16>(a, d.out_kind, sms, s) : launch_out<__half>(a, d.out_kind, sms, s);
}
