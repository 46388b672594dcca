// rms_norm.cu -- the root-mean-square norm of rows, with an optional residual
// added first and an optional 8-bit output with scales (rms_norm): per row
//   h = x + residual (residual_out gets h rounded to x's type),
//   y = h * rsqrt(mean of h^2 over each norm_size values + eps) * w * gain,
// and either y rounded to x's type, or, per scale_size values,
//   s = max(max |y| / Q, 2^-100), code = round(y / s)   (Q = 448 e4m3fn, 127 int8).
// The sum h is normalised as it is in fp32, not as rounded to x's type: one
// rounding per output.
//
// One CTA per row, the row in shared memory as fp32; each warp takes whole
// norm groups, then whole scale groups.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return PD_ERR_CUDA;
  NormArgs a{x, residual, weight, residual_out, out, out_scale, d.rows, d.N, d.norm_size, d.scale_size, eps, gain,
             d.weight_f32 ? 1 : 0};
  auto s = static_cast<cudaStream_t>(stream);
  return d.x_bf16 ? launch_out<__nv_bfloat16>(a, d.out_kind, sms, s) : launch_out<__half>(a, d.out_kind, sms, s);
}
