// fp4_writer.cu -- the writer of the 4-bit paged caches: e2m1 codes and an e4m3 scale
// for every 16 dims (write_kv_cache_fp4).
//
//   s = e4m3(amax / (6 g)), d = s g, code = e2m1(x / d)
// with g the cache's fp32 scale; the quotients are IEEE fp32 ones. As in
// kv_writer.cu they come from a reciprocal by one residual correction (Markstein):
// r = RN(1 / d), q0 = RN(x r), q1 = RN(q0 + r (x - q0 d)), here with a division per
// 16 values, since every group has its own d.
//
// 32 bytes in, 9 out for a group. A thread takes a group of K and the
// same of V: its values stay in its registers, and the group's maximum needs no
// exchange between lanes. Each is one 32-byte load (two of 16 where the rows are not
// aligned to it). Quotients go two to an instruction (32768 tokens, 4 heads, D = 256: 35.1 to
// 36.7 us, 0.7 of the copy rate; one by one 37.6; 16 CTAs an SM instead of 64 36.7; the next
// group's loads before this one's quotients 37.2). No unit is full: instructions 2.7 of 4 a cycle, the ALU pipe
// 59 %, DRAM 55; slots in order or at random take the same 33.3 us in a graph, so the scales' half sectors are not it.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pdecode.h"
#include "ptx.cuh"

namespace pd {
namespace {

constexpr int kThreads = 128;

struct WriteArgs {
  const uint8_t *k_new, *v_new;
  const int64_t* slots;
  uint8_t *k_codes, *v_codes, *k_sf, *v_sf;
  uint32_t* error_flag;
  long long items;       // groups of 16 dims of all tokens
  long long num_slots;
  int groups, head_groups;  // of a token, of a head
  int Hkv, block_size;
  float k_scale, v_scale, k_scale6, v_scale6, k_rcp6, v_rcp6;  // 6 scale, 1 / (6 scale)
  int aligned32;         // the new rows begin at a multiple of 32 bytes
  int fast;              // scales within [2^-60, 2^60]: no residual that matters meets fp32's ends
};

struct Vec32 {
  uint32_t w[8];
};
__device__ __forceinline__ Vec32 load32(const void* p, bool aligned32) {
  Vec32 v;
  if (!aligned32) {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                 "=r"(v.w[7])
               : "l"(p));
  return v;
}

template <bool BF>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (BF) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <bool BF>
__device__ __forceinline__ float2 widen(uint32_t w) {
  if constexpr (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}
__device__ __forceinline__ uint32_t e4m3_code(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
// The group's 16 values x / d as codes: fast, or by the plain division.
template <bool BF, bool FAST>
__device__ __forceinline__ uint2 codes_of(const Vec32& x, float d, float r) {
  uint32_t c[2];
  const unsigned long long r2 = f2_pack(r, r), nd2 = f2_pack(-d, -d);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = widen<BF>(x.w[4 * h + i]);
      if constexpr (FAST) {
        const unsigned long long xx = f2_pack(v.x, v.y), q0 = f2_mul(xx, r2), q1 = f2_fma(f2_fma(q0, nd2, xx), r2, q0);
        q[2 * i] = f2_lo(q1);
        q[2 * i + 1] = f2_hi(q1);
      } else {  // (beyond 8 d nothing changes the code, and infinities would)
        q[2 * i] = d > 0.f ? __fdiv_rn(fminf(fabsf(v.x), 8.f * d), d) : 0.f;
        q[2 * i + 1] = d > 0.f ? __fdiv_rn(fminf(fabsf(v.y), 8.f * d), d) : 0.f;
      }
      // (the sign of a zero too)
      q[2 * i] = copysignf(q[2 * i], v.x);
      q[2 * i + 1] = copysignf(q[2 * i + 1], v.y);
    }
    c[h] = float_to_e2m1x8(q);
  }
  return make_uint2(c[0], c[1]);
}

template <bool BF>
__device__ __forceinline__ void quantise(const Vec32& x, float scale, float scale6, float rcp6, bool fast, uint8_t* codes,
                                         uint8_t* sf) {
  uint32_t m2 = x.w[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m2 = max2_nan<BF>(m2, x.w[i] & 0x7fff7fffu);
  const float2 m = widen<BF>(m2);
  const float amax = fmaxf(m.x, m.y);
  float t;  // amax / (6 scale)
  if (fast) {
    const float q0 = amax * rcp6;
    t = fmaf(fmaf(-q0, scale6, amax), rcp6, q0);
    if (!(amax < scale6 * 512.f)) t = INFINITY;  // (at its end anyway; q0 can overflow there)
  } else {
    t = __fdiv_rn(amax, scale6);
  }
  uint32_t s = e4m3_code(t);
  const float d = e4m3_value(s) * scale;
  uint2 c;
  if (m.x != m.x || m.y != m.y) {
    s = 0x7f;
    c = make_uint2(0u, 0u);
  } else if (fast && s != 0x7e) {  // (a scale below its end: quotients up to 7, finite values)
    c = codes_of<BF, true>(x, d, d > 0.f ? __frcp_rn(d) : 0.f);
  } else {
    c = codes_of<BF, false>(x, d, 0.f);
  }
  *reinterpret_cast<uint2*>(codes) = c;
  *sf = static_cast<uint8_t>(s);
}

template <bool BF>
__global__ void __launch_bounds__(kThreads) write_fp4_kernel(const WriteArgs a) {
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < a.items; i += step) {
    const long long t = i / a.groups;
    const int gi = static_cast<int>(i - t * a.groups), h = gi / a.head_groups, gg = gi - h * a.head_groups;
    const Vec32 k = load32(a.k_new + i * 32, a.aligned32), v = load32(a.v_new + i * 32, a.aligned32);
    const int64_t slot = __ldg(a.slots + t);
    if (slot < 0) continue;  // padding token
    if (slot >= a.num_slots) {
      if (a.error_flag && gi == 0) atomicOr(a.error_flag, PD_DEVERR_SLOT);
      continue;
    }
    const uint32_t s32 = static_cast<uint32_t>(slot), blk = s32 / a.block_size, off = s32 - blk * a.block_size;
    const long long row = (static_cast<long long>(blk) * a.Hkv + h) * a.block_size + off;
    const long long at = row * a.head_groups + gg;
    quantise<BF>(k, a.k_scale, a.k_scale6, a.k_rcp6, a.fast != 0, a.k_codes + at * 8, a.k_sf + at);
    quantise<BF>(v, a.v_scale, a.v_scale6, a.v_rcp6, a.fast != 0, a.v_codes + at * 8, a.v_sf + at);
  }
}

bool misaligned(const void* p, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

}  // namespace
}  // namespace pd

using namespace pd;

extern "C" pd_status write_kv_cache_fp4(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                                        int num_tokens, void* k_cache, void* v_cache, void* k_block_scale,
                                        void* v_block_scale, const pd_dims* dims, uint32_t* error_flag, void* stream) {
  if (!dims) return PD_ERR_NULL;
  const pd_dims& d = *dims;
  if (num_tokens < 0 || d.Hkv < 1 || d.D < 16 || d.D % 16 != 0 || d.block_size < 1 || d.num_blocks < 0)
    return PD_ERR_SHAPE;
  if (d.kv_dtype != PD_KV_FP4 && d.kv_dtype != PD_KV_FP4_BF16) return PD_ERR_DTYPE;
  if (!(d.k_scale > 0.f) || !(d.v_scale > 0.f) || !std::isfinite(d.k_scale) || !std::isfinite(d.v_scale))
    return PD_ERR_SHAPE;
  const long long groups = static_cast<long long>(d.Hkv) * (d.D / 16);
  if (groups > 0x7fffffffll || static_cast<long long>(d.num_blocks) * d.block_size > 0x7fffffffll)
    return PD_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PD_OK;
  if (!k_new || !v_new || !slot_mapping || !k_cache || !v_cache || !k_block_scale || !v_block_scale) return PD_ERR_NULL;
  if (misaligned(k_new, 15) || misaligned(v_new, 15) || misaligned(k_cache, 7) || misaligned(v_cache, 7) ||
      misaligned(slot_mapping, 7) || misaligned(error_flag, 3))
    return PD_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    return PD_ERR_CUDA;
  auto moderate = [](float x) { return x >= 0x1p-60f && x <= 0x1p60f; };
  const float k6 = 6.f * d.k_scale, v6 = 6.f * d.v_scale;
  WriteArgs a{static_cast<const uint8_t*>(k_new), static_cast<const uint8_t*>(v_new), slot_mapping,
              static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), static_cast<uint8_t*>(k_block_scale),
              static_cast<uint8_t*>(v_block_scale), error_flag, num_tokens * groups,
              static_cast<long long>(d.num_blocks) * d.block_size, static_cast<int>(groups), d.D / 16, d.Hkv,
              d.block_size, d.k_scale, d.v_scale, k6, v6, 1.f / k6, 1.f / v6,
              !misaligned(k_new, 31) && !misaligned(v_new, 31), moderate(d.k_scale) && moderate(d.v_scale) ? 1 : 0};
  const long long want = (a.items + kThreads - 1) / kThreads, cap = static_cast<long long>(sms) * 64;
  const unsigned grid = static_cast<unsigned>(want < cap ? want : cap);
  auto s = static_cast<cudaStream_t>(stream);
  if (d.kv_dtype == PD_KV_FP4_BF16) write_fp4_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else write_fp4_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? PD_OK : PD_ERR_CUDA;
}
