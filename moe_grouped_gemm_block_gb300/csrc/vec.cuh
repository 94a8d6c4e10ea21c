// vec.cuh -- loads and stores of bf16 and fp32 rows and warp / CTA sums, shared by the kernels that
// work on unquantised tensors (layer norm, the MoE gate and combine, gradient clipping).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace fp8g {

inline bool aligned_to(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// A value of a tensor that the kernel only reads and whose type is known only at run time (bit 0 of `kind`).
__device__ __forceinline__ float load_any(const void* p, int32_t kind, int64_t i) {
  return kind & FP8G_F32 ? __ldg(static_cast<const float*>(p) + i)
                         : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}

// Eight values at a time, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// The same for results that the caller's next kernel reads, not this one: they need not stay in the near caches.
__device__ __forceinline__ void store8_stream(__nv_bfloat16* p, const float (&f)[8]) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])));
}
__device__ __forceinline__ void store8_stream(float* p, const float (&f)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
  __stcs(reinterpret_cast<float4*>(p + 4), make_float4(f[4], f[5], f[6], f[7]));
}

// Eight values as they lie in memory, and as four pairs for the two-wide fp32 instructions.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_stream(const __nv_bfloat16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void set(const __nv_bfloat16 (&f)[8]) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(f);
    v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  // value j by value j from memory where the mask has it, zero elsewhere
  __device__ __forceinline__ void gather(const __nv_bfloat16* p, uint32_t mask) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = mask >> j & 1u ? h[j] : 0u;
    v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  // keeps the values that the mask has, zeroes the others
  __device__ __forceinline__ void keep(uint32_t mask) {
    uint32_t* w = &v.x;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] &= (mask >> (2 * j) & 1u ? 0xFFFFu : 0u) | (mask >> (2 * j + 1) & 1u ? 0xFFFF0000u : 0u);
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void load_stream(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void gather(const float* p, uint32_t mask) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = mask >> j & 1u ? p[j] : 0.0f;
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void keep(uint32_t mask) {
    a.x = mask & 1u ? a.x : 0.0f, a.y = mask & 2u ? a.y : 0.0f;
    a.z = mask & 4u ? a.z : 0.0f, a.w = mask & 8u ? a.w : 0.0f;
    b.x = mask & 16u ? b.x : 0.0f, b.y = mask & 32u ? b.y : 0.0f;
    b.z = mask & 64u ? b.z : 0.0f, b.w = mask & 128u ? b.w : 0.0f;
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
  }
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sums of NV values over a CTA of WARPS warps, the same in every thread.  `red` holds 2 * WARPS * NV floats:
// calls alternate between its halves (`phase`), so one barrier a call is enough.
template <int WARPS, int NV>
__device__ __forceinline__ void cta_sum(float (&v)[NV], float* red, int phase) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = warp_sum(v[i]);
  if constexpr (WARPS > 1) {
    float* r = red + (phase & 1) * WARPS * NV;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[warp * NV + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) s += r[w * NV + i];
      v[i] = s;
    }
  }
}

}  // namespace fp8g
