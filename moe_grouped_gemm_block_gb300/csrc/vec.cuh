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

// A value of a tensor whose type is known only at run time (uniform over the launch).
__device__ __forceinline__ float load_any(const void* p, int32_t dtype, int64_t i) {
  return dtype == FP8G_F32 ? static_cast<const float*>(p)[i]
                           : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

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
