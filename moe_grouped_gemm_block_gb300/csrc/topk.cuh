// topk.cuh -- what the routers' kernels share: order keys, maxima and sums over the lanes of a row, a sorting network,
// rows of logits in registers.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "vec.cuh"

namespace fp8g {

// 2^x (relative error 2^-22; results below the normal range are 0).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float recip_approx(float x) {  // 1 / x to one unit in the last place
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The order of the selection as an unsigned integer: ascending in the value, NaN above everything (as a
// descending sort has it), -0 equal to +0 (the addition turns -0 into +0 and every NaN into the positive one).
// 0 is below every value's key: it stands for no logit.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// The same for two bf16 values in a word, 16 bits each.
__device__ __forceinline__ uint32_t order_key2(uint32_t w) {
  const __nv_bfloat162 z = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&w), __floats2bfloat162_rn(0.0f, 0.0f));
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&z);
  const uint32_t neg = u >> 15 & 0x00010001u;
  return u ^ ((neg << 16) - neg | 0x80008000u);
}

template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  if constexpr (LPR == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  }
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (LPR == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  } else {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  }
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// A sorting network for eight (19 exchanges, descending).
template <typename Exchange>
__device__ __forceinline__ void sort8(Exchange ex) {
  ex(0, 2), ex(1, 3), ex(4, 6), ex(5, 7);
  ex(0, 4), ex(1, 5), ex(2, 6), ex(3, 7);
  ex(0, 1), ex(2, 3), ex(4, 5), ex(6, 7);
  ex(2, 4), ex(3, 5);
  ex(1, 4), ex(3, 6);
  ex(1, 2), ex(3, 4), ex(5, 6);
}

// VPL logits of a row as they lie in memory; -inf past the row's end.
template <typename TL, int VPL>
struct Logits {
  Raw8<TL> raw[VPL / 8];
  // vec: the row's groups of 8 lie on 16-byte boundaries
  __device__ __forceinline__ void load(const TL* row, int base, int E, bool vec) {
#pragma unroll
    for (int v = 0; v < VPL / 8; ++v) {
      const int c = base + 8 * v;
      if (vec && c + 8 <= E) {
        raw[v].load(row + c);
      } else {
        TL f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < E ? row[c + i] : from_f32<TL>(-INFINITY);
        raw[v].set(f);
      }
    }
  }
  __device__ __forceinline__ void get(float2 (&f)[VPL / 2]) const {
#pragma unroll
    for (int v = 0; v < VPL / 8; ++v) raw[v].get(reinterpret_cast<float2(&)[4]>(f[4 * v]));
  }
};

}  // namespace fp8g
