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
// e^(v - mx) for v <= mx, for a row's selected experts; the difference d first, which cannot overflow to anything but -inf.
// The exponent d log2(e) is rounded, to t: what e^d differs from 2^t by, e^(d - t ln 2), is multiplied in again, so the
// relative error stays near the 2^-22 of exp2_approx however far v lies below mx (65536 x 256 bf16: 37.9 us, without it
// 37.5).  d is held above -200, where the result is 0 anyway, so that the remainder of -inf is finite; a NaN stays one.
__device__ __forceinline__ float exp_below(float v, float mx) {
  constexpr float kLn2 = 0.693147182464599609375f, kLn2Rest = -1.9046542e-9f;  // their sum is ln 2
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(v - mx), "f"(-200.0f));
  const float t = d * 1.4426950408889634f, y = exp2_approx(t);
  return fmaf(y, fmaf(-t, kLn2Rest, fmaf(-t, kLn2, d)), y);
}
// exp_below for all of f, in place, and their sum, without the remainder: a result's relative error grows with the distance
// from the row's largest, (1.3 |d| + 4) 2^-24, which the sum, weighted by the results themselves, does not feel.  A choice
// for speed: with the remainder (two fused multiply-adds, and the clamp) 65536 x 256 forward takes 39.1 us instead of
// 37.7 (bf16) and 49.2 instead of 47.2 (fp32).
template <int H>
__device__ __forceinline__ float exp_below(float2 (&f)[H], float mx) {
  const float2 m = make_float2(-mx, -mx), k = make_float2(1.4426950408889634f, 1.4426950408889634f);
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < H; ++i) {
    const float2 d = __fmul2_rn(__fadd2_rn(f[i], m), k);
    f[i] = make_float2(exp2_approx(d.x), exp2_approx(d.y));
    s = __fadd2_rn(s, f[i]);
  }
  return s.x + s.y;
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
