// adamw.cu -- one AdamW step over many tensors, with states in 32 or in 8 bits.
//
//     g = coef grad,   coef = min(1, max_norm / (norm + norm_eps))  (1 without a norm)
//     m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,   c1 = 1 - b1^t,   c2 = 1 - b2^t
//     p = p - lr (decay p + (m / c1) / (sqrt(v / c2) + eps))
//
// in fp32 whatever the types; p is the tensor itself or its fp32 master copy, whose rounding the tensor then gets.
//
// States in 8 bits are e4m3 codes with one fp32 scale, amax (1 / 448), for each 128 consecutive values, as the quantisers
// of the GEMMs' operands have them: m itself, and the root of v (e4m3's range, 2^17, is then that of the gradients and
// not of their squares).  The step itself uses the new m and v before they are rounded.  Two things differ from a GEMM
// operand's rounding.  To the nearest, a state that changes by less than half a step (3 to 6% of itself) at a time would
// never change: with b2 = 0.999 a root follows no fall of its gradients.  So a value goes up where its place between
// two codes and a number in [0, 1) are 1 or more together; the numbers run through an evenly spread sequence in the
// steps and the places of the tensor, (place A + step B) mod 2^32, so that a state is right on the average of a few
// steps and a call is repeatable.  And a root that is not 0 keeps the lowest code where it would round to 0: it is then
// too large, which makes a step too small, never too large.  A block whose largest is below 2^-60 becomes 0.
//
// Bound by memory with states in 32 bits and in 8 with masters; without them by that and some 60 instructions a value.  117M
// values in one tensor, device times and the share of the copy rate: 32 bits, fp32 with bf16 gradients 477 us (94%); 8 bits
// with masters 321 (87%), without 260 (67%).  1M values: 9.5 and 11 us, of which the step's launch before is 2.
#include <algorithm>
#include <cmath>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kAdamThreads = 256;
constexpr int adam_per_sm(int bits) { return bits == 32 ? 3 : 4; }  // resident CTAs an SM
constexpr int kAdamPass = kAdamThreads * 8;  // values a CTA takes at once: 16 lanes a block of 128, 8 values each
constexpr int32_t kAdamMaxTensors = 1 << 20;
constexpr int64_t kAdamMaxValues = int64_t{1} << 40;
constexpr uint32_t kPlaceStep = 0xC13FA9A9u, kTimeStep = 0x91E10DA5u;  // 2^32 / r and 2^32 / r^2, r^3 = r + 1
constexpr uint32_t kRootShift = 0x80000000u;

enum : uint32_t { kParamF32 = 1, kGradF32 = 2, kMaster = 4, kVectors = 8 };

struct AdamTensor {
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int64_t numel;
  float decay;
  uint32_t kind;
};
template <int CAP>
struct AdamTable {
  AdamTensor t[CAP];
  uint32_t end[CAP];  // chunks of the tensors up to and with this one
  int32_t n;
};
constexpr int kAdamCap = 384;  // tensors a launch
constexpr int kAdamFew = 64;   // of a smaller table: 1 tensor 4.1 instead of 5.0 us, 64 8.0 instead of 8.7 (one of 160: 0.1 to 0.3)
static_assert(sizeof(AdamTable<kAdamCap>) <= 32000, "kernel arguments hold 32764 bytes");

struct AdamHyper {
  float b1, nb1, b2, nb2, eps;  // nb = 1 - b, rounded once
};
// What every CTA needs of the step, made by one thread (the powers in 64 bits).
struct AdamStep {
  float coef, lr, lr1, root2;  // lr, lr / c1, 1 / sqrt(c2)
  uint32_t time, skip;
};
static_assert(sizeof(AdamStep) <= 32, "");

// b^t by squaring: off by some t 2^-53 of itself, when it counts (the library's pow takes 6 us on this GPU's fp64).
__device__ __forceinline__ double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0 && r > 0.0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

// One warp; lane 0 has beta1's power, lane 1 beta2's.
__global__ void __launch_bounds__(32) adamw_step_kernel(const float* lr_dev, double lr, double b1, double b2, int64_t* step,
                                                        const float* norm, float max_norm, float norm_eps, AdamStep* out) {
  griddep_launch_dependents();
  AdamStep s{};
  s.coef = 1.0f;
  const int64_t t = *step + 1;
  float rate = static_cast<float>(lr);
  if (lr_dev) rate = *lr_dev;
  if (norm) {
    const float n = *norm;
    s.skip = isfinite(n) ? 0u : 1u;
    s.coef = fminf(1.0f, __fmul_rn(max_norm, __frcp_rn(n + norm_eps)));
  }
  const float c = static_cast<float>(1.0 - power(threadIdx.x ? b2 : b1, t)), c2 = __shfl_sync(0xffffffffu, c, 1);
  s.time = static_cast<uint32_t>(t);
  s.lr = rate;
  s.lr1 = __fdiv_rn(rate, c);
  s.root2 = __fdiv_rn(1.0f, __fsqrt_rn(c2));
  if (threadIdx.x == 0) {
    if (!s.skip) *step = t;
    *out = s;
  }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
// A sum of products that keeps their own roundings (a two-wide sum is joined with the products, whatever it is written as).
__device__ __forceinline__ float2 add_apart(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

// How a block of 128 values falls to 16 lanes: two fours a lane, 64 values apart, as vectors (lanes' fp32 accesses then lie
// side by side); in a block that is not whole, or off the vectors' boundaries, value by value, 16 apart.
template <bool FULL>
struct Places {
  int64_t first;  // of the lane, in the tensor
  int64_t n;      // values of the tensor
  __device__ __forceinline__ Places(int64_t block, int64_t numel) : first(block + (FULL ? 4 : 1) * (threadIdx.x & 15)), n(numel) {}
  static constexpr __device__ __forceinline__ int offset(int j) { return FULL ? (j & 3) + 64 * (j >> 2) : 16 * j; }
  __device__ __forceinline__ bool has(int j) const { return FULL || first + offset(j) < n; }
};
__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float* f) {
  const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
  f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
  f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4(float* p, const float* f) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* f) {
  __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3])));
}
template <typename T, bool FULL>
__device__ __forceinline__ void get8(const T* p, const Places<FULL>& at, float (&f)[8]) {
  p += at.first;
  if constexpr (FULL) {
    load4(p, f);
    load4(p + 64, f + 4);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = at.has(j) ? to_f32(p[at.offset(j)]) : 0.0f;
  }
}
template <typename T, bool FULL>
__device__ __forceinline__ void put8(T* p, const Places<FULL>& at, const float (&f)[8]) {
  p += at.first;
  if constexpr (FULL) {
    store4(p, f);
    store4(p + 64, f + 4);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at.has(j)) p[at.offset(j)] = from_f32<T>(f[j]);
  }
}

// The roots of eight values >= 0: an approximate one and a step of Heron's iteration on its residual (Markstein), which is
// the rounded root but for one value in some 2^20 (whose true root lies so near the middle between two floats); by the
// compiler's root where one of the eight is below the normal range or not finite.  (With that and its quotient for all,
// a branch in each, 117M values with 8-bit states took 479 us.)
// -> whether all are positive for sure.
__device__ __forceinline__ bool square_roots(const float2 (&v)[4], float2 (&root)[4]) {
  float lo = v[0].x, hi = v[0].x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    lo = fminf(lo, fminf(v[j].x, v[j].y));
    hi = fmaxf(hi, fmaxf(v[j].x, v[j].y));
  }
  if (lo >= 0x1p-126f && hi < INFINITY) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 r;
      asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v[j].x));
      asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v[j].y));
      const float2 s = mul2(v[j], r), minus = make_float2(-s.x, -s.y);
      root[j] = __ffma2_rn(__ffma2_rn(minus, s, v[j]), mul2(r, both(0.5f)), s);
    }
    return true;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) root[j] = make_float2(__fsqrt_rn(v[j].x), __fsqrt_rn(v[j].y));
    return false;
  }
}
__device__ __forceinline__ float2 quotient(float2 a, float2 b) {  // two units in the last place; b is normal
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(b.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(b.y));
  return mul2(a, r);
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void decode(const uint32_t (&w)[2], float scale, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    reinterpret_cast<float2(&)[4]>(f)[j] = mul2(e4m3x2_to_f32(w[j / 2] >> (16 * (j & 1))), both(scale));
}
__device__ __forceinline__ void get_codes(const uint8_t* p, const Places<false>& at, float scale, float (&f)[8]) {
  uint32_t w[2] = {0u, 0u};
  p += at.first;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (at.has(j)) w[j / 4] |= static_cast<uint32_t>(p[at.offset(j)]) << (8 * (j & 3));
  decode(w, scale, f);
}
// The codes of a block that 16 lanes hold, and its scale (see above).  ROOT: what is not 0 gets no 0; positive: none is 0.
template <bool ROOT, bool FULL>
__device__ __forceinline__ void put_codes(uint8_t* p, float* scale, const Places<FULL>& at, uint32_t time, const float (&f)[8],
                                          bool positive = false) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[j]));
  const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, off));
  const bool live = top >= 0x1p-60f;
  const float inv = live ? __fmul_rn(448.0f, __frcp_rn(top)) : 0.0f;
  if ((threadIdx.x & 15) == 0) *scale = live ? __fmul_rn(top, 1.0f / 448.0f) : 0.0f;
  const uint32_t first = static_cast<uint32_t>(at.first) * kPlaceStep + time * kTimeStep + (ROOT ? kRootShift : 0u);
  const float lowest = live ? 0x1p-9f : 0.0f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // A code has 3 bits after the point, y 20 more: their sum with u carries into the code's or does not.  Below 2^-6
    // the codes are 2^-9 apart, as they are from 2^-6 to 2^-5: the sum with 2^-6 (what it cuts off is less than u's
    // last bit) has them at the same bits.
    const float2 x = make_float2(f[2 * j], f[2 * j + 1]);
    const float2 y = mul2(x, both(inv));
    float c[2] = {fabsf(y.x), fabsf(y.y)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float low = c[k] < 0x1p-6f ? 1.0f : 0.0f;
      const uint32_t u = (first + static_cast<uint32_t>(at.offset(2 * j + k)) * kPlaceStep) >> 12;
      c[k] = fmaf(low, -0x1p-6f, __uint_as_float((__float_as_uint(__fmaf_rz(low, 0x1p-6f, c[k])) + u) & 0xFFF00000u));
      const float own = k ? x.y : x.x;
      if (ROOT) c[k] = fmaxf(c[k], lowest);
      else c[k] = copysignf(c[k], own);
      if (ROOT && !positive) c[k] = own == 0.0f ? 0.0f : c[k];
    }
    w[j / 2] |= static_cast<uint32_t>(cvt_e4m3x2(c[1], c[0])) << (16 * (j & 1));
  }
  p += at.first;
  if constexpr (FULL) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
    *reinterpret_cast<uint32_t*>(p + 64) = w[1];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at.has(j)) p[at.offset(j)] = static_cast<uint8_t>(w[j / 4] >> (8 * (j & 3)));
  }
}

// A thread's part of whole blocks with 8-bit states, copied ahead into places of its own in its warp's (warps are at tensors
// of other types, whose places have other sizes): a block's arithmetic is long, and
// so few bytes of it are on their way at once that the loads' latency would show (117M values with masters: 335 us in place
// of 321).
constexpr int kAdamStages = 2;
constexpr int kAdamPlaces = 2 * 16 + 2 * 16 + 4 * 4 + 2 * 4;  // bytes of a thread and stage, at most
template <int BYTES>
__device__ __forceinline__ void copy_ahead(uint32_t to, const void* from) {
  if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void load_place(uint32_t from, float* f) {
  if constexpr (BYTES == 16) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(from) : "memory");
  } else {
    uint32_t a, b;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(from) : "memory");
    f[0] = __uint_as_float(a << 16), f[1] = __uint_as_float(a & 0xFFFF0000u);
    f[2] = __uint_as_float(b << 16), f[3] = __uint_as_float(b & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t load_word(uint32_t from) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(from) : "memory");
  return v;
}
template <typename T, typename TG>  // T: of what the step starts from, the param or its master copy
struct Ahead {
  static constexpr int kP = 4 * static_cast<int>(sizeof(T)), kG = 4 * static_cast<int>(sizeof(TG));
  static constexpr uint32_t kGrads = 2 * kP * 32, kCodes = kGrads + 2 * kG * 32;
  uint32_t places;  // of the warp
  __device__ __forceinline__ void copy(int stage, const AdamTensor& t, const void* from, int64_t block) const {
    const int64_t first = block + 4 * (threadIdx.x & 15);
    const uint32_t at = places + stage * (kAdamPlaces * kAdamThreads), x = threadIdx.x & 31;
    const T* p = static_cast<const T*>(from) + first;
    const TG* g = static_cast<const TG*>(t.grad) + first;
    const uint8_t *m = static_cast<const uint8_t*>(t.m) + first, *v = static_cast<const uint8_t*>(t.v) + first;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      copy_ahead<kP>(at + (i * 32 + x) * kP, p + 64 * i);
      copy_ahead<kG>(at + kGrads + (i * 32 + x) * kG, g + 64 * i);
      copy_ahead<4>(at + kCodes + (i * 32 + x) * 4, m + 64 * i);
      copy_ahead<4>(at + kCodes + ((2 + i) * 32 + x) * 4, v + 64 * i);
    }
    copy_ahead<4>(at + kCodes + (4 * 32 + x) * 4, t.m_scale + (block >> 7));
    copy_ahead<4>(at + kCodes + (5 * 32 + x) * 4, t.v_scale + (block >> 7));
  }
  __device__ __forceinline__ void load(int stage, float (&p)[8], float (&g)[8], float (&m)[8], float (&v)[8]) const {
    const uint32_t at = places + stage * (kAdamPlaces * kAdamThreads), x = threadIdx.x & 31;
    uint32_t w[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      load_place<kP>(at + (i * 32 + x) * kP, p + 4 * i);
      load_place<kG>(at + kGrads + (i * 32 + x) * kG, g + 4 * i);
      w[0][i] = load_word(at + kCodes + (i * 32 + x) * 4);
      w[1][i] = load_word(at + kCodes + ((2 + i) * 32 + x) * 4);
    }
    decode(w[0], __uint_as_float(load_word(at + kCodes + (4 * 32 + x) * 4)), m);
    decode(w[1], __uint_as_float(load_word(at + kCodes + (5 * 32 + x) * 4)), v);
  }
};

// The step of a lane's part of the block of 128 values of tensor t that starts at `block`.
template <int BITS, typename TP, typename TG, bool MASTER, bool FULL>
__device__ __forceinline__ void adam_apply(const AdamTensor& t, const AdamHyper& h, const AdamStep& s, int64_t block,
                                           const Places<FULL>& at, float (&p)[8], float (&g)[8], float (&m)[8], float (&v)[8]) {
  float2 root[4];
  auto& p2 = reinterpret_cast<float2(&)[4]>(p);
  auto& g2 = reinterpret_cast<float2(&)[4]>(g);
  auto& m2 = reinterpret_cast<float2(&)[4]>(m);
  auto& v2 = reinterpret_cast<float2(&)[4]>(v);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // (products and sums rounded one by one: the codes' rounding then is that of the formulas as they stand)
    if (BITS == 8) v2[j] = mul2(v2[j], v2[j]);
    const float2 gj = mul2(g2[j], both(s.coef));
    m2[j] = add_apart(mul2(both(h.b1), m2[j]), mul2(both(h.nb1), gj));
    v2[j] = add_apart(mul2(both(h.b2), v2[j]), mul2(mul2(both(h.nb2), gj), gj));
  }
  const bool positive = square_roots(v2, root);
  const float shrink = -s.lr * t.decay;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 to = quotient(m2[j], __ffma2_rn(root[j], both(s.root2), both(h.eps)));
    p2[j] = __ffma2_rn(both(-s.lr1), to, __ffma2_rn(both(shrink), p2[j], p2[j]));
    if (BITS == 8) v2[j] = root[j];
  }
  put8(static_cast<TP*>(t.param), at, p);
  if constexpr (MASTER) put8(t.master, at, p);
  if constexpr (BITS == 32) {
    put8(static_cast<float*>(t.m), at, m);
    put8(static_cast<float*>(t.v), at, v);
  } else {
    put_codes<false>(static_cast<uint8_t*>(t.m), t.m_scale + (block >> 7), at, s.time, m);
    put_codes<true>(static_cast<uint8_t*>(t.v), t.v_scale + (block >> 7), at, s.time, v, positive);
  }
}

template <int BITS, typename TP, typename TG, bool MASTER, bool FULL>
__device__ __forceinline__ void adam_values(const AdamTensor& t, const AdamHyper& h, const AdamStep& s, int64_t block) {
  const Places<FULL> at(block, t.numel);
  float p[8], g[8], m[8], v[8];
  get8(static_cast<const TG*>(t.grad), at, g);
  if constexpr (MASTER) get8(t.master, at, p);
  else get8(static_cast<const TP*>(t.param), at, p);
  if constexpr (BITS == 32) {
    get8(static_cast<const float*>(t.m), at, m);
    get8(static_cast<const float*>(t.v), at, v);
  } else {
    get_codes(static_cast<const uint8_t*>(t.m), at, t.m_scale[block >> 7], m);
    get_codes(static_cast<const uint8_t*>(t.v), at, t.v_scale[block >> 7], v);
  }
  adam_apply<BITS, TP, TG, MASTER, FULL>(t, h, s, block, at, p, g, m, v);
}

// The blocks of tensor t from `block` on, `step` values apart.
template <int BITS, typename TP, typename TG, bool MASTER>
__device__ __forceinline__ void adam_blocks(const AdamTensor& t, const AdamHyper& h, const AdamStep& s, int64_t block, int64_t step,
                                            uint32_t places) {
  const int64_t whole = t.kind & kVectors ? t.numel - 128 : -1;  // the last place where a whole block may start
  if constexpr (BITS == 8) {
    const Ahead<std::conditional_t<MASTER, float, TP>, TG> ahead{places};
    const void* from = MASTER ? static_cast<const void*>(t.master) : t.param;
    int64_t next = block;
    auto bring = [&](int stage) {
      if (next <= whole) ahead.copy(stage, t, from, next);
      next += step;
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAdamStages; ++i) bring(i);
    for (int stage = 0; block <= whole; block += step) {
      float p[8], g[8], m[8], v[8];
      asm volatile("cp.async.wait_group %0;" ::"n"(kAdamStages - 1) : "memory");
      ahead.load(stage, p, g, m, v);
      bring(stage);
      stage = stage + 1 == kAdamStages ? 0 : stage + 1;
      adam_apply<BITS, TP, TG, MASTER, true>(t, h, s, block, Places<true>(block, t.numel), p, g, m, v);
    }
  } else {
    for (; block <= whole; block += step) adam_values<BITS, TP, TG, MASTER, true>(t, h, s, block);
  }
  for (; block < t.numel; block += step) adam_values<BITS, TP, TG, MASTER, false>(t, h, s, block);
}

// The tensor of chunk c, from the i-th on.
template <int CAP>
__device__ __forceinline__ int adam_find(const AdamTable<CAP>& tab, uint32_t c, int i) {
  if (c < tab.end[i]) return i;
  int lo = i + 1, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c < tab.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}
// Brings the CTA's first chunk into L2, a line of 128 bytes a thread and matrix (memory cold: 150 tensors of 10000 values
// 18.9 -> 16.9 us, 16M values 82.4 -> 80.8).
template <int BITS, int CAP>
__device__ __forceinline__ void adam_prefetch(const AdamTable<CAP>& tab) {
  const int i = adam_find(tab, blockIdx.x, 0);
  const AdamTensor& t = tab.t[i];
  const int64_t first = static_cast<int64_t>(blockIdx.x - (i ? tab.end[i - 1] : 0u)) * kAdamPass;
  const int64_t n = min(t.numel - first, static_cast<int64_t>(kAdamPass));
  auto bring = [&](const void* p, int size) {
    const int64_t at = static_cast<int64_t>(threadIdx.x) * 128;
    if (p && at < n * size) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + first * size + at));
  };
  bring(t.grad, t.kind & kGradF32 ? 4 : 2);
  bring(t.master ? t.master : t.param, t.kind & (kMaster | kParamF32) ? 4 : 2);
  bring(t.m, BITS / 8);
  bring(t.v, BITS / 8);
}

// Resident CTAs walk over the chunks of 2048 values (a CTA a chunk: 16M values took 100 us, most of it the CTAs' starts).
template <int CAP, int BITS>
__global__ void __launch_bounds__(kAdamThreads, adam_per_sm(BITS)) adamw_kernel(const __grid_constant__ AdamTable<CAP> tab,
                                                                         const AdamHyper h,
                                                                         const AdamStep* __restrict__ step) {
  __shared__ __align__(16) unsigned char shared[BITS == 8 ? kAdamStages * kAdamPlaces * kAdamThreads : 16];
  const uint32_t places = smem_u32(shared) + (threadIdx.x >> 5) * (kAdamPlaces * 32), chunks = tab.end[tab.n - 1];
  adam_prefetch<BITS>(tab);  // (under the step's end: what was before that is complete)
  griddep_wait();
  AdamStep s;
  s.coef = __ldcg(&step->coef), s.lr = __ldcg(&step->lr), s.lr1 = __ldcg(&step->lr1), s.root2 = __ldcg(&step->root2);
  s.time = __ldcg(&step->time), s.skip = __ldcg(&step->skip);
  if (s.skip) return;
  int i = 0;
  const int64_t step_size = static_cast<int64_t>(gridDim.x) * kAdamPass;
  for (uint32_t c = blockIdx.x; c < chunks;) {
    i = adam_find(tab, c, i);
    const AdamTensor& t = tab.t[i];
    const int64_t block = static_cast<int64_t>(c - (i ? tab.end[i - 1] : 0u)) * kAdamPass + (threadIdx.x >> 4) * 128;
    c += (tab.end[i] - c + gridDim.x - 1) / gridDim.x * gridDim.x;  // the CTA's first chunk past this tensor's
    switch (t.kind & (kParamF32 | kGradF32 | kMaster)) {
      case 0: adam_blocks<BITS, __nv_bfloat16, __nv_bfloat16, false>(t, h, s, block, step_size, places); break;
      case kGradF32: adam_blocks<BITS, __nv_bfloat16, float, false>(t, h, s, block, step_size, places); break;
      case kMaster: adam_blocks<BITS, __nv_bfloat16, __nv_bfloat16, true>(t, h, s, block, step_size, places); break;
      case kMaster | kGradF32: adam_blocks<BITS, __nv_bfloat16, float, true>(t, h, s, block, step_size, places); break;
      case kParamF32: adam_blocks<BITS, float, __nv_bfloat16, false>(t, h, s, block, step_size, places); break;
      default: adam_blocks<BITS, float, float, false>(t, h, s, block, step_size, places); break;
    }
    __syncwarp();  // (the next tensor has other places)
  }
}

int check_adam(const fp8g_adamw_tensor* ts, int32_t n, int32_t bits) {
  if (n < 0 || n > kAdamMaxTensors || (n > 0 && !ts) || (bits != 8 && bits != 32)) return FP8G_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const fp8g_adamw_tensor& t = ts[i];
    if (t.numel < 0 || t.numel > kAdamMaxValues || !(t.weight_decay >= 0.0f) ||
        (t.param_dtype != FP8G_BF16 && t.param_dtype != FP8G_F32) ||
        (t.grad_dtype != FP8G_BF16 && t.grad_dtype != FP8G_F32) || (t.master && t.param_dtype != FP8G_BF16))
      return FP8G_ERR_INVALID_ARG;
    total += t.numel;
    if (total > kAdamMaxValues) return FP8G_ERR_INVALID_ARG;
    if (t.numel == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (bits == 8 && (!t.m_scale || !t.v_scale))) return FP8G_ERR_INVALID_ARG;
    const uintptr_t state = bits == 32 ? 4 : 1;
    if (!aligned_to(t.param, t.param_dtype == FP8G_F32 ? 4 : 2) || !aligned_to(t.grad, t.grad_dtype == FP8G_F32 ? 4 : 2) ||
        !aligned_to(t.m, state) || !aligned_to(t.v, state) || !aligned_to(t.master, 4) ||
        (bits == 8 && (!aligned_to(t.m_scale, 4) || !aligned_to(t.v_scale, 4))))
      return FP8G_ERR_ALIGNMENT;
  }
  return FP8G_OK;
}

template <int CAP, int BITS>
int adamw_launch(const fp8g_adamw_tensor* ts, int32_t n, const AdamHyper& h, const AdamStep* step,
                 const DeviceInfo* dev, cudaStream_t s) {
  AdamTable<CAP> tab;
  const uintptr_t state = BITS == 32 ? 16 : 4;
  bool first = true;
  for (int32_t i = 0; i < n;) {
    tab.n = 0;
    uint64_t chunks = 0;
    for (; i < n && tab.n < CAP; ++i) {
      const fp8g_adamw_tensor& t = ts[i];
      if (t.numel == 0) continue;
      const bool vec = aligned16(t.param) && aligned16(t.grad) && aligned16(t.master) && aligned_to(t.m, state) &&
                       aligned_to(t.v, state);
      tab.t[tab.n] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.master, t.numel, t.weight_decay,
                      (t.param_dtype == FP8G_F32 ? kParamF32 : 0u) | (t.grad_dtype == FP8G_F32 ? kGradF32 : 0u) |
                          (t.master ? kMaster : 0u) | (vec ? kVectors : 0u)};
      chunks += static_cast<uint64_t>((t.numel + kAdamPass - 1) / kAdamPass);
      tab.end[tab.n++] = static_cast<uint32_t>(chunks);
    }
    if (tab.n == 0) break;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<uint64_t>(chunks, static_cast<uint64_t>(dev->sm_count) * adam_per_sm(BITS))));
    cfg.blockDim = dim3(kAdamThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = first ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    first = false;
    if (cudaLaunchKernelEx(&cfg, adamw_kernel<CAP, BITS>, tab, h, step) != cudaSuccess) {
      cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
  }
  return FP8G_OK;
}

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_adamw(const fp8g_adamw_tensor* tensors, int32_t n, int32_t state_bits, double lr, const float* lr_dev,
                          double beta1, double beta2, double eps, int64_t* step, const float* norm, float max_norm,
                          float norm_eps, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_adam(tensors, n, state_bits);
  if (st != FP8G_OK) return st;
  if (!(lr >= 0.0) || !std::isfinite(lr) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
      !(eps >= 1e-30) || !std::isfinite(eps) || !step || (norm && (!(max_norm >= 0.0f) || !(norm_eps >= 0.0f))) || !workspace ||
      workspace_bytes < FP8G_ADAMW_WORKSPACE)
    return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(step, 8) || !aligned_to(norm, 4) || !aligned_to(lr_dev, 4) || !aligned16(workspace))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8G_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  AdamStep* out = static_cast<AdamStep*>(workspace);
  adamw_step_kernel<<<1, 32, 0, s>>>(lr_dev, lr, beta1, beta2, step, norm, max_norm, norm_eps, out);
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  const AdamHyper h{static_cast<float>(beta1), static_cast<float>(1.0 - beta1), static_cast<float>(beta2),
                    static_cast<float>(1.0 - beta2), static_cast<float>(eps)};
  auto go = state_bits == 32 ? (n <= kAdamFew ? adamw_launch<kAdamFew, 32> : adamw_launch<kAdamCap, 32>)
                             : (n <= kAdamFew ? adamw_launch<kAdamFew, 8> : adamw_launch<kAdamCap, 8>);
  return go(tensors, n, h, out, dev, s);
}
