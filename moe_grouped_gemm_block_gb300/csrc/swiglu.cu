// swiglu.cu -- the gated activation between an expert's two matrix products, quantised for the second one, and its
// gradient.
//
//     h = g s(g) u,  s(g) = 1 / (1 + e^-g)        (a row of the first product is g [F], then u [F])
//     e4m3 of h in 1 x 128 blocks: scale = amax / 448, code = e4m3(h / scale), each quotient rounded as the quantisers' of
//     unfused rows
//     dg = dh u s (1 + g (1 - s)),  du = dh g s
//
// Everything is fp32 until the one rounding of a result.  Bound by memory: forward 4 bytes read and 1 written a value
// (3 with h in bf16), backward 6 read and 4 written (6).  Device times, and the share of the copy rate:
//   33024 x 4096: 116 us (86%), with h 157 (89%), backward with h 247 (96%);  64 rows of 32 experts, masked: 4.0
// Two or four blocks of 128 a group at once were slower (123 and 157 us without h).

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kGluThreads = 256;
constexpr int kGluPerSm = 8;
constexpr int kGluGroups = kGluThreads / 16;  // 16 lanes take a block of 128 values, 8 each

struct GluArgs {
  const __nv_bfloat16* gu;
  const __nv_bfloat16* dh;
  __nv_bfloat16* h;
  __nv_bfloat16* dgu;
  uint8_t* q;
  float* sA;
  const int32_t* counts;
  int64_t ldgu, lddh, ldh, lddgu, ldq, ld_sa;
  uint32_t M, KB, cap;
  int32_t F;
};

// s(g) = 1 / (1 + e^-g) of two gates.  A gate has 8 significant bits and the first part of log2(e) 16, so that the exponent
// t of e^-g = 2^t e^(g c) is exact; of e^(g c), at most 2^-11 from 1, the first two terms.  So s is off by 8 u of itself
// (u = 2^-24: exponential 4, product and sum 1 each, reciprocal 2), and by up to 1.5 more where g nears -87; 0 where below
// 2^-126 (g < -87.3).  The library's exponential and a rounded reciprocal took 198 us (33024 x 4096 without h).
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 sigmoid(float2 g) {
  const float2 t = __fmul2_rn(g, both(-0x1.7154p+0f)), c = __fmul2_rn(g, both(-4.888495e-6f));
  float2 e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  const float2 d = __fadd2_rn(__ffma2_rn(e, c, e), both(1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return r;
}

template <bool MASKED>
__global__ void __launch_bounds__(kGluThreads, kGluPerSm) swiglu_kernel(const GluArgs a) {
  const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
  uint32_t M = a.M;
  int64_t row0 = 0;
  if (MASKED) {
    const int32_t c = __ldg(a.counts + blockIdx.y);
    M = c < 0 ? 0u : min(static_cast<uint32_t>(c), a.cap);
    row0 = static_cast<int64_t>(blockIdx.y) * a.cap;
  }
  // a CTA's groups take the same 128 columns of neighbouring rows, so that their scales lie side by side
  const uint32_t items = (M + kGluGroups - 1) / kGluGroups * a.KB;
  for (uint32_t i = blockIdx.x; i < items; i += gridDim.x) {
    const uint32_t kb = i % a.KB, m = i / a.KB * kGluGroups + group;
    const int col = static_cast<int>(kb) * 128 + lane * 8;
    if (m >= M) continue;  // (the same for a group's lanes)
    const int64_t row = row0 + m;
    float h[8] = {};
    if (col < a.F) {
      Raw8<__nv_bfloat16> rg, ru;
      const __nv_bfloat16* p = a.gu + row * a.ldgu + col;
      rg.load_stream(p);
      ru.load_stream(p + a.F);
      float2 g[4], u[4];
      rg.get(g);
      ru.get(u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __fmul2_rn(__fmul2_rn(g[j], sigmoid(g[j])), u[j]);
        h[2 * j] = p.x, h[2 * j + 1] = p.y;
      }
      if (a.h) store8_stream(a.h + row * a.ldh + col, h);
    }
    if (!a.q) continue;
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(h[j]));
    const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, off));
    // The scale is the rounded top / 448, the codes are those of the rounded quotients h / s.  Each by a product and a step on
    // its exact remainder (Markstein), where every remainder that can move a code is in the normal range; else (top
    // below 2^-60, or infinite) by divisions.  (A product with 1 / s alone: 114 us without h in place of 116.)
    float s, y[8];
    if (top >= 0x1p-60f && top < INFINITY) {
      s = top * (1.0f / 448.0f);
      s = fmaf(fmaf(-448.0f, s, top), 1.0f / 448.0f, s);
      float inv;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
      inv = fmaf(inv, fmaf(-s, inv, 1.0f), inv);
      const float2 inv2 = make_float2(inv, inv), minus = make_float2(-s, -s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = make_float2(h[2 * j], h[2 * j + 1]), first = __fmul2_rn(x, inv2);
        const float2 quotient = __ffma2_rn(__ffma2_rn(first, minus, x), inv2, first);
        y[2 * j] = quotient.x, y[2 * j + 1] = quotient.y;
      }
    } else {
      s = __fdiv_rn(top, 448.0f);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = s != 0.0f ? __fdiv_rn(h[j], s) : h[j] == h[j] ? 0.0f : h[j];  // (what is no number stays)
    }
    uint16_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = cvt_e4m3x2(y[2 * j + 1], y[2 * j]);
    *reinterpret_cast<uint2*>(a.q + row * a.ldq + col) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (lane == 0) a.sA[kb * a.ld_sa + row] = s;
  }
}

__global__ void __launch_bounds__(kGluThreads) swiglu_backward_kernel(const GluArgs a) {
  const uint32_t C = static_cast<uint32_t>(a.F) / 8;
  const uint32_t items = a.M * C;
  for (uint32_t i = blockIdx.x * kGluThreads + threadIdx.x; i < items; i += gridDim.x * kGluThreads) {
    const int64_t m = i / C;
    const int col = static_cast<int>(i % C) * 8;
    Raw8<__nv_bfloat16> rg, ru, rd;
    rg.load_stream(a.gu + m * a.ldgu + col);
    ru.load_stream(a.gu + m * a.ldgu + a.F + col);
    rd.load_stream(a.dh + m * a.lddh + col);
    float2 g2[4], u2[4], d2[4];
    rg.get(g2);
    ru.get(u2);
    rd.get(d2);
    float dg[8], du[8], h[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 s = sigmoid(g2[j]), act = __fmul2_rn(g2[j], s), p = __fmul2_rn(act, u2[j]), q = __fmul2_rn(d2[j], act);
      const float2 rest = __ffma2_rn(s, both(-1.0f), both(1.0f)), slope = __ffma2_rn(g2[j], rest, both(1.0f));
      const float2 r = __fmul2_rn(__fmul2_rn(__fmul2_rn(d2[j], u2[j]), s), slope);
      h[2 * j] = p.x, h[2 * j + 1] = p.y;
      dg[2 * j] = r.x, dg[2 * j + 1] = r.y;
      du[2 * j] = q.x, du[2 * j + 1] = q.y;
    }
    store8_stream(a.dgu + m * a.lddgu + col, dg);
    store8_stream(a.dgu + m * a.lddgu + a.F + col, du);
    if (a.h) store8_stream(a.h + m * a.ldh + col, h);
  }
}

unsigned ctas(int64_t work, int64_t per, const DeviceInfo* dev, int per_sm) {
  return static_cast<unsigned>(std::min<int64_t>((work + per - 1) / per, int64_t{1} * dev->sm_count * per_sm));
}

bool bad_rows(const void* p, int64_t ld) { return !aligned16(p) || ld % 8 != 0; }

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8_swiglu_quantize_1x128(const void* gu, int64_t M, int64_t F, int64_t ldgu, void* q, int64_t ldq,
                                         float* sA, int64_t ld_sa, void* h, int64_t ldh, void* stream) {
  if (M < 0 || F <= 0 || F % 8 != 0 || F > (1 << 29) || M > 0x7FFFFFFF || ldgu < 2 * F || (q && M && !sA) ||
      (q && (F % 128 != 0 || ldq < F || ld_sa < M)) || (h && ldh < F) || M * ((F + 127) / 128) >= (int64_t{1} << 31))
    return FP8G_ERR_INVALID_ARG;
  if (M == 0) return FP8G_OK;
  if (!gu || (!q && !h)) return FP8G_ERR_INVALID_ARG;
  if (bad_rows(gu, ldgu) || (h && bad_rows(h, ldh)) || (q && (!aligned16(q) || !aligned16(sA) || ldq % 16 || ld_sa % 4)))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  const int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  GluArgs a{};
  a.gu = static_cast<const __nv_bfloat16*>(gu), a.ldgu = ldgu;
  a.h = static_cast<__nv_bfloat16*>(h), a.ldh = ldh;
  a.q = static_cast<uint8_t*>(q), a.ldq = ldq, a.sA = sA, a.ld_sa = ld_sa;
  a.M = static_cast<uint32_t>(M), a.KB = static_cast<uint32_t>((F + 127) / 128), a.F = static_cast<int32_t>(F);
  swiglu_kernel<false><<<ctas((M + kGluGroups - 1) / kGluGroups * a.KB, 1, dev, kGluPerSm), kGluThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

extern "C" int fp8_swiglu_quantize_1x128_masked(const void* gu, int32_t E, int64_t cap, int64_t F,
                                                const int32_t* masked_m, void* q, float* sA, int64_t ld_sa,
                                                void* stream) {
  if (E < 1 || E > 65535 || cap < 0 || cap > 0x7FFFFFFF || F <= 0 || F % 128 != 0 || F > (1 << 29) ||
      ld_sa < static_cast<int64_t>(E) * cap || static_cast<int64_t>(E) * cap > 0x7FFFFFFF ||
      static_cast<int64_t>(E) * cap * (F / 128) >= (int64_t{1} << 31))
    return FP8G_ERR_INVALID_ARG;
  if (cap == 0) return FP8G_OK;
  if (!gu || !q || !sA || !masked_m) return FP8G_ERR_INVALID_ARG;
  if (!aligned16(gu) || !aligned16(q) || !aligned16(sA) || ld_sa % 4 != 0 || !aligned_to(masked_m, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  const int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  GluArgs a{};
  a.gu = static_cast<const __nv_bfloat16*>(gu), a.ldgu = 2 * F;
  a.q = static_cast<uint8_t*>(q), a.ldq = F, a.sA = sA, a.ld_sa = ld_sa;
  a.counts = masked_m;
  a.cap = static_cast<uint32_t>(cap), a.KB = static_cast<uint32_t>(F / 128), a.F = static_cast<int32_t>(F);
  const unsigned bx = std::max(1u, std::min(ctas((cap + kGluGroups - 1) / kGluGroups * a.KB, 1, dev, kGluPerSm),
                                            static_cast<unsigned>((16 * dev->sm_count + E - 1) / E)));
  swiglu_kernel<true><<<dim3(bx, static_cast<unsigned>(E)), kGluThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

extern "C" int fp8g_swiglu_backward(const void* dh, int64_t lddh, const void* gu, int64_t M, int64_t F, int64_t ldgu,
                                    void* dgu, int64_t lddgu, void* h, int64_t ldh, void* stream) {
  if (M < 0 || F <= 0 || F % 8 != 0 || F > (1 << 29) || M > 0x7FFFFFFF || M * (F / 8) >= (int64_t{1} << 31) ||
      lddh < F || ldgu < 2 * F || lddgu < 2 * F || (h && ldh < F))
    return FP8G_ERR_INVALID_ARG;
  if (M == 0) return FP8G_OK;
  if (!dh || !gu || !dgu || (dgu == gu && M > 1 && lddgu != ldgu)) return FP8G_ERR_INVALID_ARG;
  if (bad_rows(dh, lddh) || bad_rows(gu, ldgu) || bad_rows(dgu, lddgu) || (h && bad_rows(h, ldh)))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  const int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  GluArgs a{};
  a.dh = static_cast<const __nv_bfloat16*>(dh), a.lddh = lddh;
  a.gu = static_cast<const __nv_bfloat16*>(gu), a.ldgu = ldgu;
  a.dgu = static_cast<__nv_bfloat16*>(dgu), a.lddgu = lddgu;
  a.h = static_cast<__nv_bfloat16*>(h), a.ldh = ldh;
  a.M = static_cast<uint32_t>(M), a.F = static_cast<int32_t>(F);
  swiglu_backward_kernel<<<ctas(M * (F / 8), kGluThreads, dev, 8), kGluThreads, 0,
                           static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}
