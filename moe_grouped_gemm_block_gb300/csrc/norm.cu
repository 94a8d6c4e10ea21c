// norm.cu -- layer norm over the rows of a matrix and its gradients.
//
//     mu_m = mean_n x,   r_m = 1 / sqrt(mean_n (x - mu)^2 + eps),   y = (x - mu) r w + b
//     with h = (x - mu) r and g = dy w:
//     dx = r (g - mean_n g - h mean_n (g h)),   dw = sum_m dy h,   db = sum_m dy
//
// All sums are taken in fp32; the variance is the mean of the squared differences from the mean
// (a second pass over the row), not the difference of two large sums.
//
// Forms, by the row's length and alignment (rows on 16-byte boundaries whose length is a multiple of 8 go in
// vectors of 8 values):
//   warp     up to 1024 values: a row (or 2, 4 at once) per warp, all in registers, no barriers
//   cta      longer rows: a CTA per row, the row in registers
//   ring     longer rows, backward: one resident CTA walks over its rows, which bulk copies bring into a ring of
//            shared-memory stages ahead of it; the weight gradients' sums stay in its registers
//   scalar   rows off the 16-byte grid: a CTA per row (backward: resident), value by value in registers
//   any      rows longer than those hold

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kNormThreads = 256;

// ---------------------------------------------------------------- rows in registers
// Eight values as they lie in memory, and as four pairs for the two-wide fp32 instructions.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_stream(const __nv_bfloat16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
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
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
  }
};
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, const float2 (&f)[4]) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y), pack2(f[3].x, f[3].y)));
}
__device__ __forceinline__ void store_pairs(float* p, const float2 (&f)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
  __stcs(reinterpret_cast<float4*>(p + 4), make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight weights (or biases) from column n on (a multiple of 8); `fill` where there are none.  w_kind: the type, and
// kWeightVectors where the weights lie on 16-byte boundaries.
constexpr int32_t kWeightVectors = 2;
__device__ __forceinline__ void weights8(const void* w, int32_t w_kind, int64_t n, float fill, float2 (&f)[4]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = both(fill);
  } else if (w_kind == (FP8G_F32 | kWeightVectors)) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + n);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  } else if (w_kind == (FP8G_BF16 | kWeightVectors)) {
    Raw8<__nv_bfloat16> r;
    r.v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + n));
    r.get(f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(load_any(w, w_kind, n + 2 * i), load_any(w, w_kind, n + 2 * i + 1));
  }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The sum of a pair over the CTA, the same in every thread; `red` holds two rounds of 32 pairs (round `phase`),
// so one barrier a call is enough.
__device__ __forceinline__ float2 block_sum(float2 v, float2 (*red)[32], int phase) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = make_float2(warp_sum(v.x), warp_sum(v.y));
  if (warps == 1) return v;
  if (lane == 0) red[phase & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? red[phase & 1][lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}
__device__ __forceinline__ float block_sum(float v, float2 (*red)[32], int phase) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = warp_sum(v);
  if (warps == 1) return v;
  if (lane == 0) red[phase & 1][threadIdx.x >> 5].x = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[phase & 1][lane].x : 0.0f);
}

// The sum of (x - mu)^2 over NV vectors, without the vectors past the row's end.
template <typename T, int NV>
__device__ __forceinline__ float spread_sum(const Raw8<T> (&raw)[NV], const bool (&live)[NV], float mu) {
  float2 s = both(0.0f);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!live[v]) continue;
    float2 f[4];
    raw[v].get(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d = __fadd2_rn(f[i], both(-mu));
      s = __ffma2_rn(d, d, s);
    }
  }
  return s.x + s.y;
}
template <typename T, int NV>
__device__ __forceinline__ float value_sum(const Raw8<T> (&raw)[NV]) {
  float2 s = both(0.0f);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float2 f[4];
    raw[v].get(f);
    s = __fadd2_rn(s, __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3])));
  }
  return s.x + s.y;
}

// ---------------------------------------------------------------- forward
// (y may be x itself: a row is read before it is written)
// warp form: LPR lanes a row, lane l of a row holds the vectors l, l + LPR, ...
template <typename TX, typename TY, int LPR, int NV>
__global__ void __launch_bounds__(kNormThreads) layer_norm_warp_kernel(
    const TX* x, int64_t M, int32_t N, int64_t ldx, const void* __restrict__ w,
    const void* __restrict__ b, int32_t w_kind, float eps, TY* y, int64_t ldy,
    float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int kRows = kNormThreads / LPR;  // rows a CTA at once
  const int sub = threadIdx.x % LPR;
  bool live[NV];
  float2 wf[NV][4], bf[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = (v * LPR + sub) * 8;
    live[v] = col < N;
    if (live[v]) {
      weights8(w, w_kind, col, 1.0f, wf[v]);
      weights8(b, w_kind, col, 0.0f, bf[v]);
    }
  }
  const float inv_n = 1.0f / static_cast<float>(N);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  // the loop runs for whole warps (m0 is the warp's first row): the sums are taken by all its lanes
  int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows + (threadIdx.x & ~31) / LPR;
  const int64_t off = (threadIdx.x & 31) / LPR;
  Raw8<TX> next[NV];
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (live[v] && m < M) next[v].load_stream(x + m * ldx + (v * LPR + sub) * 8);
      else next[v].zero();
    }
  };
  fetch(m0 + off);
  for (; m0 < M; m0 += stride) {
    const int64_t m = m0 + off;
    Raw8<TX> raw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) raw[v] = next[v];
    if (m0 + stride < M) fetch(m + stride);
    const float mu = lanes_sum<LPR>(value_sum(raw)) * inv_n;
    const float var = lanes_sum<LPR>(spread_sum(raw, live, mu)) * inv_n;
    const float r = 1.0f / sqrtf(var + eps);
    if (m >= M) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!live[v]) continue;
      float2 f[4];
      raw[v].get(f);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[i], both(-mu)), both(r)), wf[v][i], bf[v][i]);
      store_pairs(y + m * ldy + (v * LPR + sub) * 8, f);
    }
    if (sub == 0) {
      if (mean) mean[m] = mu;
      if (rstd) rstd[m] = r;
    }
  }
}

// cta form: thread t holds the vectors t, t + blockDim.x, ...
template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(1024) layer_norm_cta_kernel(
    const TX* x, int32_t N, int64_t ldx, const void* __restrict__ w, const void* __restrict__ b,
    int32_t w_kind, float eps, TY* y, int64_t ldy, float* __restrict__ mean,
    float* __restrict__ rstd) {
  __shared__ float2 red[2][32];
  const int64_t m = blockIdx.x;
  Raw8<TX> raw[NV];
  bool live[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = (v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8;
    live[v] = col < N;
    if (live[v]) raw[v].load_stream(x + m * ldx + col);
    else raw[v].zero();
  }
  const float inv_n = 1.0f / static_cast<float>(N);
  const float mu = block_sum(value_sum(raw), red, 0) * inv_n;
  const float var = block_sum(spread_sum(raw, live, mu), red, 1) * inv_n;
  const float r = 1.0f / sqrtf(var + eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!live[v]) continue;
    const int col = (v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * 8;
    float2 f[4], wf[4], bf[4];
    weights8(w, w_kind, col, 1.0f, wf);
    weights8(b, w_kind, col, 0.0f, bf);
    raw[v].get(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[i], both(-mu)), both(r)), wf[i], bf[i]);
    store_pairs(y + m * ldy + col, f);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[m] = mu;
    if (rstd) rstd[m] = r;
  }
}

// scalar form: thread t holds the values t, t + blockDim.x, ...
template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(1024) layer_norm_scalar_kernel(
    const TX* x, int32_t N, int64_t ldx, const void* __restrict__ w, const void* __restrict__ b,
    int32_t w_kind, float eps, TY* y, int64_t ldy, float* __restrict__ mean,
    float* __restrict__ rstd) {
  __shared__ float2 red[2][32];
  const int64_t m = blockIdx.x;
  float f[NV];
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
    f[v] = col < N ? to_f32(x[m * ldx + col]) : 0.0f;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) s += f[v];
  const float inv_n = 1.0f / static_cast<float>(N);
  const float mu = block_sum(s, red, 0) * inv_n;
  s = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const float d = f[v] - mu;
    if (v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x) < N) s = fmaf(d, d, s);
  }
  const float r = 1.0f / sqrtf(block_sum(s, red, 1) * inv_n + eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
    if (col >= N) continue;
    const float wn = w ? load_any(w, w_kind, col) : 1.0f, bn = b ? load_any(b, w_kind, col) : 0.0f;
    y[m * ldy + col] = from_f32<TY>(fmaf((f[v] - mu) * r, wn, bn));
  }
  if (threadIdx.x == 0) {
    if (mean) mean[m] = mu;
    if (rstd) rstd[m] = r;
  }
}

// any form: one CTA a row, any length and alignment: the row is read three times (from L1 / L2 after the first).
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads) layer_norm_any_kernel(
    const TX* x, int64_t N, int64_t ldx, const void* __restrict__ w, const void* __restrict__ b,
    int32_t w_kind, float eps, TY* y, int64_t ldy, float* __restrict__ mean,
    float* __restrict__ rstd) {
  __shared__ float red[2 * kNormThreads / 32];
  const int64_t m = blockIdx.x;
  const TX* xr = x + m * ldx;
  TY* yr = y + m * ldy;
  float s[1] = {0.0f};
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) s[0] += to_f32(xr[n]);
  cta_sum<kNormThreads / 32>(s, red, 0);
  const float mu = s[0] / static_cast<float>(N);
  s[0] = 0.0f;
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float d = to_f32(xr[n]) - mu;
    s[0] += d * d;
  }
  cta_sum<kNormThreads / 32>(s, red, 1);
  const float r = 1.0f / sqrtf(s[0] / static_cast<float>(N) + eps);
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float wn = w ? load_any(w, w_kind, n) : 1.0f, bn = b ? load_any(b, w_kind, n) : 0.0f;
    yr[n] = from_f32<TY>((to_f32(xr[n]) - mu) * r * wn + bn);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[m] = mu;
    if (rstd) rstd[m] = r;
  }
}

// ---------------------------------------------------------------- backward
struct NormGrad {  // arguments of every backward form
  const void* dy;
  const void* x;
  void* dx;
  const void* w;
  const float* mean;
  const float* rstd;
  float* parts;  // [gridDim.x][2][N]: each CTA's sums of dy h and of dy; null where none are wanted
  int64_t M, lddy, ldx, lddx;
  int32_t N, w_kind;
  unsigned int* status;
  long long budget;
};

// One vector of a row: h = (x - mu) r and g = dy w, their row sums, and the weight gradients' terms.
struct GradPairs {
  float2 h[4], g[4];
};
__device__ __forceinline__ void grad_terms(const float2 (&xf)[4], const float2 (&yf)[4], const float2 (&wf)[4],
                                           float mu, float r, GradPairs& p, float2& s1, float2& s2,
                                           float2 (&dw)[4], float2 (&db)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p.h[i] = __fmul2_rn(__fadd2_rn(xf[i], both(-mu)), both(r));
    p.g[i] = __fmul2_rn(yf[i], wf[i]);
    s1 = __fadd2_rn(s1, p.g[i]);
    s2 = __ffma2_rn(p.g[i], p.h[i], s2);
    dw[i] = __ffma2_rn(yf[i], p.h[i], dw[i]);
    db[i] = __fadd2_rn(db[i], yf[i]);
  }
}
// dx = r (g - c1 - h c2)
__device__ __forceinline__ void grad_dx(const GradPairs& p, float c1, float c2, float r, float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = __fmul2_rn(__ffma2_rn(p.h[i], both(-c2), __fadd2_rn(p.g[i], both(-c1))), both(r));
}
__device__ __forceinline__ void store_part(float* p, const float2 (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}

// warp form, as forward; the CTA's warps add their sums up in shared memory, one after another.
constexpr int kNormGradThreads = 128;
template <typename TX, typename TY, int LPR, int NV>
__global__ void __launch_bounds__(kNormGradThreads) layer_norm_grad_warp_kernel(const NormGrad a) {
  constexpr int kRows = kNormGradThreads / LPR;
  __shared__ __align__(16) float sums[2 * LPR * NV * 8];
  griddep_launch_dependents();
  const int sub = threadIdx.x % LPR;
  const TX* x = static_cast<const TX*>(a.x);
  const TY* dy = static_cast<const TY*>(a.dy);
  bool live[NV];
  float2 wf[NV][4], dw[NV][4], db[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    live[v] = (v * LPR + sub) * 8 < a.N;
    weights8(live[v] ? a.w : nullptr, a.w_kind, (v * LPR + sub) * 8, 1.0f, wf[v]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[v][i] = db[v][i] = both(0.0f);
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows + (threadIdx.x & ~31) / LPR;
  const int64_t off = (threadIdx.x & 31) / LPR;
  Raw8<TX> nx[NV];
  Raw8<TY> ny[NV];
  float nmu = 0.0f, nr = 0.0f;
  auto fetch = [&](int64_t m) {  // rows past the end are zeros, which add nothing
    const bool in = m < a.M;
    nmu = in ? a.mean[m] : 0.0f;
    nr = in ? a.rstd[m] : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      nx[v].zero();
      ny[v].zero();
      if (live[v] && in) {
        nx[v].load_stream(x + m * a.ldx + (v * LPR + sub) * 8);
        ny[v].load_stream(dy + m * a.lddy + (v * LPR + sub) * 8);
      }
    }
  };
  fetch(m0 + off);
  for (; m0 < a.M; m0 += stride) {
    const int64_t m = m0 + off;
    const float mu = nmu, r = nr;
    GradPairs p[NV];
    float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 xf[4], yf[4];
      nx[v].get(xf);
      ny[v].get(yf);
      if (!live[v])
#pragma unroll
        for (int i = 0; i < 4; ++i) xf[i] = both(mu);  // h = 0 past the row's end
      grad_terms(xf, yf, wf[v], mu, r, p[v], s1, s2, dw[v], db[v]);
    }
    if (m0 + stride < a.M) fetch(m + stride);
    const float c1 = lanes_sum<LPR>(s1.x + s1.y) * inv_n, c2 = lanes_sum<LPR>(s2.x + s2.y) * inv_n;
    if (m >= a.M) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!live[v]) continue;
      float2 f[4];
      grad_dx(p[v], c1, c2, r, f);
      store_pairs(static_cast<TX*>(a.dx) + m * a.lddx + (v * LPR + sub) * 8, f);
    }
  }
  if (!a.parts) return;
  // over the rows that the warp's lanes shared, then over the warps
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int o = 16; o >= LPR; o >>= 1) {
        dw[v][i].x += __shfl_xor_sync(0xffffffffu, dw[v][i].x, o);
        dw[v][i].y += __shfl_xor_sync(0xffffffffu, dw[v][i].y, o);
        db[v][i].x += __shfl_xor_sync(0xffffffffu, db[v][i].x, o);
        db[v][i].y += __shfl_xor_sync(0xffffffffu, db[v][i].y, o);
      }
  constexpr int kCols = LPR * NV * 8;
  for (int w = 0; w < kNormGradThreads / 32; ++w) {
    if (threadIdx.x / 32 == w && (threadIdx.x & 31) < LPR) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2* sw = reinterpret_cast<float2*>(sums + (v * LPR + sub) * 8 + 2 * i);
          float2* sb = reinterpret_cast<float2*>(sums + kCols + (v * LPR + sub) * 8 + 2 * i);
          *sw = w == 0 ? dw[v][i] : __fadd2_rn(*sw, dw[v][i]);
          *sb = w == 0 ? db[v][i] : __fadd2_rn(*sb, db[v][i]);
        }
    }
    __syncthreads();
  }
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
  for (int n = threadIdx.x; n < a.N; n += kNormGradThreads) {
    part[n] = sums[n];
    part[a.N + n] = sums[kCols + n];
  }
}

// ring form.  The x and dy rows of `stages` rows ahead are in flight as bulk copies; a row's stage is filled again
// once every thread has passed the barrier of the row after it.
constexpr int kRingMaxStages = 8;
constexpr int kRingThreads = 512;

// Waits for a stage, at most `budget` cycles; past that it records the status and nobody waits any more (the
// results are void, the kernel ends).
__device__ __forceinline__ void ring_wait(uint32_t bar, uint32_t parity, const NormGrad& a, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*dead) return;
    if (clock64() - t0 > a.budget) {
      *dead = 1;
      record_status(a.status, FP8G_ERR_TIMEOUT);
      return;
    }
  }
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(kRingThreads, 1) layer_norm_grad_ring_kernel(const NormGrad a, int32_t stages) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full_bar[kRingMaxStages];
  __shared__ float2 red[2][32];
  __shared__ int s_dead;
  griddep_launch_dependents();
  const int tid = threadIdx.x, threads = blockDim.x;
  const uint32_t xb = static_cast<uint32_t>(a.N) * sizeof(TX), yb = static_cast<uint32_t>(a.N) * sizeof(TY);
  const int64_t P = gridDim.x;
  const int64_t rows = (a.M - blockIdx.x + P - 1) / P;  // rows blockIdx.x, blockIdx.x + P, ...
  if (tid == 0) {
    s_dead = 0;
    for (int s = 0; s < stages; ++s) mbar_init(smem_u32(&full_bar[s]), 1);
    fence_mbar_init();
  }
  __syncthreads();
  auto fill = [&](int64_t i) {  // one thread: the copies of this CTA's i-th row
    const int s = static_cast<int>(i % stages);
    const int64_t m = blockIdx.x + i * P;
    const uint32_t bar = smem_u32(&full_bar[s]), dst = smem_u32(ring) + static_cast<uint32_t>(s) * (xb + yb);
    mbar_arrive_expect_tx(true, bar, xb + yb);
    bulk_load(dst, static_cast<const TX*>(a.x) + m * a.ldx, xb, bar);
    bulk_load(dst + xb, static_cast<const TY*>(a.dy) + m * a.lddy, yb, bar);
  };
  if (tid == 0)
    for (int64_t i = 0; i < stages && i < rows; ++i) fill(i);
  bool live[NV];
  float2 wf[NV][4], dw[NV][4], db[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    live[v] = (v * threads + tid) * 8 < a.N;
    weights8(live[v] ? a.w : nullptr, a.w_kind, (v * threads + tid) * 8, 1.0f, wf[v]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[v][i] = db[v][i] = both(0.0f);
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  int s = 0;
  uint32_t parity = 0;
  // the statistics of 32 rows at a time, one row a lane (loaded 32 rows ahead: no row waits for them)
  const int lane = tid & 31;
  float mu32 = 0.0f, r32 = 0.0f, next_mu = 0.0f, next_r = 0.0f;
  auto stats = [&](int64_t i) {
    if (i + lane >= rows) return;
    next_mu = a.mean[blockIdx.x + (i + lane) * P];
    next_r = a.rstd[blockIdx.x + (i + lane) * P];
  };
  stats(0);
  for (int64_t i = 0; i < rows; ++i) {
    const int64_t m = blockIdx.x + i * P;
    if ((i & 31) == 0) {
      mu32 = next_mu;
      r32 = next_r;
      stats(i + 32);
    }
    const float mu = __shfl_sync(0xffffffffu, mu32, static_cast<int>(i & 31));
    const float r = __shfl_sync(0xffffffffu, r32, static_cast<int>(i & 31));
    ring_wait(smem_u32(&full_bar[s]), parity, a, &s_dead);
    const uint8_t* stage = ring + static_cast<size_t>(s) * (xb + yb);
    GradPairs p[NV];
    float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!live[v]) continue;
      Raw8<TX> rx;
      Raw8<TY> ry;
      rx.load(reinterpret_cast<const TX*>(stage) + (v * threads + tid) * 8);
      ry.load(reinterpret_cast<const TY*>(stage + xb) + (v * threads + tid) * 8);
      float2 xf[4], yf[4];
      rx.get(xf);
      ry.get(yf);
      grad_terms(xf, yf, wf[v], mu, r, p[v], s1, s2, dw[v], db[v]);
    }
    const float2 c = block_sum(make_float2(s1.x + s1.y, s2.x + s2.y), red, static_cast<int>(i & 1));
    // every thread has now read the row before this one
    if (tid == 0 && i > 0 && i - 1 + stages < rows) fill(i - 1 + stages);
    const float c1 = c.x * inv_n, c2 = c.y * inv_n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!live[v]) continue;
      float2 f[4];
      grad_dx(p[v], c1, c2, r, f);
      store_pairs(static_cast<TX*>(a.dx) + m * a.lddx + (v * threads + tid) * 8, f);
    }
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
  }
  if (!a.parts) return;
  float* part = a.parts + blockIdx.x * 2 * static_cast<int64_t>(a.N);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!live[v]) continue;
    store_part(part + (v * threads + tid) * 8, dw[v]);
    store_part(part + a.N + (v * threads + tid) * 8, db[v]);
  }
}

// scalar form: resident CTAs, thread t holds the columns t, t + blockDim.x, ...
template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(kRingThreads) layer_norm_grad_scalar_kernel(const NormGrad a) {
  __shared__ float2 red[2][32];
  griddep_launch_dependents();
  const int tid = threadIdx.x, threads = blockDim.x;
  const TX* x = static_cast<const TX*>(a.x);
  const TY* dy = static_cast<const TY*>(a.dy);
  float w[NV], dw[NV], db[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * threads + tid;
    w[v] = a.w && col < a.N ? load_any(a.w, a.w_kind, col) : 1.0f;
    dw[v] = db[v] = 0.0f;
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  int phase = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const float mu = a.mean[m], r = a.rstd[m];
    float h[NV], g[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = v * threads + tid;
      h[v] = col < a.N ? to_f32(x[m * a.ldx + col]) : mu;
      g[v] = col < a.N ? to_f32(dy[m * a.lddy + col]) : 0.0f;
    }
    float2 s = both(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[v] = (h[v] - mu) * r;
      dw[v] = fmaf(g[v], h[v], dw[v]);
      db[v] += g[v];
      g[v] *= w[v];
      s.x += g[v];
      s.y = fmaf(g[v], h[v], s.y);
    }
    s = block_sum(s, red, phase++);
    const float c1 = s.x * inv_n, c2 = s.y * inv_n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = v * threads + tid;
      if (col < a.N) static_cast<TX*>(a.dx)[m * a.lddx + col] = from_f32<TX>(fmaf(h[v], -c2, g[v] - c1) * r);
    }
  }
  if (!a.parts) return;
  float* part = a.parts + blockIdx.x * 2 * static_cast<int64_t>(a.N);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * threads + tid;
    if (col < a.N) {
      part[col] = dw[v];
      part[a.N + col] = db[v];
    }
  }
}

// any form: the data gradient, one CTA a row, any length and alignment.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads) layer_norm_dx_any_kernel(
    const TY* __restrict__ dy, int64_t lddy, const TX* __restrict__ x, int64_t ldx, const void* __restrict__ w,
    int32_t w_kind, const float* __restrict__ mean, const float* __restrict__ rstd, int64_t N,
    TX* __restrict__ dx, int64_t lddx) {
  __shared__ float red[2 * 2 * kNormThreads / 32];
  const int64_t m = blockIdx.x;
  const float mu = mean[m], r = rstd[m];
  const TX* xr = x + m * ldx;
  const TY* dyr = dy + m * lddy;
  float s[2] = {0.0f, 0.0f};
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float g = to_f32(dyr[n]) * (w ? load_any(w, w_kind, n) : 1.0f);
    s[0] += g;
    s[1] += g * ((to_f32(xr[n]) - mu) * r);
  }
  cta_sum<kNormThreads / 32>(s, red, 0);
  const float c1 = s[0] / static_cast<float>(N), c2 = s[1] / static_cast<float>(N);
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float g = to_f32(dyr[n]) * (w ? load_any(w, w_kind, n) : 1.0f);
    dx[m * lddx + n] = from_f32<TX>((g - c1 - (to_f32(xr[n]) - mu) * r * c2) * r);
  }
}

// Partial sums of the weight gradients, any length and alignment: thread = column, CTA row blockIdx.y = a range of rows.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads) layer_norm_dw_any_kernel(
    const TY* __restrict__ dy, int64_t lddy, const TX* __restrict__ x, int64_t ldx,
    const float* __restrict__ mean, const float* __restrict__ rstd, int64_t M, int64_t N,
    float* __restrict__ parts) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  if (n >= N) return;
  const int64_t P = gridDim.y, p = blockIdx.y;
  const int64_t lo = M * p / P, hi = M * (p + 1) / P;
  float dw = 0.0f, db = 0.0f;
  for (int64_t m = lo; m < hi; ++m) {
    const float g = to_f32(dy[m * lddy + n]);
    dw += g * ((to_f32(x[m * ldx + n]) - mean[m]) * rstd[m]);
    db += g;
  }
  parts[p * 2 * N + n] = dw;
  parts[p * 2 * N + N + n] = db;
}

// dw and db (either may be null) from the P partial rows [2][N].  A CTA takes 32 columns, its warps an equal share of
// the rows each: the additions' order follows from P alone.  The sums are short and the rows' addresses far apart, so
// the time is the loads' latency: eight in flight per lane, and many warps (P = 152, N = 7168: 6.3 us with 8 warps).
constexpr int kJoinMaxWarps = 32;
constexpr int kJoinUnroll = 8;
__global__ void __launch_bounds__(32 * kJoinMaxWarps) layer_norm_join_kernel(const float* __restrict__ parts, int32_t P,
                                                                             int64_t N, float* __restrict__ dw,
                                                                             float* __restrict__ db) {
  __shared__ float sums[kJoinMaxWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  griddep_wait();
  const int lo = static_cast<int>(static_cast<int64_t>(P) * warp / warps);
  const int hi = static_cast<int>(static_cast<int64_t>(P) * (warp + 1) / warps);
  float s = 0.0f;
  if (i < 2 * N) {
    for (int k = lo; k < hi; k += kJoinUnroll) {
      float v[kJoinUnroll];
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u)
        v[u] = k + u < hi ? __ldcg(parts + static_cast<int64_t>(k + u) * 2 * N + i) : 0.0f;
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || i >= 2 * N) return;
  float t = 0.0f;
  for (int w = 0; w < warps; ++w) t += sums[w][lane];
  if (i < N) {
    if (dw) dw[i] = t;
  } else if (db) {
    db[i - N] = t;
  }
}

bool dtype_ok(int32_t d) { return d == FP8G_BF16 || d == FP8G_F32; }
int dtype_size(int32_t d) { return d == FP8G_F32 ? 4 : 2; }

// ---------------------------------------------------------------- launches
constexpr int64_t kWarpMaxN = 1024;    // warp form: up to 4 vectors a lane
constexpr int64_t kCtaMaxN = 32768;    // cta form: up to 4 vectors a thread
constexpr int64_t kScalarMaxN = 16384; // scalar form, forward: up to 16 values a thread
constexpr int64_t kGradScalarMaxN = 8192;
constexpr int64_t kRingMaxN = 8192;    // ring form: up to 2 vectors a thread
constexpr int kRingBytes = 200 * 1024; // shared memory of a ring's stages, at most

// Rows of partial sums that the workspace has room for: the largest grid of any backward form.
int64_t norm_parts(int64_t M) { return std::min<int64_t>(M, 608); }

// Whether rows of N values of `size` bytes, `ld` apart, can be taken in vectors of 8.
bool vectors(const void* p, int size, int64_t N, int64_t ld) {
  return N % 8 == 0 && aligned16(p) && (ld * size) % 16 == 0;
}
// The weights' type as the kernels take it.
int32_t weight_kind(const void* w, const void* b, int32_t dtype) {
  return dtype | (aligned16(w) && aligned16(b) ? kWeightVectors : 0);
}
// Threads for `items` items a row at `each` a thread.
int row_threads(int64_t items, int each) { return static_cast<int>((items + each * 32 - 1) / (each * 32) * 32); }

template <typename TX, typename TY>
int layer_norm_launch(const void* xv, int64_t M, int64_t N, int64_t ldx, const void* w, const void* b,
                      int32_t w_kind, float eps, void* yv, int64_t ldy, float* mean, float* rstd,
                      const DeviceInfo* dev, cudaStream_t s) {
  const TX* x = static_cast<const TX*>(xv);
  TY* y = static_cast<TY*>(yv);
  const int n = static_cast<int>(N);
  const unsigned rows = static_cast<unsigned>(M);
  const bool vec = vectors(x, sizeof(TX), N, ldx) && vectors(y, sizeof(TY), N, ldy);
  if (vec && N <= kWarpMaxN) {
    auto go = N <= 64    ? layer_norm_warp_kernel<TX, TY, 8, 1>
              : N <= 128 ? layer_norm_warp_kernel<TX, TY, 16, 1>
              : N <= 256 ? layer_norm_warp_kernel<TX, TY, 32, 1>
              : N <= 512 ? layer_norm_warp_kernel<TX, TY, 32, 2>
                         : layer_norm_warp_kernel<TX, TY, 32, 4>;
    const int64_t per = kNormThreads / (N <= 64 ? 8 : N <= 128 ? 16 : 32);
    const int64_t ctas = std::min<int64_t>((M + per - 1) / per, 8 * static_cast<int64_t>(dev->sm_count));
    go<<<static_cast<unsigned>(ctas), kNormThreads, 0, s>>>(x, M, n, ldx, w, b, w_kind, eps, y, ldy, mean, rstd);
  } else if (vec && N <= kCtaMaxN) {
    const int64_t items = N / 8;
    // few rows: one vector a thread, for the latency; many: more a thread
    const int nv = M <= 2 * dev->sm_count && items <= 1024 ? 1 : items <= 1024 ? 2 : items <= 2048 ? 2 : 4;
    auto go = nv == 1   ? layer_norm_cta_kernel<TX, TY, 1>
              : nv == 2 ? layer_norm_cta_kernel<TX, TY, 2>
                        : layer_norm_cta_kernel<TX, TY, 4>;
    go<<<rows, row_threads(items, nv), 0, s>>>(x, n, ldx, w, b, w_kind, eps, y, ldy, mean, rstd);
  } else if (N <= kScalarMaxN) {
    const int nv = N <= 1024 ? 4 : N <= 4096 ? 8 : 16;
    auto go = nv == 4   ? layer_norm_scalar_kernel<TX, TY, 4>
              : nv == 8 ? layer_norm_scalar_kernel<TX, TY, 8>
                        : layer_norm_scalar_kernel<TX, TY, 16>;
    go<<<rows, row_threads(N, nv), 0, s>>>(x, n, ldx, w, b, w_kind, eps, y, ldy, mean, rstd);
  } else {
    layer_norm_any_kernel<TX, TY><<<rows, kNormThreads, 0, s>>>(x, N, ldx, w, b, w_kind, eps, y, ldy, mean, rstd);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

// The ring's resident CTAs per SM: one of 512 threads, more of shorter rows (their barriers and latencies overlap).
int ring_per_sm(int threads) { return std::max(1, std::min(4, 768 / threads)); }

template <typename TX, typename TY, int NV>
int ring_launch(const NormGrad& a, int threads, int64_t grid, cudaStream_t s) {
  const int stage = a.N * static_cast<int>(sizeof(TX) + sizeof(TY));
  const int stages = std::min(kRingMaxStages, kRingBytes / ring_per_sm(threads) / stage);
  auto kern = layer_norm_grad_ring_kernel<TX, TY, NV>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  kern<<<static_cast<unsigned>(grid), threads, stages * stage, s>>>(a, stages);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

template <typename TX, typename TY>
int layer_norm_backward_launch(NormGrad a, float* dw, float* db, const DeviceInfo* dev, cudaStream_t s) {
  const int64_t M = a.M, N = a.N;
  const bool vec = vectors(a.x, sizeof(TX), N, a.ldx) && vectors(a.dy, sizeof(TY), N, a.lddy) &&
                   vectors(a.dx, sizeof(TX), N, a.lddx);
  const int sms = dev->sm_count;
  int64_t P = 0;
  if (vec && N <= kWarpMaxN) {
    auto go = N <= 64    ? layer_norm_grad_warp_kernel<TX, TY, 8, 1>
              : N <= 128 ? layer_norm_grad_warp_kernel<TX, TY, 16, 1>
              : N <= 256 ? layer_norm_grad_warp_kernel<TX, TY, 32, 1>
              : N <= 512 ? layer_norm_grad_warp_kernel<TX, TY, 32, 2>
                         : layer_norm_grad_warp_kernel<TX, TY, 32, 4>;
    const int64_t per = kNormGradThreads / (N <= 64 ? 8 : N <= 128 ? 16 : 32);
    P = std::min<int64_t>({(M + per - 1) / per, 4 * static_cast<int64_t>(sms), norm_parts(M)});
    go<<<static_cast<unsigned>(P), kNormGradThreads, 0, s>>>(a);
  } else if (vec && N <= kRingMaxN) {
    const int nv = N <= 4096 ? 1 : 2, threads = row_threads(N / 8, nv);
    P = std::min<int64_t>(M, static_cast<int64_t>(sms) * ring_per_sm(threads));
    const int st = nv == 1 ? ring_launch<TX, TY, 1>(a, threads, P, s) : ring_launch<TX, TY, 2>(a, threads, P, s);
    if (st != FP8G_OK) return st;
  } else if (N <= kGradScalarMaxN) {
    const int nv = N <= 1024 ? 4 : N <= 4096 ? 8 : 16;
    const int threads = row_threads(N, nv);
    P = std::min<int64_t>({M, static_cast<int64_t>(sms) * std::max(1, std::min(4, 1024 / threads)), norm_parts(M)});
    auto go = nv == 4   ? layer_norm_grad_scalar_kernel<TX, TY, 4>
              : nv == 8 ? layer_norm_grad_scalar_kernel<TX, TY, 8>
                        : layer_norm_grad_scalar_kernel<TX, TY, 16>;
    go<<<static_cast<unsigned>(P), threads, 0, s>>>(a);
  } else {
    layer_norm_dx_any_kernel<TX, TY><<<static_cast<unsigned>(M), kNormThreads, 0, s>>>(
        static_cast<const TY*>(a.dy), a.lddy, static_cast<const TX*>(a.x), a.ldx, a.w, a.w_kind, a.mean, a.rstd, N,
        static_cast<TX*>(a.dx), a.lddx);
    if (a.parts) {
      P = norm_parts(M);
      const dim3 grid(static_cast<unsigned>((N + kNormThreads - 1) / kNormThreads), static_cast<unsigned>(P));
      layer_norm_dw_any_kernel<TX, TY><<<grid, kNormThreads, 0, s>>>(
          static_cast<const TY*>(a.dy), a.lddy, static_cast<const TX*>(a.x), a.ldx, a.mean, a.rstd, M, N, a.parts);
    }
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  if (!a.parts) return FP8G_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((2 * N + 31) / 32));
  cfg.blockDim = dim3(32 * static_cast<unsigned>(std::min<int64_t>(
                                kJoinMaxWarps, (P + kJoinUnroll - 1) / kJoinUnroll)));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, layer_norm_join_kernel, static_cast<const float*>(a.parts), static_cast<int32_t>(P), N,
                         dw, db) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_layer_norm(const void* x, int32_t x_dtype, int64_t M, int64_t N, int64_t ldx,
                               const void* weight, const void* bias, int32_t w_dtype, float eps, void* y,
                               int32_t y_dtype, int64_t ldy, float* mean, float* rstd, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype) || !dtype_ok(w_dtype)) return FP8G_ERR_INVALID_ARG;
  if (M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || ldx < N || ldy < N || !(eps >= 0.0f))
    return FP8G_ERR_INVALID_ARG;
  if (M == 0) return FP8G_OK;
  if (!x || !y) return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(x, dtype_size(x_dtype)) || !aligned_to(y, dtype_size(y_dtype)) ||
      !aligned_to(weight, dtype_size(w_dtype)) || !aligned_to(bias, dtype_size(w_dtype)) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  auto go = x_dtype == FP8G_F32
                ? (y_dtype == FP8G_F32 ? layer_norm_launch<float, float> : layer_norm_launch<float, __nv_bfloat16>)
                : (y_dtype == FP8G_F32 ? layer_norm_launch<__nv_bfloat16, float>
                                       : layer_norm_launch<__nv_bfloat16, __nv_bfloat16>);
  return go(x, M, N, ldx, weight, bias, weight_kind(weight, bias, w_dtype), eps, y, ldy, mean, rstd, dev,
            static_cast<cudaStream_t>(stream));
}

extern "C" int fp8g_layer_norm_backward_workspace(int64_t M, int64_t N, int64_t* bytes) {
  if (M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = norm_parts(M) * 2 * N * 4;
  return FP8G_OK;
}

extern "C" int fp8g_layer_norm_backward(const void* dy, int32_t dy_dtype, int64_t lddy, const void* x,
                                        int32_t x_dtype, int64_t ldx, const void* weight, int32_t w_dtype,
                                        const float* mean, const float* rstd, int64_t M, int64_t N, void* dx,
                                        int64_t lddx, float* dweight, float* dbias, void* workspace,
                                        int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(x_dtype) || !dtype_ok(dy_dtype) || !dtype_ok(w_dtype)) return FP8G_ERR_INVALID_ARG;
  if (M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || lddy < N || ldx < N || lddx < N)
    return FP8G_ERR_INVALID_ARG;
  if (M > 0 && (!dy || !x || !mean || !rstd || !dx)) return FP8G_ERR_INVALID_ARG;
  if ((dweight || dbias) && M > 0 && (!workspace || workspace_bytes < norm_parts(M) * 2 * N * 4))
    return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(dy, dtype_size(dy_dtype)) || !aligned_to(x, dtype_size(x_dtype)) ||
      !aligned_to(dx, dtype_size(x_dtype)) || !aligned_to(weight, dtype_size(w_dtype)) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4) || !aligned_to(dweight, 4) || !aligned_to(dbias, 4) || !aligned16(workspace))
    return FP8G_ERR_ALIGNMENT;
  if (M == 0 && !dweight && !dbias) return FP8G_OK;
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {  // sums over no rows
    if ((dweight && cudaMemsetAsync(dweight, 0, static_cast<size_t>(N) * 4, s) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, static_cast<size_t>(N) * 4, s) != cudaSuccess)) {
      cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
    return FP8G_OK;
  }
  auto go = x_dtype == FP8G_F32
                ? (dy_dtype == FP8G_F32 ? layer_norm_backward_launch<float, float>
                                        : layer_norm_backward_launch<float, __nv_bfloat16>)
                : (dy_dtype == FP8G_F32 ? layer_norm_backward_launch<__nv_bfloat16, float>
                                        : layer_norm_backward_launch<__nv_bfloat16, __nv_bfloat16>);
  NormGrad a{};
  a.dy = dy, a.x = x, a.dx = dx, a.w = weight, a.mean = mean, a.rstd = rstd;
  a.parts = dweight || dbias ? static_cast<float*>(workspace) : nullptr;
  a.M = M, a.lddy = lddy, a.ldx = ldx, a.lddx = lddx;
  a.N = static_cast<int32_t>(N), a.w_kind = weight_kind(weight, nullptr, w_dtype);
  a.status = dev->status, a.budget = wait_budget_cycles();
  return go(a, dweight, dbias, dev, s);
}
