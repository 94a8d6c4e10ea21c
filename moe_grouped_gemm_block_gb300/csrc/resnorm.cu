// resnorm.cu -- the root-mean-square norms around a block, fused with its residual: the norm after a block with its gate
// and residual scale, and the norm before the next one, in one pass; and their gradient.
//
//     u = f r_f post (r_f = 1 / sqrt(mean_n f^2 + eps)), or f without the norm after the block
//     h = x + scale gate u,   r = 1 / sqrt(mean_n h^2 + eps),   y = h r w
//   backward, from dy and dh (the gradient that reaches h on other ways), with e = h r, g = dy w, k = f r_f (or f):
//     dx = dh + r (g - e mean_n (g e)),   q = dx scale gate post,   df = r_f (q - k mean_n (q k)), or q
//     dw = sum_m dy e,   S = scale sum_m dx k,   dgate = S post,   dpost = S gate
//
// All sums are fp32, a result is rounded once; y is formed from h before its rounding.  A row is held in registers by a
// part of a warp (short rows) or by a CTA, 8 values of a thread at a time: in vectors where all rows lie on the 16-byte
// grid, else value by value with neighbouring threads on neighbouring values.  Longer rows than those hold are read
// again for each step ("any").  One sum a column serves both dgate and dpost, as S does not depend on them.
//
// Bound by memory.

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kResMaxThreads = 512;
constexpr int kResMaxParts = 608;  // CTAs, and partial sums, of a backward call

struct ResArgs {
  const void *x, *f, *w, *post, *gate, *dy, *dh;  // backward: x is h
  void *h, *y, *dx, *df;
  float *rstd, *rstd_f;  // results of the forward, inputs of the backward call
  float* parts;          // [CTAs][2][N]
  int64_t M, ldx, ldf, ldh, ldy, lddy, lddh, lddx, lddf;
  int32_t N, w_kind, vec, wvec, norm_f;
  float scale, eps, inv_n;
};

// Value j of a thread's v-th eight: the column, where R threads take a row.
template <int V>
struct Columns {
  int t, R, N;
  bool vec;
  __device__ __forceinline__ int at(int v, int j) const { return vec ? 8 * (t + v * R) + j : t + (8 * v + j) * R; }
  __device__ __forceinline__ bool none(int v) const { return at(v, 0) >= N; }
  template <typename T>
  __device__ __forceinline__ void load(Raw8<T>& r, const T* row, int v, bool real) const {
    if (vec) {  // N is a multiple of 8 here
      if (real && at(v, 0) < N) r.load_stream(row + at(v, 0));
      else r.zero();
    } else {
      T f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = real && at(v, j) < N ? row[at(v, j)] : from_f32<T>(0.0f);
      r.set(f);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int v, const float (&f)[8]) const {
    if (vec) {
      if (at(v, 0) < N) store8_stream(row + at(v, 0), f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at(v, j) < N) row[at(v, j)] = from_f32<T>(f[j]);
    }
  }
  // f[j] *= the weights
  __device__ __forceinline__ void times(const void* w, int kind, bool wvec, int v, float (&f)[8]) const {
    if (!w) return;
    if (vec && wvec) {
      if (at(v, 0) >= N) return;
      float g[8];
      if (kind == FP8G_F32) load8(static_cast<const float*>(w) + at(v, 0), g);
      else load8(static_cast<const __nv_bfloat16*>(w) + at(v, 0), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= g[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at(v, j) < N) f[j] *= load_any(w, kind, at(v, j));
    }
  }
};
template <typename T>
__device__ __forceinline__ void get8(const Raw8<T>& r, float (&f)[8]) {
  r.get(reinterpret_cast<float2(&)[4]>(f));
}

// The sum over the threads of a row: LPR lanes of a warp, or (LPR 0) the CTA.
template <int LPR>
__device__ __forceinline__ float res_sum(float v, float (*red)[32], int& phase) {
  if constexpr (LPR > 0) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  } else {
    v = warp_sum(v);
    float* r = red[phase & 1];
    ++phase;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kResMaxThreads / 128; ++i) {  // the entries past the CTA's warps are 0
      const float4 q = *reinterpret_cast<const float4*>(r + 4 * i);
      s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
    }
    return (s.x + s.y) + (s.z + s.w);
  }
}
__device__ __forceinline__ float root_inverse(float mean_square, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(mean_square + eps));
}

template <typename TS, typename TB, int LPR, int V>
__global__ void __launch_bounds__(LPR ? 256 : kResMaxThreads) residual_norm_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  const int rows = LPR ? 256 / (LPR ? LPR : 1) : 1;
  const int mine = LPR ? static_cast<int>(threadIdx.x) / (LPR ? LPR : 1) : 0;
  const Columns<V> col{LPR ? static_cast<int>(threadIdx.x) % (LPR ? LPR : 1) : static_cast<int>(threadIdx.x),
                       LPR ? LPR : static_cast<int>(blockDim.x), a.N, a.vec != 0};
  if (!LPR) {
    if (threadIdx.x < 64) (&red[0][0])[threadIdx.x] = 0.0f;
    if (blockDim.x < 64 && threadIdx.x + 32 < 64) (&red[0][0])[threadIdx.x + 32] = 0.0f;
    __syncthreads();
  }
  int phase = 0;
  for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * rows; m0 < a.M; m0 += static_cast<int64_t>(gridDim.x) * rows) {
    const int64_t m = m0 + mine;
    const bool real = m < a.M;
    Raw8<TS> rx[V];
    Raw8<TB> rf[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      col.load(rx[v], static_cast<const TS*>(a.x) + m * a.ldx, v, real);
      if (a.f) col.load(rf[v], static_cast<const TB*>(a.f) + m * a.ldf, v, real);
    }
    float x[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) get8(rx[v], x[v]);
    if (a.f) {
      float by = a.scale;
      if (a.norm_f) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float f[8];
          get8(rf[v], f);
#pragma unroll
          for (int j = 0; j < 8; ++j) s = fmaf(f[j], f[j], s);
        }
        s = root_inverse(res_sum<LPR>(s, red, phase) * a.inv_n, a.eps);
        if (col.t == 0 && real && a.rstd_f) a.rstd_f[m] = s;
        by *= s;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        get8(rf[v], f);
        col.times(a.post, a.w_kind, a.wvec, v, f);
        col.times(a.gate, a.w_kind, a.wvec, v, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = fmaf(by, f[j], x[v][j]);
        if (real && a.h) col.store(static_cast<TS*>(a.h) + m * a.ldh, v, x[v]);
      }
    }
    if (!a.y) continue;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(x[v][j], x[v][j], s);
    s = root_inverse(res_sum<LPR>(s, red, phase) * a.inv_n, a.eps);
    if (col.t == 0 && real && a.rstd) a.rstd[m] = s;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] *= s;
      col.times(a.w, a.w_kind, a.wvec, v, x[v]);
      if (real) col.store(static_cast<TB*>(a.y) + m * a.ldy, v, x[v]);
    }
  }
}

template <typename TS, typename TB, int LPR, int V>
__global__ void __launch_bounds__(LPR ? 256 : kResMaxThreads) residual_norm_backward_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  extern __shared__ float sums[];  // LPR: [2][N]
  griddep_launch_dependents();
  const int rows = LPR ? 256 / (LPR ? LPR : 1) : 1;
  const int mine = LPR ? static_cast<int>(threadIdx.x) / (LPR ? LPR : 1) : 0;
  const Columns<V> col{LPR ? static_cast<int>(threadIdx.x) % (LPR ? LPR : 1) : static_cast<int>(threadIdx.x),
                       LPR ? LPR : static_cast<int>(blockDim.x), a.N, a.vec != 0};
  if (!LPR) {
    if (threadIdx.x < 64) (&red[0][0])[threadIdx.x] = 0.0f;
    if (blockDim.x < 64 && threadIdx.x + 32 < 64) (&red[0][0])[threadIdx.x + 32] = 0.0f;
    __syncthreads();
  }
  int phase = 0;
  float dw[V][8], df_sum[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = df_sum[v][j] = 0.0f;
  for (int64_t m0 = static_cast<int64_t>(blockIdx.x) * rows; m0 < a.M; m0 += static_cast<int64_t>(gridDim.x) * rows) {
    const int64_t m = m0 + mine;
    const bool real = m < a.M;
    Raw8<TS> rh[V], rd[V];
    Raw8<TB> ry[V], rf[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (a.dy) {
        col.load(rh[v], static_cast<const TS*>(a.x) + m * a.ldx, v, real);
        col.load(ry[v], static_cast<const TB*>(a.dy) + m * a.lddy, v, real);
      }
      if (a.dh) col.load(rd[v], static_cast<const TS*>(a.dh) + m * a.lddh, v, real);
      else rd[v].zero();
      if (a.f) col.load(rf[v], static_cast<const TB*>(a.f) + m * a.ldf, v, real);
    }
    float dx[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) get8(rd[v], dx[v]);
    if (a.dy) {
      const float r = real ? a.rstd[m] : 0.0f;
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float g[8], e[8];
        get8(ry[v], g);
        get8(rh[v], e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] *= r;
          dw[v][j] = fmaf(g[j], e[j], dw[v][j]);
        }
        col.times(a.w, a.w_kind, a.wvec, v, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(g[j], e[j], s);
      }
      s = res_sum<LPR>(s, red, phase) * a.inv_n * r;  // e once more is h r
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float g[8], e[8];
        get8(ry[v], g);
        get8(rh[v], e);
        col.times(a.w, a.w_kind, a.wvec, v, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[v][j] = fmaf(r, g[j] - e[j] * s, dx[v][j]);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (real) col.store(static_cast<TS*>(a.dx) + m * a.lddx, v, dx[v]);
    if (!a.df) continue;
    const float rf_ = a.norm_f && real ? a.rstd_f[m] : 1.0f;
    if (a.f) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float k[8];
        get8(rf[v], k);
#pragma unroll
        for (int j = 0; j < 8; ++j) df_sum[v][j] = fmaf(dx[v][j], k[j] * rf_, df_sum[v][j]);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dx[v][j] *= a.scale;
      col.times(a.post, a.w_kind, a.wvec, v, dx[v]);
      col.times(a.gate, a.w_kind, a.wvec, v, dx[v]);
      if (a.norm_f) {
        float k[8];
        get8(rf[v], k);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(dx[v][j], k[j], s);
      }
    }
    if (a.norm_f) {
      s = res_sum<LPR>(s, red, phase) * a.inv_n * rf_ * rf_;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float k[8];
        get8(rf[v], k);
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[v][j] = rf_ * (dx[v][j] - k[j] * s);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (real) col.store(static_cast<TB*>(a.df) + m * a.lddf, v, dx[v]);
  }
  if (!a.parts) return;
  float* out = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
  if constexpr (LPR == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col.at(v, j) < a.N) {
          out[col.at(v, j)] = dw[v][j];
          out[a.N + col.at(v, j)] = df_sum[v][j];
        }
  } else {
    // the rows of a warp, then its CTA's warps one after the other
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int off = 16; off >= (LPR ? LPR : 1); off >>= 1) {
          dw[v][j] += __shfl_xor_sync(0xffffffffu, dw[v][j], off);
          df_sum[v][j] += __shfl_xor_sync(0xffffffffu, df_sum[v][j], off);
        }
    for (int w = 0; w < 8; ++w) {
      if (static_cast<int>(threadIdx.x >> 5) == w && (threadIdx.x & 31) < LPR) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col.at(v, j) < a.N) {
              float* s = sums + col.at(v, j);
              s[0] = (w ? s[0] : 0.0f) + dw[v][j];
              s[a.N] = (w ? s[a.N] : 0.0f) + df_sum[v][j];
            }
      }
      __syncthreads();
    }
    for (int n = threadIdx.x; n < 2 * a.N; n += blockDim.x) out[n] = sums[n];
  }
}

// Rows of any length: a CTA a row, which reads it again for each step.  Backward, a CTA adds its rows' column sums up in
// its own place of the workspace.
template <typename TS, typename TB>
__global__ void __launch_bounds__(kResMaxThreads) residual_norm_any_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  if (threadIdx.x < 64) (&red[0][0])[threadIdx.x] = 0.0f;
  __syncthreads();
  int phase = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const TS* x = static_cast<const TS*>(a.x) + m * a.ldx;
    const TB* f = a.f ? static_cast<const TB*>(a.f) + m * a.ldf : nullptr;
    float by = a.scale;
    if (f && a.norm_f) {
      float s = 0.0f;
      for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) s = fmaf(to_f32(f[n]), to_f32(f[n]), s);
      s = root_inverse(res_sum<0>(s, red, phase) * a.inv_n, a.eps);
      if (threadIdx.x == 0 && a.rstd_f) a.rstd_f[m] = s;
      by *= s;
    }
    auto value = [&](int n) {
      float v = to_f32(x[n]);
      if (f) {
        float k = to_f32(f[n]);
        if (a.post) k *= load_any(a.post, a.w_kind, n);
        if (a.gate) k *= load_any(a.gate, a.w_kind, n);
        v = fmaf(by, k, v);
      }
      return v;
    };
    float s = 0.0f;
    if (a.y) {
      for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) {
        const float v = value(n);
        s = fmaf(v, v, s);
      }
      s = root_inverse(res_sum<0>(s, red, phase) * a.inv_n, a.eps);
      if (threadIdx.x == 0 && a.rstd) a.rstd[m] = s;
    }
    for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) {  // (h may be x: a value is read before it is written)
      const float v = value(n);
      if (a.y) static_cast<TB*>(a.y)[m * a.ldy + n] = from_f32<TB>(v * s * (a.w ? load_any(a.w, a.w_kind, n) : 1.0f));
      if (f && a.h) static_cast<TS*>(a.h)[m * a.ldh + n] = from_f32<TS>(v);
    }
  }
}
template <typename TS, typename TB>
__global__ void __launch_bounds__(kResMaxThreads) residual_norm_backward_any_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  griddep_launch_dependents();
  if (threadIdx.x < 64) (&red[0][0])[threadIdx.x] = 0.0f;
  __syncthreads();
  int phase = 0;
  float* out = a.parts ? a.parts + static_cast<int64_t>(blockIdx.x) * 2 * a.N : nullptr;
  if (out)
    for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) out[n] = out[a.N + n] = 0.0f;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const TS* h = static_cast<const TS*>(a.x) + m * a.ldx;
    const TB* dy = a.dy ? static_cast<const TB*>(a.dy) + m * a.lddy : nullptr;
    const TS* dh = a.dh ? static_cast<const TS*>(a.dh) + m * a.lddh : nullptr;
    const TB* f = a.f ? static_cast<const TB*>(a.f) + m * a.ldf : nullptr;
    const float r = dy ? a.rstd[m] : 0.0f, rf = a.norm_f ? a.rstd_f[m] : 1.0f;
    auto grad_y = [&](int n) { return to_f32(dy[n]) * (a.w ? load_any(a.w, a.w_kind, n) : 1.0f); };
    float s = 0.0f, s2 = 0.0f;
    if (dy) {
      for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) s = fmaf(grad_y(n), to_f32(h[n]), s);
      s = res_sum<0>(s, red, phase) * a.inv_n * r * r;
    }
    auto grad_x = [&](int n) {
      const float d = dh ? to_f32(dh[n]) : 0.0f;
      return dy ? fmaf(r, grad_y(n) - to_f32(h[n]) * s, d) : d;
    };
    auto grad_u = [&](float dx, int n) {
      float q = dx * a.scale;
      if (a.post) q *= load_any(a.post, a.w_kind, n);
      if (a.gate) q *= load_any(a.gate, a.w_kind, n);
      return q;
    };
    if (a.df && a.norm_f) {
      for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) s2 = fmaf(grad_u(grad_x(n), n), to_f32(f[n]), s2);
      s2 = res_sum<0>(s2, red, phase) * a.inv_n * rf * rf;
    }
    for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) {  // (dx may be dh: read before it is written)
      const float dx = grad_x(n);
      if (out && dy) out[n] = fmaf(to_f32(dy[n]), to_f32(h[n]) * r, out[n]);
      if (out && f) out[a.N + n] = fmaf(dx, to_f32(f[n]) * rf, out[a.N + n]);
      if (a.df) {
        float q = grad_u(dx, n);
        if (a.norm_f) q = rf * (q - to_f32(f[n]) * s2);
        static_cast<TB*>(a.df)[m * a.lddf + n] = from_f32<TB>(q);
      }
      static_cast<TS*>(a.dx)[m * a.lddx + n] = from_f32<TS>(dx);
    }
  }
}

// The columns' sums from the CTAs' partial ones, in their order: 32 columns a CTA, 8 threads a column.
struct ResJoin {
  const float* parts;
  const void *post, *gate;
  float *dw, *dgate, *dpost;
  int32_t P, N, w_kind;
  float scale;
};
__global__ void __launch_bounds__(256) residual_norm_join_kernel(const ResJoin a) {
  __shared__ float s[2][8][33];
  griddep_wait();
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5, n = blockIdx.x * 32 + c;
  float w = 0.0f, f = 0.0f;
  if (n < a.N)
    for (int p = k; p < a.P; p += 8) {
      w += __ldcg(a.parts + static_cast<int64_t>(p) * 2 * a.N + n);
      f += __ldcg(a.parts + (static_cast<int64_t>(p) * 2 + 1) * a.N + n);
    }
  s[0][k][c] = w;
  s[1][k][c] = f;
  __syncthreads();
  if (k > 0 || n >= a.N) return;
  w = f = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) w += s[0][i][c], f += s[1][i][c];
  f *= a.scale;
  if (a.dw) a.dw[n] = w;
  if (a.dgate) a.dgate[n] = f * (a.post ? load_any(a.post, a.w_kind, n) : 1.0f);
  if (a.dpost) a.dpost[n] = f * (a.gate ? load_any(a.gate, a.w_kind, n) : 1.0f);
}

// The form of a row's length: LPR lanes of a warp (0: a CTA), V eights a thread; -1: any.
struct ResForm {
  int lpr, v, threads, rows;  // rows a CTA at once
};
ResForm res_form(int64_t N) {
  const int64_t eights = (N + 7) / 8;
  if (eights <= 8) return {8, 1, 256, 32};
  if (eights <= 16) return {16, 1, 256, 16};
  if (eights <= 32) return {32, 1, 256, 8};
  if (eights <= 64) return {32, 2, 256, 8};
  const int v = eights <= 512 ? 1 : eights <= 1024 ? 2 : 4;
  if (eights > 4 * kResMaxThreads) return {-1, 1, kResMaxThreads, 1};
  return {0, v, static_cast<int>(((eights + v - 1) / v + 31) / 32 * 32), 1};
}

int64_t res_ctas(const ResForm& f, int64_t M, bool backward) {
  const int64_t rows = (M + f.rows - 1) / f.rows;
  // about 2048 threads an SM forward; backward as many as its registers let stay
  const int64_t most = backward ? (f.lpr > 0 ? 304 : f.threads <= 256 ? 456 : f.v == 1 ? 304 : 152)
                                : int64_t{152} * std::max(1, 1024 / f.threads) * 2;
  return std::min(rows, std::min<int64_t>(most, backward ? kResMaxParts : most));
}

template <typename TS, typename TB>
int res_forward(const ResArgs& a, cudaStream_t s) {
  const ResForm f = res_form(a.N);
  const unsigned ctas = static_cast<unsigned>(res_ctas(f, a.M, false));
  auto go = f.lpr == 8    ? residual_norm_kernel<TS, TB, 8, 1>
            : f.lpr == 16 ? residual_norm_kernel<TS, TB, 16, 1>
            : f.lpr == 32 ? (f.v == 1 ? residual_norm_kernel<TS, TB, 32, 1> : residual_norm_kernel<TS, TB, 32, 2>)
            : f.lpr < 0   ? residual_norm_any_kernel<TS, TB>
            : f.v == 1    ? residual_norm_kernel<TS, TB, 0, 1>
            : f.v == 2    ? residual_norm_kernel<TS, TB, 0, 2>
                          : residual_norm_kernel<TS, TB, 0, 4>;
  go<<<ctas, f.threads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

template <typename TS, typename TB>
int res_backward(const ResArgs& a, const ResJoin& j, cudaStream_t s) {
  const ResForm f = res_form(a.N);
  const unsigned ctas = static_cast<unsigned>(res_ctas(f, a.M, true));
  auto go = f.lpr == 8    ? residual_norm_backward_kernel<TS, TB, 8, 1>
            : f.lpr == 16 ? residual_norm_backward_kernel<TS, TB, 16, 1>
            : f.lpr == 32 ? (f.v == 1 ? residual_norm_backward_kernel<TS, TB, 32, 1>
                                      : residual_norm_backward_kernel<TS, TB, 32, 2>)
            : f.lpr < 0   ? residual_norm_backward_any_kernel<TS, TB>
            : f.v == 1    ? residual_norm_backward_kernel<TS, TB, 0, 1>
            : f.v == 2    ? residual_norm_backward_kernel<TS, TB, 0, 2>
                          : residual_norm_backward_kernel<TS, TB, 0, 4>;
  if (ctas) go<<<ctas, f.threads, f.lpr > 0 ? 8 * a.N : 0, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  if (!a.parts) return FP8G_OK;
  ResJoin join = j;
  join.P = static_cast<int32_t>(ctas);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + 31) / 32));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = ctas ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, residual_norm_join_kernel, join) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

bool bad_type(int32_t t) { return t != FP8G_BF16 && t != FP8G_F32; }
int64_t type_size(int32_t t) { return t == FP8G_F32 ? 4 : 2; }
// A matrix's rows lie on the 16-byte grid (null: there is none).
bool on_grid(const void* p, int64_t ld, int64_t M) { return !p || (aligned16(p) && (M == 1 || ld % 8 == 0)); }

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_residual_rms_norm(const void* x, int64_t ldx, const void* f, int64_t ldf, int32_t stream_dtype,
                                      int32_t block_dtype, int64_t M, int64_t N, int32_t post_norm,
                                      const void* post_weight, const void* gate, float scale, const void* weight,
                                      int32_t w_dtype, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                                      float* rstd_f, float* rstd, void* stream) {
  if (bad_type(stream_dtype) || bad_type(block_dtype) || bad_type(w_dtype) || M < 0 || M > 0x7FFFFFFF || N < 1 ||
      N > 0x7FFFFFF0 || ldx < N || (f && ldf < N) || (h && ldh < N) || (y && ldy < N) || (post_norm & ~1) ||
      !(eps >= 0.0f) || (post_weight && !post_norm))
    return FP8G_ERR_INVALID_ARG;
  if (M == 0) return FP8G_OK;  // (no rows: their addresses may all be null)
  if (!x || (!h && !y) || (!f && (post_norm || post_weight || gate || h))) return FP8G_ERR_INVALID_ARG;
  const int64_t ss = type_size(stream_dtype), bs = type_size(block_dtype), ws = type_size(w_dtype);
  if (!aligned_to(x, ss) || !aligned_to(h, ss) || !aligned_to(f, bs) || !aligned_to(y, bs) || !aligned_to(weight, ws) ||
      !aligned_to(post_weight, ws) || !aligned_to(gate, ws) || !aligned_to(rstd, 4) || !aligned_to(rstd_f, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  const int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  ResArgs a{};
  a.x = x, a.ldx = ldx, a.f = f, a.ldf = ldf, a.w = weight, a.post = post_weight, a.gate = gate;
  a.h = h, a.ldh = ldh, a.y = y, a.ldy = ldy, a.rstd = rstd, a.rstd_f = rstd_f;
  a.M = M, a.N = static_cast<int32_t>(N), a.w_kind = w_dtype, a.norm_f = post_norm;
  a.scale = scale, a.eps = eps, a.inv_n = 1.0f / static_cast<float>(N);
  a.vec = N % 8 == 0 && on_grid(x, ldx, M) && on_grid(f, ldf, M) && on_grid(h, ldh, M) && on_grid(y, ldy, M);
  a.wvec = aligned16(weight) && aligned16(post_weight) && aligned16(gate);
  auto go = stream_dtype == FP8G_F32 ? (block_dtype == FP8G_F32 ? res_forward<float, float> : res_forward<float, __nv_bfloat16>)
                                     : (block_dtype == FP8G_F32 ? res_forward<__nv_bfloat16, float>
                                                                : res_forward<__nv_bfloat16, __nv_bfloat16>);
  return go(a, static_cast<cudaStream_t>(stream));
}

extern "C" int fp8g_residual_rms_norm_backward_workspace(int64_t M, int64_t N, int64_t* bytes) {
  if (M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFF0 || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = std::max<int64_t>(16, res_ctas(res_form(N), M, true) * 2 * N * 4);
  return FP8G_OK;
}

extern "C" int fp8g_residual_rms_norm_backward(
    const void* dy, int64_t lddy, const void* dh, int64_t lddh, const void* h, int64_t ldh, const void* f, int64_t ldf,
    int32_t stream_dtype, int32_t block_dtype, int64_t M, int64_t N, int32_t post_norm, const void* post_weight,
    const void* gate, float scale, const void* weight, int32_t w_dtype, const float* rstd_f, const float* rstd, void* dx,
    int64_t lddx, void* df, int64_t lddf, float* dweight, float* dgate, float* dpost, void* workspace,
    int64_t workspace_bytes, void* stream) {
  const bool sums = dweight || dgate || dpost;
  if (bad_type(stream_dtype) || bad_type(block_dtype) || bad_type(w_dtype) || M < 0 || M > 0x7FFFFFFF || N < 1 ||
      N > 0x7FFFFFF0 || lddx < N || (dy && (lddy < N || ldh < N)) || (dh && lddh < N) || (f && ldf < N) ||
      (df && lddf < N) || (post_norm & ~1) || (post_weight && !post_norm) || (dgate && !gate) || (dpost && !post_weight))
    return FP8G_ERR_INVALID_ARG;
  if (M > 0 && (!dx || (!dy && !dh) || (!df && (f || post_norm || dgate || dpost)) || (dy && (!h || !rstd)) || (post_norm && (!f || !rstd_f)) ||
                ((dgate || dpost) && !f) || (dweight && !dy)))
    return FP8G_ERR_INVALID_ARG;
  int64_t need = 0;
  fp8g_residual_rms_norm_backward_workspace(M, N, &need);
  if (sums && (!workspace || workspace_bytes < need)) return FP8G_ERR_INVALID_ARG;
  if (M == 0 && !sums) return FP8G_OK;
  const int64_t ss = type_size(stream_dtype), bs = type_size(block_dtype), ws = type_size(w_dtype);
  if (!aligned_to(h, ss) || !aligned_to(dh, ss) || !aligned_to(dx, ss) || !aligned_to(f, bs) || !aligned_to(dy, bs) ||
      !aligned_to(df, bs) || !aligned_to(weight, ws) || !aligned_to(post_weight, ws) || !aligned_to(gate, ws) ||
      !aligned_to(rstd, 4) || !aligned_to(rstd_f, 4) || !aligned_to(dweight, 4) || !aligned_to(dgate, 4) ||
      !aligned_to(dpost, 4) || (sums && !aligned16(workspace)))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  const int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  ResArgs a{};
  a.x = dy ? h : nullptr, a.ldx = ldh, a.f = f, a.ldf = ldf, a.w = weight, a.post = post_weight, a.gate = gate;
  a.dy = dy, a.lddy = lddy, a.dh = dh, a.lddh = lddh, a.dx = dx, a.lddx = lddx, a.df = df, a.lddf = lddf;
  a.rstd = const_cast<float*>(rstd), a.rstd_f = const_cast<float*>(rstd_f);
  a.parts = sums ? static_cast<float*>(workspace) : nullptr;
  a.M = M, a.N = static_cast<int32_t>(N), a.w_kind = w_dtype, a.norm_f = post_norm;
  a.scale = scale, a.inv_n = 1.0f / static_cast<float>(N);
  a.vec = N % 8 == 0 && on_grid(a.x, ldh, M) && on_grid(f, ldf, M) && on_grid(dy, lddy, M) && on_grid(dh, lddh, M) &&
          on_grid(dx, lddx, M) && on_grid(df, lddf, M);
  a.wvec = aligned16(weight) && aligned16(post_weight) && aligned16(gate);
  const ResJoin j{a.parts, post_weight, gate, dweight, dgate, dpost, 0, a.N, w_dtype, scale};
  auto go = stream_dtype == FP8G_F32 ? (block_dtype == FP8G_F32 ? res_backward<float, float> : res_backward<float, __nv_bfloat16>)
                                     : (block_dtype == FP8G_F32 ? res_backward<__nv_bfloat16, float>
                                                                : res_backward<__nv_bfloat16, __nv_bfloat16>);
  return go(a, j, static_cast<cudaStream_t>(stream));
}
