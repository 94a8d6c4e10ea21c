// resnorm_grad.cu -- the gradient of the norms around a block (the formulas: resnorm.cu).
//
// A row takes two sums, one after the other, and gives two results; a column's sums over the rows stay in the registers
// of the threads that have the column, and leave a partial sum a CTA that a second, dependent launch joins in order.

#include "resnorm.cuh"

namespace fp8g {
namespace {

// (V 4: a row's values are read again from their stage for the second step, instead of held in registers.)
template <typename TS, typename TB, int LPR, int V, bool VEC>
__global__ void __launch_bounds__(LPR ? 256 : kResMaxThreads, LPR ? 2 : 1)
    residual_norm_backward_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  extern __shared__ __align__(16) unsigned char stage_memory[];  // (in the end, LPR: [2][N] sums)
  using Cols = Columns<VEC, V>;
  constexpr bool kAgain = V == 4;
  griddep_launch_dependents();
  constexpr int kRows = LPR ? 256 / (LPR ? LPR : 1) : 1;
  const int mine = LPR ? static_cast<int>(threadIdx.x) / (LPR ? LPR : 1) : 0;
  const Cols col{LPR ? static_cast<int>(threadIdx.x) % (LPR ? LPR : 1) : static_cast<int>(threadIdx.x),
                 LPR ? LPR : static_cast<int>(blockDim.x), a.N,
                 VEC && a.M > 1 ? static_cast<int>((blockIdx.x * kRows + mine) % 8 * (a.lddx & 7)) & 7 : 0};
  if (!LPR) res_sum_init(red);
  const uint32_t slots = smem_u32(stage_memory);
  const uint32_t one_s = blockDim.x * Cols::template slot_bytes<TS>(), one_b = blockDim.x * Cols::template slot_bytes<TB>();
  const uint32_t y_at = one_s, dh_at = a.dy ? one_s + one_b : 0u, f_at = dh_at + (a.dh ? one_s : 0u);
  const uint32_t stage = f_at + (a.f ? one_b : 0u);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const TS *h_rows = static_cast<const TS*>(a.x), *dh_rows = static_cast<const TS*>(a.dh);
  const TB *dy_rows = static_cast<const TB*>(a.dy), *f_rows = static_cast<const TB*>(a.f);
  // the weights of dy, and of dx: post gate scale
  float* kept = reinterpret_cast<float*>(stage_memory + a.stages * stage);
  float *kept_w = nullptr, *kept_f = nullptr;
  const bool w_weights = a.dy && a.w, f_weights = a.df && (a.post || a.gate);
  if (a.keep) {
    if (w_weights) col.keep_weights(kept_w = kept, a.w, nullptr, a.w_kind, 1.0f);
    if (f_weights) col.keep_weights(kept_f = kept + (w_weights ? blockDim.x * Cols::weight_bytes() / 4 : 0), a.post, a.gate, a.w_kind, a.scale);
  }
  auto bring = [&](int64_t m, int s) {
    if (m < a.M) {
      const uint32_t to = slots + s * stage;
      if (dy_rows) {
        col.copy(to, h_rows + m * a.ldx);
        col.copy(to + y_at, dy_rows + m * a.lddy);
      }
      if (dh_rows) col.copy(to + dh_at, dh_rows + m * a.lddh);
      if (f_rows) col.copy(to + f_at, f_rows + m * a.ldf);
    }
    cp_async_commit();
  };
  int phase = 0, st = 0;
  float2 dw[V][4], df_sum[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[v][j] = df_sum[v][j] = both(0.0f);
  int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows;
  for (int i = 0; i < a.stages; ++i) bring(m0 + mine + i * step, i);
  // the rows' statistics, a row ahead
  float next_r = 0.0f, next_rf = 1.0f;
  auto statistics = [&](int64_t m) {
    if (m < a.M) {
      if (dy_rows) next_r = a.rstd[m];
      if (a.norm_f) next_rf = a.rstd_f[m];
    }
  };
  statistics(m0 + mine);
  for (; m0 < a.M; m0 += step) {
    const int64_t m = m0 + mine;
    const bool real = m < a.M;
    const uint32_t from = slots + st * stage;
    Raw8<TS> rh[V], rd[V];
    Raw8<TB> ry[V], rf[V];
    auto load_first = [&](int v) {
      col.load(rh[v], from, h_rows + m * a.ldx, v, real);
      col.load(ry[v], from + y_at, dy_rows + m * a.lddy, v, real);
    };
    auto load_second = [&](int v) {
      if (dh_rows) col.load(rd[v], from + dh_at, dh_rows + m * a.lddh, v, real);
      else rd[v].zero();
      if (f_rows) col.load(rf[v], from + f_at, f_rows + m * a.ldf, v, real);
    };
    const float r = next_r, rf_ = next_rf;
    statistics(m + step);
    cp_async_wait(a.stages - 1);
    float s = 0.0f;
    if constexpr (!kAgain) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (dy_rows) load_first(v);
        load_second(v);
      }
      bring(m + a.stages * step, st);
    }
    if (dy_rows) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (kAgain) load_first(v);
        float2 g[4], e[4];
        ry[v].get(g);
        rh[v].get(e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = __fmul2_rn(e[j], both(r));
          dw[v][j] = __ffma2_rn(g[j], e[j], dw[v][j]);
        }
        if (w_weights) col.times(kept_w, a.w, nullptr, a.w_kind, 1.0f, v, g);
        float2 sum = both(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = __ffma2_rn(g[j], e[j], sum);
        s += sum.x + sum.y;
      }
      s = res_sum<LPR>(s, red, phase) * a.inv_n * r;  // e once more is h r
    }
    float2 dx[V][4];
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (kAgain) {
        if (dy_rows) load_first(v);
        load_second(v);
      }
      rd[v].get(dx[v]);
      if (dy_rows) {
        float2 g[4], e[4];
        ry[v].get(g);
        rh[v].get(e);
        if (w_weights) col.times(kept_w, a.w, nullptr, a.w_kind, 1.0f, v, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) dx[v][j] = __ffma2_rn(both(r), __ffma2_rn(e[j], both(-s), g[j]), dx[v][j]);
      }
      if (real) col.store(static_cast<TS*>(a.dx) + m * a.lddx, v, dx[v]);
      if (!a.df) continue;
      float2 k[4];
      if (f_rows) {
        rf[v].get(k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          k[j] = __fmul2_rn(k[j], both(rf_));
          df_sum[v][j] = __ffma2_rn(dx[v][j], k[j], df_sum[v][j]);
        }
      }
      if (f_weights) {
        col.times(kept_f, a.post, a.gate, a.w_kind, a.scale, v, dx[v]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) dx[v][j] = __fmul2_rn(dx[v][j], both(a.scale));
      }
      if (a.norm_f) {
        float2 sum = both(0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = __ffma2_rn(dx[v][j], k[j], sum);
        q += sum.x + sum.y;
      }
    }
    if (a.df) {
      if (a.norm_f) q = res_sum<LPR>(q, red, phase) * a.inv_n;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.norm_f) {
          float2 k[4];
          if constexpr (kAgain) col.load(rf[v], from + f_at, f_rows + m * a.ldf, v, real);
          rf[v].get(k);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dx[v][j] = __fmul2_rn(both(rf_), __ffma2_rn(k[j], both(-q * rf_), dx[v][j]));
        }
        if (real) col.store(static_cast<TB*>(a.df) + m * a.lddf, v, dx[v]);
      }
    }
    if constexpr (kAgain) bring(m + a.stages * step, st);
    if (++st == a.stages) st = 0;
  }
  if (!a.parts) return;
  float* out = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
  if constexpr (LPR == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col.has(v, j)) {
          out[col.at(v, j)] = j & 1 ? dw[v][j / 2].y : dw[v][j / 2].x;
          out[a.N + col.at(v, j)] = j & 1 ? df_sum[v][j / 2].y : df_sum[v][j / 2].x;
        }
  } else {
    // the CTA's rows one after the other (their columns may lie shifted)
    float* sums = reinterpret_cast<float*>(stage_memory);
    cp_async_wait(0);
    __syncthreads();  // nobody's stage is in use any more
    for (int r = 0; r < kRows; ++r) {
      if (mine == r) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col.has(v, j)) {
              float* p = sums + col.at(v, j);
              p[0] = (r ? p[0] : 0.0f) + (j & 1 ? dw[v][j / 2].y : dw[v][j / 2].x);
              p[a.N] = (r ? p[a.N] : 0.0f) + (j & 1 ? df_sum[v][j / 2].y : df_sum[v][j / 2].x);
            }
      }
      __syncthreads();
    }
    for (int n = threadIdx.x; n < 2 * a.N; n += blockDim.x) out[n] = sums[n];
  }
}

// Rows of any length: a CTA a row, which reads it again for each step and adds its column sums up in its place of the
// workspace.
template <typename TS, typename TB>
__global__ void __launch_bounds__(kResMaxThreads) residual_norm_backward_any_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  griddep_launch_dependents();
  res_sum_init(red);
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


// CTAs that are resident on an SM: 512 threads of 128 registers.
int res_grad_per_sm(const ResForm& f) { return f.lpr > 0 ? 2 : f.lpr < 0 ? 1 : std::min(4, std::max(1, 512 / f.threads)); }
// CTAs of a call: rows have to stay with their CTA for the column sums, so no more than are resident.
int64_t res_grad_ctas(const ResForm& f, int64_t M) {
  return std::min<int64_t>((M + f.rows - 1) / f.rows, 152 * res_grad_per_sm(f));
}

template <typename TS, typename TB, bool VEC>
int res_backward(ResArgs a, const ResJoin& j, bool shifted, cudaStream_t s) {
  const ResForm f = res_form(a.N, shifted, true);
  unsigned ctas = static_cast<unsigned>(res_grad_ctas(f, a.M));
  auto go = f.lpr == 8    ? residual_norm_backward_kernel<TS, TB, VEC ? 8 : 32, 1, VEC>
            : f.lpr == 16 ? residual_norm_backward_kernel<TS, TB, VEC ? 16 : 32, 1, VEC>
            : f.lpr == 32 ? (f.v == 1 ? residual_norm_backward_kernel<TS, TB, 32, 1, VEC>
                                      : residual_norm_backward_kernel<TS, TB, 32, 2, VEC>)
            : f.v == 2    ? residual_norm_backward_kernel<TS, TB, 0, 2, VEC>
                          : residual_norm_backward_kernel<TS, TB, 0, 4, VEC>;
  if (ctas) {
    const int64_t ts = VEC || sizeof(TS) == 4 ? sizeof(TS) : 0, tb = VEC || sizeof(TB) == 4 ? sizeof(TB) : 0;
    const int64_t values = static_cast<int64_t>(f.threads) * f.v * 8;
    const ResShared sh = res_shared(values * ((a.dy ? ts + tb : 0) + (a.dh ? ts : 0) + (a.f ? tb : 0)),
                                    values * 4 * ((a.dy && a.w ? 1 : 0) + (a.df && (a.post || a.gate) ? 1 : 0)),
                                    res_grad_per_sm(f));
    if (f.lpr < 0 || sh.stages == 0) {
      residual_norm_backward_any_kernel<TS, TB><<<ctas, kResMaxThreads, 0, s>>>(a);
    } else {
      a.stages = sh.stages;
      a.keep = sh.weights && a.M > int64_t{4} * f.rows * ctas;  // (few rows a CTA: not worth it)
      const size_t smem = static_cast<size_t>(std::max<int64_t>(sh.bytes, f.lpr > 0 ? 8 * a.N : 0));
      const int st = allow_shared_memory(reinterpret_cast<const void*>(go), smem + 1024);  // (and what is static)
      if (st != FP8G_OK) return st;
      go<<<ctas, f.threads, smem, s>>>(a);
    }
    if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  }
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

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_residual_rms_norm_backward_workspace(int64_t M, int64_t N, int64_t* bytes) {
  if (M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFF0 || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = std::max<int64_t>(16, std::max(res_grad_ctas(res_form(N, false, true), M), res_grad_ctas(res_form(N, true, true), M)) * 2 * N * 4);
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
  const ResGrid grid = res_grid(M, N, {{a.x, ldh}, {f, ldf}, {dy, lddy}, {dh, lddh}, {dx, lddx}, {df, lddf}});
  const bool vec = grid != ResGrid::kNone;
  const ResJoin j{a.parts, post_weight, gate, dweight, dgate, dpost, 0, a.N, w_dtype, scale};
  using B = __nv_bfloat16;
  auto go = stream_dtype == FP8G_F32
                ? (block_dtype == FP8G_F32 ? (vec ? res_backward<float, float, true> : res_backward<float, float, false>)
                                           : (vec ? res_backward<float, B, true> : res_backward<float, B, false>))
                : (block_dtype == FP8G_F32 ? (vec ? res_backward<B, float, true> : res_backward<B, float, false>)
                                           : (vec ? res_backward<B, B, true> : res_backward<B, B, false>));
  return go(a, j, grid == ResGrid::kShifted, static_cast<cudaStream_t>(stream));
}
