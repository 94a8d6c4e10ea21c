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
// part of a warp (short rows) or by a CTA (see Columns), while the next ones are on their way.  Longer rows than those hold
// are read again for each step ("any").  One sum a column serves both dgate and dpost, as S does not depend on them.
// (The gradient is in resnorm_grad.cu.)
//
// Bound by memory.

#include "resnorm.cuh"

namespace fp8g {
namespace {

template <typename TS, typename TB, int LPR, int V, bool VEC>
__global__ void __launch_bounds__(LPR ? 256 : kResMaxThreads, V == 4 || !VEC ? 1 : 2) residual_norm_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  extern __shared__ __align__(16) unsigned char stage_memory[];
  using Cols = Columns<VEC, V>;
  constexpr int kRows = LPR ? 256 / (LPR ? LPR : 1) : 1;
  const int mine = LPR ? static_cast<int>(threadIdx.x) / (LPR ? LPR : 1) : 0;
  const Cols col{LPR ? static_cast<int>(threadIdx.x) % (LPR ? LPR : 1) : static_cast<int>(threadIdx.x),
                 LPR ? LPR : static_cast<int>(blockDim.x), a.N,
                 VEC && a.M > 1 ? static_cast<int>((blockIdx.x * kRows + mine) % 8 * (a.ldx & 7)) & 7 : 0};
  if (!LPR) res_sum_init(red);
  const uint32_t slots = smem_u32(stage_memory), f_at = blockDim.x * Cols::template slot_bytes<TS>();
  const uint32_t stage = f_at + (a.f ? blockDim.x * Cols::template slot_bytes<TB>() : 0u);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  const TS* x_rows = static_cast<const TS*>(a.x);
  const TB* f_rows = static_cast<const TB*>(a.f);
  // the weights of y, and of f: post gate scale
  float* kept = reinterpret_cast<float*>(stage_memory + a.stages * stage);
  float *kept_w = nullptr, *kept_f = nullptr;
  const bool f_weights = a.post || a.gate;
  if (a.keep) {
    if (a.w) col.keep_weights(kept_w = kept, a.w, nullptr, a.w_kind, 1.0f);
    if (f_weights) col.keep_weights(kept_f = kept + (a.w ? blockDim.x * Cols::weight_bytes() / 4 : 0), a.post, a.gate, a.w_kind, a.scale);
  }
  auto bring = [&](int64_t m, int s) {
    if (m < a.M) {
      col.copy(slots + s * stage, x_rows + m * a.ldx);
      if (f_rows) col.copy(slots + s * stage + f_at, f_rows + m * a.ldf);
    }
    cp_async_commit();
  };
  int phase = 0, s = 0;
  int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows;
  for (int i = 0; i < a.stages; ++i) bring(m0 + mine + i * step, i);
  for (; m0 < a.M; m0 += step) {
    const int64_t m = m0 + mine;
    const bool real = m < a.M;
    Raw8<TB> rf[V];
    float2 x[V][4];
    cp_async_wait(a.stages - 1);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Raw8<TS> r;
      col.load(r, slots + s * stage, x_rows + m * a.ldx, v, real);
      r.get(x[v]);
      if (f_rows) col.load(rf[v], slots + s * stage + f_at, f_rows + m * a.ldf, v, real);
    }
    bring(m + a.stages * step, s);
    if (++s == a.stages) s = 0;
    if (f_rows) {
      float by = f_weights ? 1.0f : a.scale;
      if (a.norm_f) {
        float2 sq = both(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float2 f[4];
          rf[v].get(f);
#pragma unroll
          for (int j = 0; j < 4; ++j) sq = __ffma2_rn(f[j], f[j], sq);
        }
        float q = sq.x + sq.y;
        q = root_inverse(res_sum<LPR>(q, red, phase) * a.inv_n, a.eps);
        if (col.t == 0 && real && a.rstd_f) a.rstd_f[m] = q;
        by *= q;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 f[4];
        rf[v].get(f);
        if (f_weights) col.times(kept_f, a.post, a.gate, a.w_kind, a.scale, v, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[v][j] = __ffma2_rn(both(by), f[j], x[v][j]);
        if (real && a.h) col.store(static_cast<TS*>(a.h) + m * a.ldh, v, x[v]);
      }
    }
    if (!a.y) continue;
    float2 sq = both(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) sq = __ffma2_rn(x[v][j], x[v][j], sq);
    float q = sq.x + sq.y;
    q = root_inverse(res_sum<LPR>(q, red, phase) * a.inv_n, a.eps);
    if (col.t == 0 && real && a.rstd) a.rstd[m] = q;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[v][j] = __fmul2_rn(x[v][j], both(q));
      if (a.w) col.times(kept_w, a.w, nullptr, a.w_kind, 1.0f, v, x[v]);
      if (real) col.store(static_cast<TB*>(a.y) + m * a.ldy, v, x[v]);
    }
  }
}

// Rows of any length: a CTA a row, which reads it again for each step.
template <typename TS, typename TB>
__global__ void __launch_bounds__(kResMaxThreads) residual_norm_any_kernel(const ResArgs a) {
  __shared__ __align__(16) float red[2][32];
  res_sum_init(red);
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

template <typename TS, typename TB, bool VEC>
int res_forward(ResArgs a, bool shifted, const DeviceInfo* dev, cudaStream_t s) {
  const ResForm f = res_form(a.N, shifted, false);
  auto go = f.lpr == 8    ? residual_norm_kernel<TS, TB, VEC ? 8 : 32, 1, VEC>
            : f.lpr == 16 ? residual_norm_kernel<TS, TB, VEC ? 16 : 32, 1, VEC>
            : f.lpr == 32 ? (f.v == 1 ? residual_norm_kernel<TS, TB, 32, 1, VEC> : residual_norm_kernel<TS, TB, 32, 2, VEC>)
            : f.v == 1    ? residual_norm_kernel<TS, TB, 0, 1, VEC>
            : f.v == 2    ? residual_norm_kernel<TS, TB, 0, 2, VEC>
                          : residual_norm_kernel<TS, TB, 0, 4, VEC>;
  const int rows = f.lpr > 0 && !VEC ? 8 : f.rows;
  const int per_sm = f.v == 4 || f.lpr < 0 ? 1 : std::max(2, 1024 / f.threads);
  const int64_t values = static_cast<int64_t>(f.threads) * f.v * 8;
  const ResShared sh = res_shared(values * ((VEC || sizeof(TS) == 4 ? sizeof(TS) : 0) +
                                            (a.f && (VEC || sizeof(TB) == 4) ? sizeof(TB) : 0)),
                                  values * 4 * ((a.w ? 1 : 0) + (a.post || a.gate ? 1 : 0)), per_sm);
  const bool any = f.lpr < 0 || sh.stages == 0;
  if (any) {
    residual_norm_any_kernel<TS, TB><<<static_cast<unsigned>(std::min<int64_t>(a.M, 2 * dev->sm_count)), kResMaxThreads, 0,
                                       s>>>(a);
  } else {
    a.stages = sh.stages;
    const int st = allow_shared_memory(reinterpret_cast<const void*>(go), sh.bytes + 1024);  // (and what is static)
    if (st != FP8G_OK) return st;
    // (a multiple of 8 where a CTA takes more than one row: see Columns)
    const int64_t ctas = std::min<int64_t>((a.M + rows - 1) / rows, int64_t{1} * dev->sm_count / 8 * 8 * per_sm);
    a.keep = sh.weights && a.M > 4 * rows * ctas;  // (few rows a CTA: not worth it)
    go<<<static_cast<unsigned>(ctas), f.threads, static_cast<size_t>(sh.bytes), s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

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
  const ResGrid grid = res_grid(M, N, {{x, ldx}, {f, ldf}, {h, ldh}, {y, ldy}});
  const bool vec = grid != ResGrid::kNone;
  using B = __nv_bfloat16;
  auto go = stream_dtype == FP8G_F32
                ? (block_dtype == FP8G_F32 ? (vec ? res_forward<float, float, true> : res_forward<float, float, false>)
                                           : (vec ? res_forward<float, B, true> : res_forward<float, B, false>))
                : (block_dtype == FP8G_F32 ? (vec ? res_forward<B, float, true> : res_forward<B, float, false>)
                                           : (vec ? res_forward<B, B, true> : res_forward<B, B, false>));
  return go(a, grid == ResGrid::kShifted, dev, static_cast<cudaStream_t>(stream));
}
