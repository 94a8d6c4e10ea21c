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
// Bound by memory, below some tens of MB by a call's fixed part, and in clusters by their barrier (0.6 us, twice a row).
// Device times, forward, and the share of the copy rate (fp32 / bf16: the stream's and the block's type):
//   8192 x 7168 fp32 / bf16: 124 us (84%);  4096 x 7168 bf16: 41 (84%);  16384 x 512 bf16: 12 (83%)
//   4096 x 12288 fp32 / bf16 with both norms: 201 (44%), without the one after the block 134 (66%)
//   4160 x 7168 fp32 / fp32: 84 us (84%);  58560 x 512 fp32 / bf16: 60 (88%)
//   off the grid alike: 1021 x 4099 fp32 with both norms 15.5 (64%), 4096 x 4099 bf16 28 (71%), with both norms 36 (54%)
//   on grids of their own: 4096 x 4096 with both norms, bf16 102 (19%), fp32 71 (56%);  64 x 7168: 4.4
//   read again for each step: 1024 x 20000 bf16 with both norms 189 (13%)

#include "resnorm.cuh"

namespace fp8g {
namespace {

template <typename TS, typename TB, int LPR, int EIGHTS, int MODE>
__global__ void __launch_bounds__(LPR ? 256 : kResMaxThreads, LPR || MODE != kSingle ? 2 : 1)
    residual_norm_kernel(const ResArgs a) {
  __shared__ float red[2][32];
  extern __shared__ __align__(16) unsigned char shared[];
  constexpr int G = res_unit<TS, TB>(), V = EIGHTS * 8 / G, H = G / 2;
  using Cols = Columns<MODE, G, V>;
  using SX = Source<TS, MODE, G, V>;
  using SF = Source<TB, MODE, G, V>;
  FP8G_RES_ROWS(a.ldx)
  if (!LPR) res_sum_init(red, a.ranks);
  // the weights of y, and of f: post gate scale; the stages
  float4 *w_at = reinterpret_cast<float4*>(shared), *f_at = w_at + 2 * EIGHTS * blockDim.x;
  col.keep_weights(w_at, a.w, nullptr, a.w_kind, 1.0f);
  if (a.f) col.keep_weights(f_at, a.post, a.gate, a.w_kind, a.scale);
  const uint32_t stages = smem_u32(a.f ? f_at + 2 * EIGHTS * blockDim.x : f_at);
  const uint32_t x_bytes = blockDim.x * SX::thread_bytes(), f_bytes = blockDim.x * SF::thread_bytes();
  SX sx{};
  SF sf{};
  int64_t ahead = m_first + mine;  // the row that is copied next
  sx.init(a.x, ahead, a.ldx, step, stages, x_bytes, a.stages, col);
  if (a.f) sf.init(a.f, ahead, a.ldf, step, stages + a.stages * x_bytes, f_bytes, a.stages_f, col);
  // f's row, which may lie one behind the others', is a group of its own before theirs
  int64_t ahead_f = ahead;
  auto bring_f = [&](int s) {
    if (a.f && ahead_f < a.M) sf.copy(s, col);
    if (SF::kStaged) sf.row += sf.step;
    ahead_f += step;
    cp_async_commit();
  };
  auto bring = [&](int s) {
    if (ahead < a.M) sx.copy(s, col);
    if (SX::kStaged) sx.row += sx.step;
    ahead += step;
    cp_async_commit();
  };
  const int later = a.stages == a.stages_f ? 2 * a.stages - 2 : 2 * a.stages_f - 1;
  int phase = 0, s = 0, s_f = 0;
  for (int i = 0; i < a.stages; ++i) {
    if (i >= a.stages - a.stages_f) bring_f(i - (a.stages - a.stages_f));
    bring(i);
  }
  for (int64_t m0 = m_first; m0 < a.M; m0 += step) {
    const int64_t m = m0 + mine;
    const bool real = LPR == 0 || m < a.M;
    Unit<TB, G> rf[V];
    float2 x[V][H];
    cp_async_wait(later);
    if (!SX::kStaged && !real) sx.row = nullptr;
    if (!SF::kStaged && !real) sf.row = nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Unit<TS, G> r;
      sx.load(r, s, v, col);
      r.get(x[v]);
      if (a.f) sf.load(rf[v], s_f, v, col);
    }
    if (!SX::kStaged) sx.row += sx.step;
    if (!SF::kStaged) sf.row += sf.step;
    bring_f(s_f);
    bring(s);
    if (++s == a.stages) s = 0;
    if (++s_f == a.stages_f) s_f = 0;
    if (a.f) {
      float by = 1.0f;
      if (a.norm_f) {
        float2 sq = both(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float2 f[H];
          rf[v].get(f);
#pragma unroll
          for (int j = 0; j < H; ++j) sq = __ffma2_rn(f[j], f[j], sq);
        }
        by = root_inverse(res_sum<LPR>(sq.x + sq.y, red, phase, a.ranks) * a.inv_n, a.eps);
        if (col.t == 0 && rank == 0 && real && a.rstd_f) a.rstd_f[m] = by;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 f[H];
        rf[v].get(f);
        col.times(f_at, v, f);
#pragma unroll
        for (int j = 0; j < H; ++j) x[v][j] = __ffma2_rn(both(by), f[j], x[v][j]);
      }
      if (real && a.h) {
#pragma unroll
        for (int v = 0; v < V; ++v) col.store(static_cast<TS*>(a.h) + m * a.ldh, v, x[v]);
      }
    }
    if (!a.y) continue;
    float2 sq = both(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < H; ++j) sq = __ffma2_rn(x[v][j], x[v][j], sq);
    const float r = root_inverse(res_sum<LPR>(sq.x + sq.y, red, phase, a.ranks) * a.inv_n, a.eps);
    if (col.t == 0 && rank == 0 && real && a.rstd) a.rstd[m] = r;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int j = 0; j < H; ++j) x[v][j] = __fmul2_rn(x[v][j], both(r));
      col.times(w_at, v, x[v]);
      if (real) col.store(static_cast<TB*>(a.y) + m * a.ldy, v, x[v]);
    }
  }
  if (!LPR && a.ranks > 1) cluster_sync();  // (nobody leaves while it may still be written to)
}

// Rows of any length: a CTA a row, which reads it again for each step.
template <typename TS, typename TB>
__global__ void __launch_bounds__(kResMaxThreads) residual_norm_any_kernel(const ResArgs a) {
  __shared__ float red[2][32];
  res_sum_init(red, 1);
  int phase = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const TS* x = static_cast<const TS*>(a.x) + m * a.ldx;
    const TB* f = a.f ? static_cast<const TB*>(a.f) + m * a.ldf : nullptr;
    float by = a.scale;
    if (f && a.norm_f) {
      float s = 0.0f;
      for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) s = fmaf(to_f32(f[n]), to_f32(f[n]), s);
      s = root_inverse(res_sum<0>(s, red, phase, 1) * a.inv_n, a.eps);
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
      s = root_inverse(res_sum<0>(s, red, phase, 1) * a.inv_n, a.eps);
      if (threadIdx.x == 0 && a.rstd) a.rstd[m] = s;
    }
    for (int n = threadIdx.x; n < a.N; n += kResMaxThreads) {  // (h may be x: a value is read before it is written)
      const float v = value(n);
      if (a.y) static_cast<TB*>(a.y)[m * a.ldy + n] = from_f32<TB>(v * s * (a.w ? load_any(a.w, a.w_kind, n) : 1.0f));
      if (f && a.h) static_cast<TS*>(a.h)[m * a.ldh + n] = from_f32<TS>(v);
    }
  }
}

template <typename TS, typename TB, int MODE>
int res_forward(ResArgs a, const DeviceInfo* dev, cudaStream_t s) {
  const ResPlan plan = res_forward_plan(a.N, static_cast<ResMode>(MODE), sizeof(TS), sizeof(TB), a.f != nullptr);
  const ResForm& f = plan.form;
  const ResShared& sh = plan.shared;
  if (sh.stages == 0) {
    residual_norm_any_kernel<TS, TB><<<static_cast<unsigned>(std::min<int64_t>(a.M, 2 * dev->sm_count)), kResMaxThreads, 0,
                                       s>>>(a);
    return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
  }
  constexpr int kSmall = MODE == kSingle ? 32 : 8, kSome = MODE == kSingle ? 32 : 16;
  auto go = f.lpr == 8    ? residual_norm_kernel<TS, TB, kSmall, 1, MODE>
            : f.lpr == 16 ? residual_norm_kernel<TS, TB, kSome, 1, MODE>
            : f.lpr == 32 ? (f.v == 1 ? residual_norm_kernel<TS, TB, 32, 1, MODE> : residual_norm_kernel<TS, TB, 32, 2, MODE>)
            : f.v == 1    ? residual_norm_kernel<TS, TB, 0, 1, MODE>
                          : residual_norm_kernel<TS, TB, 0, 2, MODE>;
  a.stages = sh.stages, a.stages_f = sh.stages_f, a.ranks = f.ranks;
  // (row blocks: a multiple of 8 where a CTA takes more than one, see Columns)
  const int64_t blocks = std::min<int64_t>((a.M + f.rows - 1) / f.rows, int64_t{1} * dev->sm_count * plan.per_sm / f.ranks / 8 * 8);
  return res_launch(go, blocks * f.ranks, f.threads, sh.bytes, f.ranks, a, s);
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
      N > kResMaxCols || ldx < N || (f && ldf < N) || (h && ldh < N) || (y && ldy < N) || (post_norm & ~1) ||
      !(eps >= 0.0f) || (post_weight && !post_norm))
    return FP8G_ERR_INVALID_ARG;
  if (M == 0) return FP8G_OK;  // (no rows: their addresses may all be null)
  if (h == x && h && M > 1 && ldh != ldx) return FP8G_ERR_INVALID_ARG;  // (its rows would lie on others that are still read)
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
  const ResMode mode = res_mode(M, N, {{x, ldx}, {f, ldf}, {h, ldh}, {y, ldy}});
  using B = __nv_bfloat16;
  auto pick = [mode](auto aligned, auto shifted, auto single) {
    return mode == kAligned ? aligned : mode == kShifted ? shifted : single;
  };
  auto go = stream_dtype == FP8G_F32
                ? (block_dtype == FP8G_F32
                       ? pick(res_forward<float, float, kAligned>, res_forward<float, float, kShifted>, res_forward<float, float, kSingle>)
                       : pick(res_forward<float, B, kAligned>, res_forward<float, B, kShifted>, res_forward<float, B, kSingle>))
                : (block_dtype == FP8G_F32
                       ? pick(res_forward<B, float, kAligned>, res_forward<B, float, kShifted>, res_forward<B, float, kSingle>)
                       : pick(res_forward<B, B, kAligned>, res_forward<B, B, kShifted>, res_forward<B, B, kSingle>));
  return go(a, dev, static_cast<cudaStream_t>(stream));
}
