// resnorm_grad.cu -- the gradient of the norms around a block (the formulas: resnorm.cu).
//
// A row takes two means, of which the second needs the first's result, and gives two results; a column's sums over the rows
// stay in the registers of the threads that have the column, and leave a partial sum a CTA that a second, dependent
// launch joins in order.
//
// Bound by memory where a matrix is fp32 and by its instructions' latencies where all are bf16 (an SM holds 16 warps of 128
// registers; 39 instructions a value, of which the unpacking of bf16, twice, is a fifth):
//   8192 x 7168, fp32 stream and bf16 block: 192 us (81% of the copy rate);  16384 x 4096: 195 (91%)
//   4096 x 7168 bf16: 87 (60%);  16384 x 2048 bf16: 84 (71%);  16384 x 64 bf16: 12 (16%)
//   with both norms: 4096 x 12288 bf16 203 (44%), fp32 stream 241 (55%);  4096 x 4099 bf16 92 (32%), fp32 118 (50%);  4096 x
//   4096 on grids of their own bf16 119 (25%), fp32 126 (47%);  1024 x 20000 bf16 632 (6%)
//   a plain residual, whose f is not read: 8192 x 7168, fp32 stream 158 us (88%), bf16 128 (68%)
// What was slower: fp32 rows in eights a thread (a warp's accesses then touch twice the sectors: 252 us), both means from
// one sum over the row (sum q k = sum p dh k + r (sum p g k - s sum p e k): as fast with fp32, 103 instead of 90 us with
// bf16), bulk copies with a barrier a stage (equal, and 222 instead of 194 us at 16384 x 4096), a second stage for three of
// the four matrices (kept, worth 1%), 32 warps with a unit each (equal).

#include "resnorm.cuh"

namespace fp8g {
namespace {

template <typename TS, typename TB, int LPR, int EIGHTS, int MODE>
__global__ void __launch_bounds__(LPR ? 256 : kResMaxThreads, LPR ? 2 : 1) residual_norm_backward_kernel(const ResArgs a) {
  __shared__ float red[2][32];
  extern __shared__ __align__(16) unsigned char shared[];  // (in the end, LPR: [2][N] sums)
  constexpr int G = res_unit<TS, TB>(), V = EIGHTS * 8 / G, H = G / 2;
  using Cols = Columns<MODE, G, V>;
  using SS = Source<TS, MODE, G, V>;
  using SB = Source<TB, MODE, G, V>;
  griddep_launch_dependents();
  FP8G_RES_ROWS(a.lddx)
  if (!LPR) res_sum_init(red, a.ranks);
  // the weights of dy, and of dx: post gate scale; zeros for a matrix that is not there; the stages
  float4 *w_at = reinterpret_cast<float4*>(shared), *f_at = w_at + 2 * EIGHTS * blockDim.x;
  col.keep_weights(w_at, a.w, nullptr, a.w_kind, 1.0f);
  col.keep_weights(f_at, a.post, a.gate, a.w_kind, a.scale);
  const uint32_t one_s = blockDim.x * SS::thread_bytes(), one_b = blockDim.x * SB::thread_bytes();
  const uint32_t zeros = smem_u32(f_at + 2 * EIGHTS * blockDim.x);
  const bool missing = !a.dy || !a.dh || !a.f;
  const uint32_t h_at = zeros + (missing ? max(one_s, one_b) : 0u), dy_at = h_at + (a.dy ? one_s : 0u);
  const uint32_t dh_at = dy_at + (a.dy ? one_b : 0u), stage = dh_at + (a.dh ? one_s : 0u) - h_at;
  const uint32_t k_at = h_at + a.stages * stage;
  SS sh, sd;
  SB sy, sf;
  int64_t ahead = m_first + mine;  // the row that is copied next
  sh.init(a.dy ? a.x : nullptr, ahead, a.ldx, step, a.dy ? h_at : zeros, stage, a.stages, col);
  sy.init(a.dy, ahead, a.lddy, step, a.dy ? dy_at : zeros, stage, a.stages, col);
  sd.init(a.dh, ahead, a.lddh, step, a.dh ? dh_at : zeros, stage, a.stages, col);
  sf.init(a.f, ahead, a.ldf, step, a.f ? k_at : zeros, one_b, a.stages_f, col);
  // f's row, which may lie one behind the others', is a group of its own before theirs
  int64_t ahead_f = ahead;
  auto bring_f = [&](int s) {
    if (ahead_f < a.M) sf.copy(s, col);
    ahead_f += step;
    cp_async_commit();
  };
  auto bring = [&](int s) {
    if (ahead < a.M) {
      sh.copy(s, col);
      sy.copy(s, col);
      sd.copy(s, col);
    }
    ahead += step;
    cp_async_commit();
  };
  auto advance = [&] {
    if (a.dy) sh.row += sh.step, sy.row += sy.step;
    if (a.dh) sd.row += sd.step;
  };
  auto advance_f = [&] {
    if (a.f) sf.row += sf.step;
  };
  // the rows' statistics, a row ahead
  float next_r = 0.0f, next_rf = 1.0f;
  auto statistics = [&](int64_t m) {
    if (m < a.M) {
      if (a.dy) next_r = a.rstd[m];
      if (a.norm_f) next_rf = a.rstd_f[m];
    }
  };
  statistics(ahead);
  int phase = 0, st = 0, st_f = 0;
  float2 dw[V][H], df_sum[V][H];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < H; ++j) dw[v][j] = df_sum[v][j] = both(0.0f);
  // (where a matrix is not staged but loaded at its row's turn, all keep to one stage)
  constexpr bool kAhead = SS::kStaged && SB::kStaged;
  const int later = !kAhead ? 0 : a.stages == a.stages_f ? 2 * a.stages - 2 : 2 * a.stages_f - 1;
  for (int i = 0; i < a.stages; ++i) {
    if (i >= a.stages - a.stages_f) {
      bring_f(i - (a.stages - a.stages_f));
      if (kAhead) advance_f();
    }
    bring(i);
    if (kAhead) advance();
  }
  for (int64_t m0 = m_first; m0 < a.M; m0 += step) {
    const int64_t m = m0 + mine;
    const bool real = LPR == 0 || m < a.M;
    const float r = next_r, rf = next_rf;
    statistics(m + step);
    Unit<TS, G> rh[V], rd[V];
    Unit<TB, G> ry[V], rk[V];
    cp_async_wait(later);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (real) {
        sh.load(rh[v], st, v, col);
        sy.load(ry[v], st, v, col);
        sd.load(rd[v], st, v, col);
        sf.load(rk[v], st_f, v, col);
      } else {
        rh[v].zero(), ry[v].zero(), rd[v].zero(), rk[v].zero();
      }
    }
    if (!kAhead) advance(), advance_f();
    bring_f(st_f);
    bring(st);
    if (kAhead) advance(), advance_f();
    if (++st == a.stages) st = 0;
    if (++st_f == a.stages_f) st_f = 0;
    float2 sum = both(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float2 g[H], e[H];
      ry[v].get(g);
      rh[v].get(e);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        e[j] = __fmul2_rn(e[j], both(r));
        dw[v][j] = __ffma2_rn(g[j], e[j], dw[v][j]);
      }
      col.times(w_at, v, g);
#pragma unroll
      for (int j = 0; j < H; ++j) sum = __ffma2_rn(g[j], e[j], sum);
    }
    const float s = a.dy ? -res_sum<LPR>(sum.x + sum.y, red, phase, a.ranks) * a.inv_n * r : 0.0f;  // (e once more is h r)
    float2 dx[V][H];
    sum = both(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float2 g[H], h[H], k[H];
      rd[v].get(dx[v]);
      ry[v].get(g);
      rh[v].get(h);
      rk[v].get(k);
      col.times(w_at, v, g);
#pragma unroll
      for (int j = 0; j < H; ++j) dx[v][j] = __ffma2_rn(both(r), __ffma2_rn(h[j], both(s), g[j]), dx[v][j]);
      if (real) col.store(static_cast<TS*>(a.dx) + m * a.lddx, v, dx[v]);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        k[j] = __fmul2_rn(k[j], both(rf));
        df_sum[v][j] = __ffma2_rn(dx[v][j], k[j], df_sum[v][j]);
      }
      col.times(f_at, v, dx[v]);
#pragma unroll
      for (int j = 0; j < H; ++j) sum = __ffma2_rn(dx[v][j], k[j], sum);
    }
    if (!a.df) continue;
    if (a.norm_f) {
      const float c = -res_sum<LPR>(sum.x + sum.y, red, phase, a.ranks) * a.inv_n * rf;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 k[H];
        rk[v].get(k);
#pragma unroll
        for (int j = 0; j < H; ++j) dx[v][j] = __fmul2_rn(both(rf), __ffma2_rn(k[j], both(c), dx[v][j]));
      }
    }
    if (real) {
#pragma unroll
      for (int v = 0; v < V; ++v) col.store(static_cast<TB*>(a.df) + m * a.lddf, v, dx[v]);
    }
  }
  if (!LPR && a.ranks > 1) cluster_sync();  // (nobody leaves while it may still be written to)
  if (!a.parts) return;
  float* out = a.parts + block * 2 * a.N;
  if constexpr (LPR == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (col.has(v, j)) {
          out[col.at(v, j)] = j & 1 ? dw[v][j / 2].y : dw[v][j / 2].x;
          out[a.N + col.at(v, j)] = j & 1 ? df_sum[v][j / 2].y : df_sum[v][j / 2].x;
        }
  } else {
    // the rows of a warp, where they have the same columns, then the warps (else the rows) one after the other
    float* sums = reinterpret_cast<float*>(shared);
    cp_async_wait(0);
    __syncthreads();  // nobody's places are in use any more
    if constexpr (MODE != kShifted) {
#pragma unroll
      for (int off = 16; off >= (LPR ? LPR : 1); off >>= 1)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            dw[v][j].x += __shfl_xor_sync(0xffffffffu, dw[v][j].x, off);
            dw[v][j].y += __shfl_xor_sync(0xffffffffu, dw[v][j].y, off);
            df_sum[v][j].x += __shfl_xor_sync(0xffffffffu, df_sum[v][j].x, off);
            df_sum[v][j].y += __shfl_xor_sync(0xffffffffu, df_sum[v][j].y, off);
          }
    }
    constexpr int kTurns = MODE == kShifted ? kRows : 8;
    const int turn = MODE == kShifted ? mine : (threadIdx.x & 31) < (LPR ? LPR : 1) ? static_cast<int>(threadIdx.x >> 5) : -1;
    for (int q = 0; q < kTurns; ++q) {
      if (turn == q) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int j = 0; j < G; ++j)
            if (col.has(v, j)) {
              float* p = sums + col.at(v, j);
              p[0] = (q ? p[0] : 0.0f) + (j & 1 ? dw[v][j / 2].y : dw[v][j / 2].x);
              p[a.N] = (q ? p[a.N] : 0.0f) + (j & 1 ? df_sum[v][j / 2].y : df_sum[v][j / 2].x);
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
  __shared__ float red[2][32];
  griddep_launch_dependents();
  res_sum_init(red, 1);
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
      s = res_sum<0>(s, red, phase, 1) * a.inv_n * r * r;
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
      s2 = res_sum<0>(s2, red, phase, 1) * a.inv_n * rf * rf;
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

// The columns' sums from the CTAs' partial ones, in a fixed order: 32 columns a CTA, 32 threads a column with four loads of
// each kind on their way (with 8 threads and one, 16384 x 64 took 24 us instead of 13).
struct ResJoin {
  const float* parts;
  const void *post, *gate;
  float *dw, *dgate, *dpost;
  int32_t P, N, w_kind;
  float scale;
};
constexpr int kJoinSlices = 32;
__global__ void __launch_bounds__(32 * kJoinSlices) residual_norm_join_kernel(const ResJoin a) {
  __shared__ float s[2][kJoinSlices][33];
  griddep_wait();
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5, n = blockIdx.x * 32 + c;
  float w = 0.0f, f = 0.0f;
  if (n < a.N) {
    const float* p = a.parts + n;
    const int64_t row = 2 * static_cast<int64_t>(a.N);
#pragma unroll 4
    for (int i = k; i < a.P; i += kJoinSlices) {
      w += __ldcg(p + i * row);
      f += __ldcg(p + i * row + a.N);
    }
  }
  s[0][k][c] = w;
  s[1][k][c] = f;
  __syncthreads();
  // warp k has column k of the CTA's: a lane a slice
  const int col = blockIdx.x * 32 + k;
  w = warp_sum(s[0][c][k]);
  f = warp_sum(s[1][c][k]) * a.scale;
  if (c > 0 || col >= a.N) return;
  if (a.dw) a.dw[col] = w;
  if (a.dgate) a.dgate[col] = f * (a.post ? load_any(a.post, a.w_kind, col) : 1.0f);
  if (a.dpost) a.dpost[col] = f * (a.gate ? load_any(a.gate, a.w_kind, col) : 1.0f);
}

// CTAs that are resident on an SM: 512 threads of 128 registers.
int res_grad_per_sm(const ResForm& f) { return f.lpr > 0 ? 2 : f.lpr < 0 ? 1 : std::min(4, std::max(1, 512 / f.threads)); }
// Blocks of rows, and partial sums, of a call: rows stay with their CTAs for the column sums, so no more than are resident
// (and, where a block takes several rows, a multiple of 8 of them, see Columns) on the 152 SMs of this GPU: the workspace's
// size, which they are, is asked for without a device.
constexpr int64_t kResGradSms = 152;
int64_t res_grad_blocks(const ResForm& f, int64_t M) {
  return std::min<int64_t>((M + f.rows - 1) / f.rows, kResGradSms * res_grad_per_sm(f) / f.ranks / 8 * 8);
}

template <typename TS, typename TB, int MODE>
int res_backward(ResArgs a, const ResJoin& j, cudaStream_t s) {
  constexpr ResMode kMode = static_cast<ResMode>(MODE);
  const ResForm f = res_form(a.N, kMode, true);
  const unsigned blocks = static_cast<unsigned>(res_grad_blocks(f, a.M));
  if (blocks) {
    const int64_t one_s = f.threads * res_thread_bytes(kMode, f.v, sizeof(TS)), one_b = f.threads * res_thread_bytes(kMode, f.v, sizeof(TB));
    const ResShared sh = res_shared((a.dy ? one_s + one_b : 0) + (a.dh ? one_s : 0), a.f ? one_b : 0,
                                    static_cast<int64_t>(f.threads) * f.v * 64 +
                                        (a.dy && a.dh && a.f ? 0 : std::max(one_s, one_b)), res_grad_per_sm(f));
    if (f.lpr < 0 || sh.stages == 0) {
      residual_norm_backward_any_kernel<TS, TB><<<blocks, kResMaxThreads, 0, s>>>(a);
      if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
    } else {
      constexpr int kSmall = MODE == kSingle ? 32 : 8, kSome = MODE == kSingle ? 32 : 16;
      auto go = f.lpr == 8    ? residual_norm_backward_kernel<TS, TB, kSmall, 1, MODE>
                : f.lpr == 16 ? residual_norm_backward_kernel<TS, TB, kSome, 1, MODE>
                : f.lpr == 32 ? (f.v == 1 ? residual_norm_backward_kernel<TS, TB, 32, 1, MODE>
                                          : residual_norm_backward_kernel<TS, TB, 32, 2, MODE>)
                              : residual_norm_backward_kernel<TS, TB, 0, 2, MODE>;
      a.stages = sh.stages, a.stages_f = sh.stages_f;
      if (MODE == kSingle && sizeof(TS) + sizeof(TB) < 8) a.stages = a.stages_f = 1;  // (see kAhead)
      a.ranks = f.ranks;
      const int st = res_launch(go, int64_t{1} * blocks * f.ranks, f.threads, std::max<int64_t>(sh.bytes, f.lpr > 0 ? 8 * a.N : 0),
                                f.ranks, a, s);
      if (st != FP8G_OK) return st;
    }
  }
  if (!a.parts) return FP8G_OK;
  ResJoin join = j;
  join.P = static_cast<int32_t>(blocks);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((a.N + 31) / 32));
  cfg.blockDim = dim3(32 * kJoinSlices);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = blocks ? 1 : 0;
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
  if (M < 0 || M > 0x7FFFFFFF || N < 1 || N > kResMaxCols || !bytes) return FP8G_ERR_INVALID_ARG;
  int64_t P = 0;
  for (const ResMode mode : {kAligned, kShifted, kSingle}) P = std::max(P, res_grad_blocks(res_form(N, mode, true), M));
  *bytes = std::max<int64_t>(16, P * 2 * N * 4);
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
      N > kResMaxCols || lddx < N || (dy && (lddy < N || ldh < N)) || (dh && lddh < N) || (f && ldf < N) ||
      (df && lddf < N) || (post_norm & ~1) || (post_weight && !post_norm) || (dgate && !gate) || (dpost && !post_weight))
    return FP8G_ERR_INVALID_ARG;
  if (M > 0 && (!dx || (!dy && !dh) || (!df && (f || post_norm || dgate || dpost)) || (dy && (!h || !rstd)) || (post_norm && (!f || !rstd_f)) ||
                ((dgate || dpost) && !f) || (dweight && !dy)))
    return FP8G_ERR_INVALID_ARG;
  if (dx && dx == dh && M > 1 && lddx != lddh) return FP8G_ERR_INVALID_ARG;
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
  // (f is read where something depends on it: df of a plain residual does not, whatever f holds)
  a.x = dy ? h : nullptr, a.ldx = ldh, a.f = post_norm || dgate ? f : nullptr, a.ldf = ldf, a.w = weight, a.post = post_weight, a.gate = gate;
  a.dy = dy, a.lddy = lddy, a.dh = dh, a.lddh = lddh, a.dx = dx, a.lddx = lddx, a.df = df, a.lddf = lddf;
  a.rstd = const_cast<float*>(rstd), a.rstd_f = const_cast<float*>(rstd_f);
  a.parts = sums ? static_cast<float*>(workspace) : nullptr;
  a.M = M, a.N = static_cast<int32_t>(N), a.w_kind = w_dtype, a.norm_f = post_norm;
  a.scale = scale, a.inv_n = 1.0f / static_cast<float>(N);
  const ResMode mode = res_mode(M, N, {{a.x, ldh}, {a.f, ldf}, {dy, lddy}, {dh, lddh}, {dx, lddx}, {df, lddf}});
  const ResJoin j{a.parts, post_weight, gate, dweight, dgate, dpost, 0, a.N, w_dtype, scale};
  using B = __nv_bfloat16;
  auto pick = [mode](auto aligned, auto shifted, auto single) {
    return mode == kAligned ? aligned : mode == kShifted ? shifted : single;
  };
  auto go = stream_dtype == FP8G_F32
                ? (block_dtype == FP8G_F32
                       ? pick(res_backward<float, float, kAligned>, res_backward<float, float, kShifted>, res_backward<float, float, kSingle>)
                       : pick(res_backward<float, B, kAligned>, res_backward<float, B, kShifted>, res_backward<float, B, kSingle>))
                : (block_dtype == FP8G_F32
                       ? pick(res_backward<B, float, kAligned>, res_backward<B, float, kShifted>, res_backward<B, float, kSingle>)
                       : pick(res_backward<B, B, kAligned>, res_backward<B, B, kShifted>, res_backward<B, B, kSingle>));
  return go(a, j, static_cast<cudaStream_t>(stream));
}
