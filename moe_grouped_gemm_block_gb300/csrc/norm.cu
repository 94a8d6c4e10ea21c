// norm.cu -- layer norm over the rows of a matrix and its gradients.
//
//     mu_m = mean_n x,   r_m = 1 / sqrt(mean_n (x - mu)^2 + eps),   y = (x - mu) r w + b
//     with h = (x - mu) r and g = dy w:
//     dx = r (g - mean_n g - h mean_n (g h)),   dw = sum_m dy h,   db = sum_m dy
//
// All sums are taken in fp32; the variance is the mean of the squared differences from the mean
// (a second pass over the row), not the difference of two large sums.

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormMaxParts = 304;  // partial rows of the weight gradients' sums

// One CTA a row, any length and alignment: the row is read three times (from L1 / L2 after the first).
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads) layer_norm_any_kernel(
    const TX* __restrict__ x, int64_t N, int64_t ldx, const void* __restrict__ w, const void* __restrict__ b,
    int32_t w_dtype, float eps, TY* __restrict__ y, int64_t ldy, float* __restrict__ mean,
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
    const float wn = w ? load_any(w, w_dtype, n) : 1.0f, bn = b ? load_any(b, w_dtype, n) : 0.0f;
    yr[n] = from_f32<TY>((to_f32(xr[n]) - mu) * r * wn + bn);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[m] = mu;
    if (rstd) rstd[m] = r;
  }
}

// The data gradient, one CTA a row, any length and alignment.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads) layer_norm_dx_any_kernel(
    const TY* __restrict__ dy, int64_t lddy, const TX* __restrict__ x, int64_t ldx, const void* __restrict__ w,
    int32_t w_dtype, const float* __restrict__ mean, const float* __restrict__ rstd, int64_t N,
    TX* __restrict__ dx, int64_t lddx) {
  __shared__ float red[2 * 2 * kNormThreads / 32];
  const int64_t m = blockIdx.x;
  const float mu = mean[m], r = rstd[m];
  const TX* xr = x + m * ldx;
  const TY* dyr = dy + m * lddy;
  float s[2] = {0.0f, 0.0f};
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float g = to_f32(dyr[n]) * (w ? load_any(w, w_dtype, n) : 1.0f);
    s[0] += g;
    s[1] += g * ((to_f32(xr[n]) - mu) * r);
  }
  cta_sum<kNormThreads / 32>(s, red, 0);
  const float c1 = s[0] / static_cast<float>(N), c2 = s[1] / static_cast<float>(N);
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float g = to_f32(dyr[n]) * (w ? load_any(w, w_dtype, n) : 1.0f);
    dx[m * lddx + n] = from_f32<TX>((g - c1 - (to_f32(xr[n]) - mu) * r * c2) * r);
  }
}

// Partial sums of the weight gradients: thread = column, CTA row blockIdx.y = a range of rows.
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

// dw and db (either may be null) from the partial rows, summed in their order.
__global__ void __launch_bounds__(kNormThreads) layer_norm_dw_join_kernel(
    const float* __restrict__ parts, int64_t P, int64_t N, float* __restrict__ dw, float* __restrict__ db) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  if (i >= 2 * N) return;
  float s = 0.0f;
  for (int64_t p = 0; p < P; ++p) s += parts[p * 2 * N + i];
  if (i < N) {
    if (dw) dw[i] = s;
  } else if (db) {
    db[i - N] = s;
  }
}

int64_t norm_parts(int64_t M) { return std::min<int64_t>(M, kNormMaxParts); }

bool dtype_ok(int32_t d) { return d == FP8G_BF16 || d == FP8G_F32; }
uintptr_t dtype_size(int32_t d) { return d == FP8G_F32 ? 4 : 2; }

template <typename TX, typename TY>
int layer_norm_launch(const void* x, int64_t M, int64_t N, int64_t ldx, const void* w, const void* b,
                      int32_t w_dtype, float eps, void* y, int64_t ldy, float* mean, float* rstd,
                      cudaStream_t s) {
  layer_norm_any_kernel<TX, TY><<<static_cast<unsigned>(M), kNormThreads, 0, s>>>(
      static_cast<const TX*>(x), N, ldx, w, b, w_dtype, eps, static_cast<TY*>(y), ldy, mean, rstd);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

template <typename TX, typename TY>
int layer_norm_backward_launch(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                               int32_t w_dtype, const float* mean, const float* rstd, int64_t M, int64_t N,
                               void* dx, int64_t lddx, float* dw, float* db, float* parts, cudaStream_t s) {
  layer_norm_dx_any_kernel<TX, TY><<<static_cast<unsigned>(M), kNormThreads, 0, s>>>(
      static_cast<const TY*>(dy), lddy, static_cast<const TX*>(x), ldx, w, w_dtype, mean, rstd, N,
      static_cast<TX*>(dx), lddx);
  if (dw || db) {
    const int64_t P = norm_parts(M);
    const dim3 grid(static_cast<unsigned>((N + kNormThreads - 1) / kNormThreads), static_cast<unsigned>(P));
    layer_norm_dw_any_kernel<TX, TY><<<grid, kNormThreads, 0, s>>>(
        static_cast<const TY*>(dy), lddy, static_cast<const TX*>(x), ldx, mean, rstd, M, N, parts);
    layer_norm_dw_join_kernel<<<static_cast<unsigned>((2 * N + kNormThreads - 1) / kNormThreads), kNormThreads, 0,
                                s>>>(parts, P, N, dw, db);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
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
  return go(x, M, N, ldx, weight, bias, w_dtype, eps, y, ldy, mean, rstd, static_cast<cudaStream_t>(stream));
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
  return go(dy, lddy, x, ldx, weight, w_dtype, mean, rstd, M, N, dx, lddx, dweight, dbias,
            static_cast<float*>(workspace), s);
}
