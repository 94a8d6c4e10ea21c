// clip.cu -- the global norm of many gradient tensors, and clipping by it.
//
//     norm = sqrt(sum over all tensors of g^2),   out = g min(1, max_norm / (norm + eps))
//
// The tensors' addresses, sizes and types travel as kernel arguments (up to kClipCap tensors a launch), so
// nothing is copied to the device and a call can be captured into a graph.  Each tensor is cut into chunks;
// a CTA works through the chunks blockIdx.x, blockIdx.x + gridDim.x, ...  Sums of squares are fp32 within a
// CTA and fp64 over the CTAs, in a fixed order.

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipCap = 1024;       // tensors a launch
constexpr int kClipMaxCtas = 608;    // partial sums a launch
constexpr int64_t kClipChunk = 8192; // values a chunk
constexpr int32_t kClipMaxTensors = 1 << 20;
constexpr int64_t kClipMaxValues = int64_t{1} << 42;  // of all tensors together

struct ClipTable {
  const void* grad[kClipCap];
  void* out[kClipCap];
  int64_t numel[kClipCap];
  uint32_t end[kClipCap];  // chunks of the tensors up to and with this one
  uint8_t dtype[kClipCap];
  int32_t n;
};
static_assert(sizeof(ClipTable) <= 32000, "kernel arguments hold 32764 bytes");

// The tensor that chunk c belongs to.
__device__ __forceinline__ int find_tensor(const ClipTable& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c < t.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_part_kernel(const __grid_constant__ ClipTable t,
                                                                      float* __restrict__ parts) {
  __shared__ float red[2 * kClipThreads / 32];
  float s[1] = {0.0f};
  const uint32_t chunks = t.end[t.n - 1];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const int64_t lo = static_cast<int64_t>(c - (i ? t.end[i - 1] : 0u)) * kClipChunk;
    const int64_t hi = min(lo + kClipChunk, t.numel[i]);
    for (int64_t k = lo + threadIdx.x; k < hi; k += kClipThreads) {
      const float v = load_any(t.grad[i], t.dtype[i], k);
      s[0] += v * v;
    }
  }
  cta_sum<kClipThreads / 32>(s, red, 0);
  if (threadIdx.x == 0) parts[blockIdx.x] = s[0];
}

// The norm from the partial sums: the same value in every CTA that calls it.
__device__ __forceinline__ float join_norm(const float* __restrict__ parts, int32_t P) {
  __shared__ double s_sum[kClipThreads];
  double s = 0.0;
  for (int i = threadIdx.x; i < P; i += kClipThreads) s += static_cast<double>(parts[i]);
  s_sum[threadIdx.x] = s;
  __syncthreads();
  for (int off = kClipThreads / 2; off > 0; off >>= 1) {
    if (threadIdx.x < off) s_sum[threadIdx.x] += s_sum[threadIdx.x + off];
    __syncthreads();
  }
  return static_cast<float>(sqrt(s_sum[0]));
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_join_kernel(const float* __restrict__ parts, int32_t P,
                                                                      float* __restrict__ norm) {
  const float n = join_norm(parts, P);
  if (threadIdx.x == 0) *norm = n;
}

__global__ void __launch_bounds__(kClipThreads) grad_clip_kernel(const __grid_constant__ ClipTable t,
                                                                 const float* __restrict__ parts, int32_t P,
                                                                 float max_norm, float eps,
                                                                 float* __restrict__ norm) {
  const float n = join_norm(parts, P);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm) *norm = n;
  const float coef = n + eps <= max_norm ? 1.0f : max_norm / (n + eps);  // a NaN norm makes every output NaN
  const uint32_t chunks = t.end[t.n - 1];
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    if (coef == 1.0f && t.out[i] == t.grad[i]) continue;  // in place and nothing to scale
    const int64_t lo = static_cast<int64_t>(c - (i ? t.end[i - 1] : 0u)) * kClipChunk;
    const int64_t hi = min(lo + kClipChunk, t.numel[i]);
    for (int64_t k = lo + threadIdx.x; k < hi; k += kClipThreads) {
      const float v = load_any(t.grad[i], t.dtype[i], k) * coef;
      if (t.dtype[i] == FP8G_F32) static_cast<float*>(t.out[i])[k] = v;
      else static_cast<__nv_bfloat16*>(t.out[i])[k] = __float2bfloat16_rn(v);
    }
  }
}

// Fills one launch's table from the tensors first, first + 1, ...; empty tensors are left out.  Returns the
// tensor after the last one taken.  (check_tensors bounds the chunks of all tensors together below 2^31.)
int32_t fill_table(ClipTable& t, const void* const* grads, void* const* outs, const int64_t* numels,
                   const int32_t* dtypes, int32_t first, int32_t n) {
  t.n = 0;
  uint64_t chunks = 0;
  int32_t i = first;
  for (; i < n && t.n < kClipCap; ++i) {
    if (numels[i] == 0) continue;
    chunks += static_cast<uint64_t>((numels[i] + kClipChunk - 1) / kClipChunk);
    t.grad[t.n] = grads[i];
    t.out[t.n] = outs ? outs[i] : nullptr;
    t.numel[t.n] = numels[i];
    t.end[t.n] = static_cast<uint32_t>(chunks);
    t.dtype[t.n] = static_cast<uint8_t>(dtypes[i]);
    ++t.n;
  }
  return i;
}

int64_t clip_launches(int32_t n) { return (static_cast<int64_t>(n) + kClipCap - 1) / kClipCap; }

int check_tensors(const void* const* grads, void* const* outs, const int64_t* numels, const int32_t* dtypes,
                  int32_t n) {
  if (n < 0 || n > kClipMaxTensors || (n > 0 && (!grads || !numels || !dtypes))) return FP8G_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numels[i] < 0 || numels[i] > kClipMaxValues || (dtypes[i] != FP8G_BF16 && dtypes[i] != FP8G_F32))
      return FP8G_ERR_INVALID_ARG;
    total += numels[i];
    if (total > kClipMaxValues) return FP8G_ERR_INVALID_ARG;
    if (numels[i] == 0) continue;
    const uintptr_t size = dtypes[i] == FP8G_F32 ? 4 : 2;
    if (!grads[i] || (outs && !outs[i])) return FP8G_ERR_INVALID_ARG;
    if (!aligned_to(grads[i], size) || (outs && !aligned_to(outs[i], size))) return FP8G_ERR_ALIGNMENT;
  }
  return FP8G_OK;
}

// Partial sums of all the tensors; *P is how many were written.
int norm_parts_launch(const void* const* grads, const int64_t* numels, const int32_t* dtypes, int32_t n,
                      float* parts, int32_t* P, cudaStream_t s) {
  *P = 0;
  ClipTable t;
  for (int32_t i = 0; i < n;) {
    i = fill_table(t, grads, nullptr, numels, dtypes, i, n);
    if (t.n == 0) continue;
    const uint32_t ctas = std::min<uint32_t>(t.end[t.n - 1], kClipMaxCtas);
    grad_norm_part_kernel<<<ctas, kClipThreads, 0, s>>>(t, parts + *P);
    *P += static_cast<int32_t>(ctas);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_grad_norm_workspace(int32_t n, int64_t* bytes) {
  if (n < 0 || n > kClipMaxTensors || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = std::max<int64_t>(1, clip_launches(n)) * kClipMaxCtas * 4;
  return FP8G_OK;
}

extern "C" int fp8g_grad_norm(const void* const* grads, const int64_t* numels, const int32_t* dtypes, int32_t n,
                              float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_tensors(grads, nullptr, numels, dtypes, n);
  if (st != FP8G_OK) return st;
  if (!norm || !workspace || workspace_bytes < std::max<int64_t>(1, clip_launches(n)) * kClipMaxCtas * 4)
    return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(norm, 4) || !aligned16(workspace)) return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8G_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* parts = static_cast<float*>(workspace);
  int32_t P = 0;
  st = norm_parts_launch(grads, numels, dtypes, n, parts, &P, s);
  if (st != FP8G_OK) return st;
  grad_norm_join_kernel<<<1, kClipThreads, 0, s>>>(parts, P, norm);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

extern "C" int fp8g_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels,
                                   const int32_t* dtypes, int32_t n, float max_norm, float eps, float* norm,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_tensors(grads, outs, numels, dtypes, n);
  if (st != FP8G_OK) return st;
  if ((n > 0 && !outs) || !(max_norm >= 0.0f) || !(eps >= 0.0f) || !norm || !workspace ||
      workspace_bytes < std::max<int64_t>(1, clip_launches(n)) * kClipMaxCtas * 4)
    return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(norm, 4) || !aligned16(workspace)) return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8G_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* parts = static_cast<float*>(workspace);
  int32_t P = 0;
  st = norm_parts_launch(grads, numels, dtypes, n, parts, &P, s);
  if (st != FP8G_OK) return st;
  if (P == 0) {  // no values at all
    grad_norm_join_kernel<<<1, kClipThreads, 0, s>>>(parts, 0, norm);
    return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
  }
  ClipTable t;
  for (int32_t i = 0; i < n;) {
    i = fill_table(t, grads, outs, numels, dtypes, i, n);
    if (t.n == 0) continue;
    const uint32_t ctas = std::min<uint32_t>(t.end[t.n - 1], kClipMaxCtas);
    grad_clip_kernel<<<ctas, kClipThreads, 0, s>>>(t, parts, P, max_norm, eps, norm);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}
