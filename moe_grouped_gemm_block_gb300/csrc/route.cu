// route.cu -- the router with sigmoid or softmax scores, a bias for balance and expert groups, and its gradient.
//
//     s_t = sigmoid(l_t) or softmax(l_t);  c_t = s_t + bias (the choice alone);  the experts lie in G equal groups, whose
//     score is the sum of the two largest c in them; the topk_groups best groups stay, and of their experts the topk
//     largest c are taken.  w_t = scale s_t[ids], over their sum where renormalised.
//   backward (the choice held fixed): the gradient of w through the division and the scores; the bias has none.
//
// The choice is that of scores in 64 bits, whatever the kernel's form: two scores that fp32 cannot tell apart are.

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kRouteMaxExperts = 2048;
constexpr int kRouteMaxTopk = 32;
constexpr int kRouteMaxGroups = 32;
constexpr int kRouteWarps = 4;

struct RouteArgs {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  int32_t* counts;
  const float* dweights;
  void* dlogits;
  int64_t T, ldl, ldd;
  int32_t E, topk, groups, kept, softmax, renorm, vec;
  float scale;
};

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One row by a warp, in 64 bits.  `c`: E doubles of the warp's own.  A place that holds NaN is not to be had (a score
// that is not a number ranks first: it stands as infinity).
template <typename TL>
__device__ __noinline__ void route_row(const RouteArgs& a, int64_t t, double* c, int& pick, float& weight) {
  const int lane = threadIdx.x & 31, E = a.E, per = E / a.groups;
  const TL* row = static_cast<const TL*>(a.logits) + t * a.ldl;
  const double nan = __longlong_as_double(0x7FF8000000000000LL), inf = INFINITY;
  double mx = 0.0, inv = 1.0;
  if (a.softmax) {
    mx = -inf;
    for (int e = lane; e < E; e += 32) mx = fmax(mx, static_cast<double>(to_f32(row[e])));
    mx = warp_max(mx);
    if (mx == -inf) mx = 0.0;
    double s = 0.0;
    for (int e = lane; e < E; e += 32) s += exp(static_cast<double>(to_f32(row[e])) - mx);
    s = warp_sum(s);
    inv = s == 0.0 ? 0.0 : 1.0 / s;
  }
  auto score = [&](double l) { return a.softmax ? exp(l - mx) * inv : 1.0 / (1.0 + exp(-l)); };
  for (int e = lane; e < E; e += 32) {
    const double l = to_f32(row[e]), b = a.bias ? static_cast<double>(a.bias[e]) : 0.0;
    const double v = l == -inf || b == -inf ? -inf : score(l) + b;
    c[e] = v == v ? v : inf;
  }
  __syncwarp();
  uint32_t open = 0xffffffffu;
  if (a.groups > 1) {
    double first = -inf, second = -inf;
    if (lane < a.groups)
      for (int i = 0; i < per; ++i) {
        const double v = c[lane * per + i];
        if (v > first) second = first, first = v;
        else if (v > second) second = v;
      }
    const double mine = second == -inf ? first : first + second;
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double other = __shfl_sync(0xffffffffu, mine, g);
      better += other > mine || (other == mine && g < lane) ? 1 : 0;
    }
    open = __ballot_sync(0xffffffffu, lane < a.groups && better < a.kept);
  }
  for (int e = lane; e < E; e += 32) {
    double v = c[e];
    if (!a.bias && v != -inf) {  // the scores order as the logits do
      v = to_f32(row[e]);
      v = v == v ? v : inf;
    }
    c[e] = open >> (e / per) & 1u ? v : nan;
  }
  pick = 0;
  for (int j = 0; j < a.topk; ++j) {
    double best = nan;
    int at = kRouteMaxExperts;
    for (int e = lane; e < E; e += 32)
      if (c[e] > best || (best != best && c[e] == c[e])) best = c[e], at = e;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double v = __shfl_xor_sync(0xffffffffu, best, off);
      const int i = __shfl_xor_sync(0xffffffffu, at, off);
      if (v > best || (v == best && i < at) || (best != best && v == v)) best = v, at = i;
    }
    if (lane == j) pick = at;
    if ((at & 31) == lane) c[at] = nan;
    __syncwarp();
  }
  weight = 0.0f;
  if (lane < a.topk) {
    const double l = to_f32(row[pick]);
    weight = l == -inf || (a.bias && a.bias[pick] == -INFINITY) ? 0.0f : static_cast<float>(score(l));
  }
  __syncwarp();
}

template <typename TL>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_kernel(const RouteArgs a) {
  extern __shared__ double choice[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp; t < a.T; t += gridDim.x * kRouteWarps) {
    int id;
    float w;
    route_row<TL>(a, t, choice + warp * a.E, id, w);
    const bool real = !a.mask || a.mask[t];
    const float sum = warp_sum(w);
    if (a.renorm) w = sum == 0.0f ? 0.0f : __fdiv_rn(w, sum);
    if (lane < a.topk) {
      a.ids[t * a.topk + lane] = id;
      a.weights[t * a.topk + lane] = real ? w * a.scale : 0.0f;
      if (real) atomicAdd(a.counts + id, 1);  // whole numbers: the order does not matter
    }
  }
}

// A warp a row; lane j < topk has the row's j-th choice.
template <typename TL>
__global__ void __launch_bounds__(256) moe_route_backward_kernel(const RouteArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp; t < a.T; t += gridDim.x * 8) {
    const TL* row = static_cast<const TL*>(a.logits) + t * a.ldl;
    TL* out = static_cast<TL*>(a.dlogits) + t * a.ldd;
    const bool real = !a.mask || a.mask[t];
    int id = -1;
    float d = 0.0f, l = -INFINITY;
    if (lane < a.topk) {
      id = a.ids[t * a.topk + lane];
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        d = a.dweights[t * a.topk + lane] * a.scale;
        l = to_f32(row[id]);
      }
    }
    float mx = 0.0f, inv = 1.0f, s, slope = 0.0f;
    if (a.softmax) {
      mx = -INFINITY;
      for (int e = lane; e < E; e += 32) mx = fmaxf(mx, to_f32(row[e]));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      if (mx == -INFINITY) mx = 0.0f;
      float sum = 0.0f;
      for (int e = lane; e < E; e += 32) sum += expf(to_f32(row[e]) - mx);
      sum = warp_sum(sum);
      inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      s = expf(l - mx) * inv;
    } else {
      const float x = expf(-fabsf(l)), r = __fdiv_rn(1.0f, 1.0f + x);
      s = l >= 0.0f ? r : x * r;
      slope = x * r * r;  // s (1 - s)
    }
    if (id < 0) s = 0.0f;
    if (a.renorm) {
      const float sum = warp_sum(s), inner = warp_sum(d * s);
      const float by = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      d = (d - inner * by) * by;
    }
    if (id < 0) d = 0.0f;
    const float q = a.softmax ? warp_sum(d * s) : 0.0f;
    // the same expert twice gets the sum of both
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    if (__any_sync(0xffffffffu, id >= 0 && __popc(same) > 1)) {
      float all = 0.0f;
      for (int j = 0; j < 32; ++j) {
        const float v = __shfl_sync(0xffffffffu, d, j);
        if (same >> j & 1u) all += v;
      }
      d = all;
    }
    for (int e = lane; e < E; e += 32) {
      const float v = a.softmax && real ? -q * (expf(to_f32(row[e]) - mx) * inv) : 0.0f;
      out[e] = from_f32<TL>(v);
    }
    __syncwarp();
    if (id >= 0 && real) out[id] = from_f32<TL>(a.softmax ? s * (d - q) : d * slope);
    __syncwarp();
  }
}

int check_route(int32_t dtype, int64_t T, int32_t E, int64_t ldl, int32_t topk, int32_t score, int32_t renorm) {
  if ((dtype != FP8G_BF16 && dtype != FP8G_F32) || T < 0 || T > 0x7FFFFFFF || E < 1 || E > kRouteMaxExperts || ldl < E ||
      topk < 1 || topk > std::min(E, kRouteMaxTopk) || T * topk > 0x7FFFFFFF || (score & ~1) || (renorm & ~1))
    return FP8G_ERR_INVALID_ARG;
  return FP8G_OK;
}

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_moe_route(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ldl, int32_t topk,
                              const float* bias, int32_t score, int32_t groups, int32_t topk_groups, int32_t renormalize,
                              float scale, const uint8_t* token_mask, int32_t* topk_ids, float* topk_weights,
                              int32_t* counts, void* stream) {
  int st = check_route(dtype, T, E, ldl, topk, score, renormalize);
  if (st != FP8G_OK) return st;
  if (groups < 1 || groups > kRouteMaxGroups || E % groups != 0 || topk_groups < 1 || topk_groups > groups ||
      static_cast<int64_t>(topk_groups) * (E / groups) < topk || !counts || scale != scale)
    return FP8G_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !topk_ids || !topk_weights)) return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(logits, dtype == FP8G_F32 ? 4 : 2) || !aligned_to(bias, 4) || !aligned_to(topk_ids, 4) ||
      !aligned_to(topk_weights, 4) || !aligned_to(counts, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8G_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(counts, 0, static_cast<size_t>(E) * 4, s) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  if (T == 0) return FP8G_OK;
  RouteArgs a{};
  a.logits = logits, a.bias = bias, a.mask = token_mask, a.ids = topk_ids, a.weights = topk_weights, a.counts = counts;
  a.T = T, a.ldl = ldl, a.E = E, a.topk = topk, a.groups = groups, a.kept = topk_groups, a.softmax = score;
  a.renorm = renormalize, a.scale = scale;
  const size_t smem = sizeof(double) * kRouteWarps * static_cast<size_t>(E);
  auto kernel = dtype == FP8G_F32 ? moe_route_kernel<float> : moe_route_kernel<__nv_bfloat16>;
  st = allow_shared_memory(reinterpret_cast<const void*>(kernel), smem);
  if (st != FP8G_OK) return st;
  const unsigned ctas = static_cast<unsigned>(std::min<int64_t>((T + kRouteWarps - 1) / kRouteWarps, 8 * dev->sm_count));
  kernel<<<ctas, 32 * kRouteWarps, smem, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

extern "C" int fp8g_moe_route_backward(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ldl, int32_t topk,
                                       int32_t score, int32_t renormalize, float scale, const uint8_t* token_mask,
                                       const int32_t* topk_ids, const float* dweights, void* dlogits, int64_t ldd,
                                       void* stream) {
  int st = check_route(dtype, T, E, ldl, topk, score, renormalize);
  if (st != FP8G_OK) return st;
  if (ldd < E || scale != scale) return FP8G_ERR_INVALID_ARG;
  if (T == 0) return FP8G_OK;
  if (!logits || !topk_ids || !dweights || !dlogits) return FP8G_ERR_INVALID_ARG;
  const uintptr_t size = dtype == FP8G_F32 ? 4 : 2;
  if (!aligned_to(logits, size) || !aligned_to(dlogits, size) || !aligned_to(topk_ids, 4) || !aligned_to(dweights, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  st = current_device(&dev);
  if (st != FP8G_OK) return st;
  RouteArgs a{};
  a.logits = logits, a.mask = token_mask, a.ids = const_cast<int32_t*>(topk_ids), a.dweights = dweights;
  a.dlogits = dlogits, a.T = T, a.ldl = ldl, a.ldd = ldd, a.E = E, a.topk = topk, a.softmax = score;
  a.renorm = renormalize, a.scale = scale;
  auto kernel = dtype == FP8G_F32 ? moe_route_backward_kernel<float> : moe_route_backward_kernel<__nv_bfloat16>;
  const unsigned ctas = static_cast<unsigned>(std::min<int64_t>((T + 7) / 8, 8 * dev->sm_count));
  kernel<<<ctas, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}
