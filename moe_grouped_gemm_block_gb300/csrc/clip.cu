// clip.cu -- the global norm of many gradient tensors, and clipping by it.
//
//     norm = sqrt(sum over all tensors of g^2),   out = g min(1, max_norm / (norm + eps))
//
// Two passes over the data, both bound by memory: one reads everything and leaves a partial sum per CTA, the
// other sums those (each CTA all of them, in the same order), reads everything again and writes it scaled.  The
// tensors' addresses, sizes and types travel as kernel arguments (up to kClipCap tensors a launch), so nothing is
// copied to the device and a call can be captured into a graph.
//
// Every tensor is cut into chunks of U 16-byte groups a thread on the 16-byte grid of its addresses, whatever its own
// alignment: only a tensor's first and last group can be partial, and those are taken value by value.  U = 16 keeps
// more loads in flight, U = 4 gives fewer megabytes to more CTAs (small_chunks).
//
// 470 MB of bf16 gradients: 220 us.  The first pass reads at the copy rate, the second moves 800 MB (77 MB of its reads
// are still in L2), reads and writes mixed, at 85% of it.  Cache hints on either side and the order of the chunks
// changed nothing beyond 1%.

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipCap = 1024;       // tensors a launch; tables of 64 and 256 are there for their size (the arguments'
                                     // copies are most of a small call's host time)
constexpr int kClipMaxCtas = 608;    // partial sums a launch: 4 CTAs an SM (8 are within 1% of it, or slower)
constexpr int kClipJoinLoads = (kClipMaxCtas + kClipThreads - 1) / kClipThreads;
constexpr int32_t kClipMaxTensors = 1 << 20;
constexpr int64_t kClipMaxValues = int64_t{1} << 42;  // of all tensors together

template <int CAP>
struct ClipTable {
  const void* grad[CAP];
  void* out[CAP];
  int64_t numel[CAP];
  uint32_t end[CAP];  // chunks of the tensors up to and with this one
  uint8_t dtype[CAP];
  int32_t n;
};
static_assert(sizeof(ClipTable<kClipCap>) <= 32000, "kernel arguments hold 32764 bytes");

// The tensor that chunk c belongs to: among [lo, hi].
template <int CAP>
__device__ __forceinline__ int find_tensor(const ClipTable<CAP>& t, uint32_t c, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c < t.end[mid]) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// A chunk of tensor i: values [lo, hi) of the tensor; the value at lo + k lies k values after a 16-byte boundary
// (lo is negative in a first chunk whose tensor does not start on one).
template <typename T, int U>
struct Chunk {
  static constexpr int kGroups = kClipThreads * U;
  static constexpr int kPer = 16 / sizeof(T);  // values a group
  const T* g;
  T* o;
  int64_t lo, hi, numel;
  bool whole;
  template <int CAP>
  __device__ __forceinline__ Chunk(const ClipTable<CAP>& t, int i, uint32_t c) {
    g = static_cast<const T*>(t.grad[i]);
    o = static_cast<T*>(t.out[i]);
    numel = t.numel[i];
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T));
    lo = static_cast<int64_t>(c - (i ? t.end[i - 1] : 0u)) * (kGroups * kPer) - mis;
    hi = min(lo + kGroups * kPer, numel);
    whole = lo >= 0 && hi == lo + kGroups * kPer;
  }
};

__device__ __forceinline__ float square_sum(const uint4& v, float) {
  const float a = __uint_as_float(v.x), b = __uint_as_float(v.y), c = __uint_as_float(v.z), d = __uint_as_float(v.w);
  return (a * a + b * b) + (c * c + d * d);
}
__device__ __forceinline__ float square_sum(const uint4& v, __nv_bfloat16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
    s[0] = fmaf(a, a, s[0]);
    s[1] = fmaf(b, b, s[1]);
  }
  return s[0] + s[1];
}

// A thread's share of a chunk's sum of squares: its groups' sums, joined in a tree.
template <typename T, int U, int CAP>
__device__ __forceinline__ float chunk_square_sum(const ClipTable<CAP>& t, int i, uint32_t c) {
  const Chunk<T, U> ch(t, i, c);
  float s[U] = {};
  if (ch.whole) {
    const uint4* p = reinterpret_cast<const uint4*>(ch.g + ch.lo) + threadIdx.x;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldg(p + u * kClipThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = square_sum(v[u], T());
  } else {  // four groups at a time: the whole ones' loads together, then the partial ones (two of a tensor, at most)
#pragma unroll 1
    for (int u0 = 0; u0 < U; u0 += 4) {
      uint4 v[4];
      float e = 0.0f;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t k = ch.lo + ((u0 + u) * kClipThreads + threadIdx.x) * ch.kPer;
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (k >= 0 && k + ch.kPer <= ch.hi) {
          v[u] = __ldg(reinterpret_cast<const uint4*>(ch.g + k));
        } else {
          for (int64_t q = max(k, int64_t{0}); q < min(k + ch.kPer, ch.hi); ++q) {
            const float f = to_f32(ch.g[q]);
            e = fmaf(f, f, e);
          }
        }
      }
      s[0] += e + ((square_sum(v[0], T()) + square_sum(v[1], T())) + (square_sum(v[2], T()) + square_sum(v[3], T())));
    }
    return s[0];
  }
#pragma unroll
  for (int d = 1; d < U; d *= 2)
#pragma unroll
    for (int u = 0; u + d < U; u += 2 * d) s[u] += s[u + d];
  return s[0];
}

template <int CAP, int U>
__global__ void __launch_bounds__(kClipThreads) grad_norm_part_kernel(const __grid_constant__ ClipTable<CAP> t,
                                                                      float* __restrict__ parts) {
  __shared__ float red[2 * kClipThreads / 32];
  griddep_launch_dependents();  // the scaling pass may start (it waits for this grid's sums)
  float s[1] = {0.0f};
  const uint32_t chunks = t.end[t.n - 1];
  int i = 0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    i = c < t.end[i] ? i : find_tensor(t, c, i, t.n - 1);
    s[0] += t.dtype[i] == FP8G_F32 ? chunk_square_sum<float, U>(t, i, c)
                                    : chunk_square_sum<__nv_bfloat16, U>(t, i, c);
  }
  cta_sum<kClipThreads / 32>(s, red, 0);
  if (threadIdx.x == 0) parts[blockIdx.x] = s[0];
}

// A sum and what its roundings lost: the exact sum of two floats is their rounded sum and its error (Knuth).
struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float v, float v_lo) {
    const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)), v_lo));
    hi = s;
  }
};

// The norm from the partial sums: the same value in every CTA that calls it.  The sums are pairs of floats, not
// doubles: every CTA of the second pass takes them, and this GPU's fp64 rate made that 15 us of a 26 MB call's 30.
__device__ __forceinline__ float join_norm(const float* __restrict__ parts, int32_t P) {
  __shared__ Sum2 s_sum[kClipThreads / 32];
  float v[kClipJoinLoads];
#pragma unroll
  for (int i = 0; i < kClipJoinLoads; ++i) {
    const int k = i * kClipThreads + static_cast<int>(threadIdx.x);
    v[i] = k < P ? __ldcg(parts + k) : 0.0f;
  }
  Sum2 s{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kClipJoinLoads; ++i) s.add(v[i], 0.0f);
  for (int k = kClipJoinLoads * kClipThreads + static_cast<int>(threadIdx.x); k < P; k += kClipThreads)
    s.add(__ldcg(parts + k), 0.0f);  // (more than one launch's)
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    s.add(__shfl_xor_sync(0xffffffffu, s.hi, off), __shfl_xor_sync(0xffffffffu, s.lo, off));
  if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = s;
  __syncthreads();
  s = s_sum[0];
#pragma unroll
  for (int w = 1; w < kClipThreads / 32; ++w) s.add(s_sum[w].hi, s_sum[w].lo);
  // (an infinite sum's error is not a number)
  return sqrtf(isinf(s.hi) ? s.hi : s.hi + s.lo);
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_join_kernel(const float* __restrict__ parts, int32_t P,
                                                                      float* __restrict__ norm) {
  const float n = join_norm(parts, P);
  if (threadIdx.x == 0) *norm = n;
}

__device__ __forceinline__ uint4 scaled(const uint4& v, float c, float) {
  return make_uint4(__float_as_uint(__uint_as_float(v.x) * c), __float_as_uint(__uint_as_float(v.y) * c),
                    __float_as_uint(__uint_as_float(v.z) * c), __float_as_uint(__uint_as_float(v.w) * c));
}
__device__ __forceinline__ uint32_t scaled2(uint32_t w, float c) {
  return pack2(__uint_as_float(w << 16) * c, __uint_as_float(w & 0xFFFF0000u) * c);
}
__device__ __forceinline__ uint4 scaled(const uint4& v, float c, __nv_bfloat16) {
  return make_uint4(scaled2(v.x, c), scaled2(v.y, c), scaled2(v.z, c), scaled2(v.w, c));
}

template <typename T, int U, int CAP>
__device__ __forceinline__ void chunk_scale(const ClipTable<CAP>& t, int i, uint32_t c, float coef) {
  const Chunk<T, U> ch(t, i, c);
  // 16-byte stores where the result's groups lie on its own 16-byte grid too
  const bool same = ((reinterpret_cast<uintptr_t>(ch.g) ^ reinterpret_cast<uintptr_t>(ch.o)) & 15u) == 0;
  if (ch.whole && same) {
    const uint4* p = reinterpret_cast<const uint4*>(ch.g + ch.lo) + threadIdx.x;
    uint4* q = reinterpret_cast<uint4*>(ch.o + ch.lo) + threadIdx.x;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldcs(p + u * kClipThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) __stcs(q + u * kClipThreads, scaled(v[u], coef, T()));
    return;
  }
#pragma unroll 1
  for (int u0 = 0; u0 < U; u0 += 4) {  // as in the sum; without a common grid value by value
    uint4 v[4];
    bool full[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t k = ch.lo + ((u0 + u) * kClipThreads + threadIdx.x) * ch.kPer;
      full[u] = same && k >= 0 && k + ch.kPer <= ch.hi;
      if (full[u]) v[u] = __ldcs(reinterpret_cast<const uint4*>(ch.g + k));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t k = ch.lo + ((u0 + u) * kClipThreads + threadIdx.x) * ch.kPer;
      if (full[u]) {
        *reinterpret_cast<uint4*>(ch.o + k) = scaled(v[u], coef, T());
      } else {
        for (int64_t q = max(k, int64_t{0}); q < min(k + ch.kPer, ch.hi); ++q)
          ch.o[q] = from_f32<T>(to_f32(ch.g[q]) * coef);
      }
    }
  }
}

// The chunks in descending order: the first pass ended with the last ones, so some of them are still in L2.
template <int CAP, int U>
__global__ void __launch_bounds__(kClipThreads) grad_clip_kernel(const __grid_constant__ ClipTable<CAP> t,
                                                                 const float* __restrict__ parts, int32_t P,
                                                                 float max_norm, float eps,
                                                                 float* __restrict__ norm) {
  griddep_wait();
  const float n = join_norm(parts, P);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  const float coef = n + eps <= max_norm ? 1.0f : max_norm / (n + eps);  // a NaN norm makes every output NaN
  const uint32_t chunks = t.end[t.n - 1];
  int i = t.n - 1;
  for (uint32_t b = blockIdx.x; b < chunks; b += gridDim.x) {
    const uint32_t c = chunks - 1 - b;
    i = i == 0 || c >= t.end[i - 1] ? i : find_tensor(t, c, 0, i);
    if (coef == 1.0f && t.out[i] == t.grad[i]) continue;  // in place and nothing to scale
    if (t.dtype[i] == FP8G_F32) chunk_scale<float, U>(t, i, c, coef);
    else chunk_scale<__nv_bfloat16, U>(t, i, c, coef);
  }
}

// Fills one launch's table from the tensors first, first + 1, ...; empty tensors are left out.  Returns the
// tensor after the last one taken.  (check_tensors bounds the chunks of all tensors together below 2^31.)
template <int CAP, int U>
int32_t fill_table(ClipTable<CAP>& t, const void* const* grads, void* const* outs, const int64_t* numels,
                   const int32_t* dtypes, int32_t first, int32_t n) {
  t.n = 0;
  uint64_t chunks = 0;
  int32_t i = first;
  for (; i < n && t.n < CAP; ++i) {
    if (numels[i] == 0) continue;
    const int64_t size = dtypes[i] == FP8G_F32 ? 4 : 2, per = static_cast<int64_t>(kClipThreads) * U * (16 / size);
    const int64_t mis = static_cast<int64_t>(reinterpret_cast<uintptr_t>(grads[i]) & 15u) / size;
    chunks += static_cast<uint64_t>((numels[i] + mis + per - 1) / per);
    t.grad[t.n] = grads[i];
    t.out[t.n] = outs ? outs[i] : nullptr;
    t.numel[t.n] = numels[i];
    t.end[t.n] = static_cast<uint32_t>(chunks);
    t.dtype[t.n] = static_cast<uint8_t>(dtypes[i]);
    ++t.n;
  }
  return i;
}

// Whether the chunks are the 16 KB ones (U = 4): up to 256 MB.  17 MB of odd tensors took 14.5 us with them and 19 with
// 64 KB chunks, 36 MB of bf16 21 and 23, 470 MB 230 and 220.
bool small_chunks(const int64_t* numels, const int32_t* dtypes, int32_t n) {
  int64_t bytes = 0;
  for (int32_t i = 0; i < n; ++i) bytes += numels[i] * (dtypes[i] == FP8G_F32 ? 4 : 2);
  return bytes <= int64_t{256} << 20;
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
template <int CAP, int U>
int norm_parts_launch(ClipTable<CAP>& t, const void* const* grads, void* const* outs, const int64_t* numels,
                      const int32_t* dtypes, int32_t n, float* parts, int32_t* P, cudaStream_t s) {
  *P = 0;
  for (int32_t i = 0; i < n;) {
    i = fill_table<CAP, U>(t, grads, outs, numels, dtypes, i, n);
    if (t.n == 0) continue;
    const uint32_t ctas = std::min<uint32_t>(t.end[t.n - 1], kClipMaxCtas);
    grad_norm_part_kernel<CAP, U><<<ctas, kClipThreads, 0, s>>>(t, parts + *P);
    *P += static_cast<int32_t>(ctas);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

template <int CAP, int U>
int grad_norm_launch(const void* const* grads, const int64_t* numels, const int32_t* dtypes, int32_t n, float* norm,
                     float* parts, cudaStream_t s) {
  ClipTable<CAP> t;
  int32_t P = 0;
  const int st = norm_parts_launch<CAP, U>(t, grads, nullptr, numels, dtypes, n, parts, &P, s);
  if (st != FP8G_OK) return st;
  grad_norm_join_kernel<<<1, kClipThreads, 0, s>>>(parts, P, norm);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

template <int CAP, int U>
int clip_launch(const void* const* grads, void* const* outs, const int64_t* numels, const int32_t* dtypes, int32_t n,
                float max_norm, float eps, float* norm, float* parts, cudaStream_t s) {
  ClipTable<CAP> t;
  int32_t P = 0;
  const int st = norm_parts_launch<CAP, U>(t, grads, outs, numels, dtypes, n, parts, &P, s);
  if (st != FP8G_OK) return st;
  if (P == 0) {  // no values at all
    grad_norm_join_kernel<<<1, kClipThreads, 0, s>>>(parts, 0, norm);
    return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
  }
  const bool one = n <= CAP;  // then the table is already the whole one
  for (int32_t i = 0; i < n;) {
    i = one ? n : fill_table<CAP, U>(t, grads, outs, numels, dtypes, i, n);
    if (t.n == 0) continue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(std::min<uint32_t>(t.end[t.n - 1], kClipMaxCtas));
    cfg.blockDim = dim3(kClipThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = one ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, grad_clip_kernel<CAP, U>, t, static_cast<const float*>(parts), P, max_norm, eps,
                           norm) != cudaSuccess) {
      cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
  }
  return FP8G_OK;
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
  const bool small = small_chunks(numels, dtypes, n);
  auto go = n <= 64    ? (small ? grad_norm_launch<64, 4> : grad_norm_launch<64, 16>)
            : n <= 256 ? (small ? grad_norm_launch<256, 4> : grad_norm_launch<256, 16>)
                       : (small ? grad_norm_launch<kClipCap, 4> : grad_norm_launch<kClipCap, 16>);
  return go(grads, numels, dtypes, n, norm, static_cast<float*>(workspace), static_cast<cudaStream_t>(stream));
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
  const bool small = small_chunks(numels, dtypes, n);
  auto go = n <= 64    ? (small ? clip_launch<64, 4> : clip_launch<64, 16>)
            : n <= 256 ? (small ? clip_launch<256, 4> : clip_launch<256, 16>)
                       : (small ? clip_launch<kClipCap, 4> : clip_launch<kClipCap, 16>);
  return go(grads, outs, numels, dtypes, n, max_norm, eps, norm, static_cast<float*>(workspace),
            static_cast<cudaStream_t>(stream));
}
