// moe.cu -- the two ends of a MoE block around its grouped GEMMs: the gate (softmax, top-k, per-expert
// counts and the balance loss, with their gradient) and the combine (the experts' rows back to their tokens, with
// its gradient).

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

// ---------------------------------------------------------------- gate
//     p_t = softmax(l_t),  ids_t = the k largest logits (ties: the lowest index),  w_t = p_t[ids_t], over their sum
//     where renormalised;  c_e = how many unmasked (t, j) chose e;  Tv = the unmasked tokens
//     loss = coef E sum_e f_e P_e,   f_e = c_e / (k Tv),   P_e = (1 / Tv) sum over the unmasked t of p_te
constexpr int kGateThreads = 256;
constexpr int kGateWarps = kGateThreads / 32;
constexpr int kGateMaxExperts = 2048;  // the routed layout's limit
constexpr int kGateMaxTopk = 32;       // a selected expert per lane
constexpr int kGateMaxCtas = 304;      // partial sums

// The order of the selection as an unsigned integer: ascending in the value, NaN above everything (as a
// descending sort has it), -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// One warp a row; a warp's rows, and so each partial sum's terms and their order, follow from the grid alone.
// Shared memory: per warp the row's logits [E], and per CTA its sums of p [WARPS][E] and its counts [E].
template <typename TL>
__global__ void __launch_bounds__(kGateThreads) moe_gate_kernel(
    const TL* __restrict__ logits, int64_t T, int32_t E, int64_t ldl, int32_t topk, int32_t renorm,
    const uint8_t* __restrict__ mask, int32_t* __restrict__ ids, float* __restrict__ weights,
    float* __restrict__ part_p, int32_t* __restrict__ part_c) {
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row = smem + warp * E;
  float* sum_p = smem + kGateWarps * E + warp * E;
  int32_t* cnt = reinterpret_cast<int32_t*>(smem + 2 * kGateWarps * E);
  for (int e = lane; e < E; e += 32) sum_p[e] = 0.0f;
  for (int e = threadIdx.x; e < E; e += kGateThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp; t < T; t += stride) {
    float mx = -INFINITY;
    for (int e = lane; e < E; e += 32) {
      const float v = to_f32(logits[t * ldl + e]);
      row[e] = v;
      mx = fmaxf(mx, v);
    }
    mx = warp_max(mx);
    float s = 0.0f;
    if (mx == -INFINITY) mx = 0.0f;  // every expert masked: exp gives 0 for all of them (NaN stays NaN)
    for (int e = lane; e < E; e += 32) s += expf(row[e] - mx);
    s = warp_sum(s);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    const bool real = !mask || mask[t];
    if (real)
      for (int e = lane; e < E; e += 32) sum_p[e] += expf(row[e] - mx) * inv;
    // k rounds: the largest key that is left, the lowest index of equal ones.  A taken expert is marked by
    // its lane (bit i = expert lane + 32 i).
    uint64_t taken = 0;
    float my_v = 0.0f;
    int my_id = 0;
    for (int j = 0; j < topk; ++j) {
      uint32_t best = 0;
      int at = E;
      for (int e = lane, i = 0; e < E; e += 32, ++i) {
        const uint32_t key = order_key(row[e]);
        if (!(taken >> i & 1) && (at == E || key > best)) {
          best = key;
          at = e;
        }
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, at < E ? best : 0u);
      const int e = __reduce_min_sync(0xffffffffu, at < E && best == top ? at : E);
      if ((e & 31) == lane) taken |= uint64_t{1} << (e >> 5);
      if (lane == j) {
        my_id = e;
        my_v = row[e];
      }
    }
    float w = lane < topk ? expf(my_v - mx) : 0.0f;
    const float total = warp_sum(w);
    w *= renorm ? (total == 0.0f ? 0.0f : 1.0f / total) : inv;
    if (lane < topk) {
      ids[t * topk + lane] = my_id;
      weights[t * topk + lane] = real ? w : 0.0f;
      if (real) atomicAdd(cnt + my_id, 1);  // whole numbers: the order does not matter
    }
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kGateThreads) {
    float s = 0.0f;
    for (int w = 0; w < kGateWarps; ++w) s += smem[kGateWarps * E + w * E + e];
    part_p[static_cast<int64_t>(blockIdx.x) * E + e] = s;
    part_c[static_cast<int64_t>(blockIdx.x) * E + e] = cnt[e];
  }
}

// Counts and loss from the CTAs' partial sums, in their order.
__global__ void __launch_bounds__(kGateThreads) moe_gate_join_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int32_t P, int32_t E, int32_t topk,
    float coef, int32_t* __restrict__ counts, float* __restrict__ loss) {
  __shared__ float red[2 * 2 * kGateWarps];
  float v[2] = {0.0f, 0.0f};  // sum_e c_e P_e, sum_e c_e
  for (int e = threadIdx.x; e < E; e += kGateThreads) {
    float p = 0.0f;
    int32_t c = 0;
    for (int i = 0; i < P; ++i) {
      p += part_p[static_cast<int64_t>(i) * E + e];
      c += part_c[static_cast<int64_t>(i) * E + e];
    }
    counts[e] = c;
    v[0] += static_cast<float>(c) * p;
    v[1] += static_cast<float>(c);
  }
  cta_sum<kGateWarps>(v, red, 0);
  if (threadIdx.x == 0 && loss) {
    const float tv = v[1] / static_cast<float>(topk);
    *loss = tv > 0.0f ? coef * static_cast<float>(E) * (v[0] / (static_cast<float>(topk) * tv * tv)) : 0.0f;
  }
}

// dl_te = p_te (G_te - sum_e G_te p_te),  G_te = g_e + sum_j [ids_tj = e] dp_tj,
// g_e = dloss coef E c_e / (k Tv^2),  dp_tj = dw_tj, or (dw_tj - sum_i dw_ti w_ti) / S_t where renormalised
// (S_t = the selected probabilities' sum).  Masked tokens get zeros.  One warp a row.
template <typename TL>
__global__ void __launch_bounds__(kGateThreads) moe_gate_backward_kernel(
    const TL* logits, int64_t T, int32_t E, int64_t ldl, int32_t topk, int32_t renorm,
    const uint8_t* __restrict__ mask, float coef, const int32_t* __restrict__ ids,
    const int32_t* __restrict__ counts, const float* __restrict__ dweights, const float* __restrict__ dloss,
    TL* dlogits, int64_t ldd) {
  extern __shared__ float smem[];
  __shared__ float red[2 * kGateWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* g = smem;
  float* row = smem + E + warp * E;
  float n[1] = {0.0f};
  for (int e = threadIdx.x; e < E; e += kGateThreads) n[0] += static_cast<float>(counts[e]);
  cta_sum<kGateWarps>(n, red, 0);
  const float tv = n[0] / static_cast<float>(topk);
  const float scale =
      dloss && tv > 0.0f ? *dloss * coef * static_cast<float>(E) / (static_cast<float>(topk) * tv * tv) : 0.0f;
  for (int e = threadIdx.x; e < E; e += kGateThreads) g[e] = scale * static_cast<float>(counts[e]);
  __syncthreads();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + warp; t < T; t += stride) {
    if (mask && !mask[t]) {
      for (int e = lane; e < E; e += 32) dlogits[t * ldd + e] = from_f32<TL>(0.0f);
      continue;
    }
    float mx = -INFINITY;
    for (int e = lane; e < E; e += 32) {
      const float v = to_f32(logits[t * ldl + e]);
      row[e] = v;
      mx = fmaxf(mx, v);
    }
    mx = warp_max(mx);
    if (mx == -INFINITY) mx = 0.0f;
    float s = 0.0f;
    for (int e = lane; e < E; e += 32) {
      const float v = expf(row[e] - mx);
      row[e] = v;
      s += v;
    }
    s = warp_sum(s);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    float inner = 0.0f;
    for (int e = lane; e < E; e += 32) {
      row[e] *= inv;
      inner += g[e] * row[e];
    }
    __syncwarp();
    int id = -1;
    float p = 0.0f, dp = 0.0f;
    if (dweights && lane < topk) {
      id = ids[t * topk + lane];
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        p = row[id];
        dp = dweights[t * topk + lane];
      }
    }
    if (renorm) {
      const float total = warp_sum(p);
      const float it = total == 0.0f ? 0.0f : 1.0f / total;
      dp = (dp - warp_sum(dp * p) * it) * it;
    }
    inner = warp_sum(inner + dp * p);
    __syncwarp();
    for (int e = lane; e < E; e += 32) row[e] *= g[e] - inner;
    __syncwarp();
    if (id >= 0) atomicAdd(row + id, p * dp);  // a gate's ids differ: one term an expert
    __syncwarp();
    for (int e = lane; e < E; e += 32) dlogits[t * ldd + e] = from_f32<TL>(row[e]);
    __syncwarp();
  }
}

// ---------------------------------------------------------------- combine
//     out_t = residual_t + sum_j w_tj D[row_tj]
constexpr int kCombineThreads = 128;

// The row of an entry, or -1 where it is dropped or out of range (the latter is flagged).
__device__ __forceinline__ int32_t entry(const int32_t* __restrict__ entry_row, int64_t i, int64_t M,
                                         unsigned int* status) {
  const int32_t r = entry_row[i];
  if (r >= M) {
    record_status(status, FP8G_ERR_DEVICE_ASSERT);
    return -1;
  }
  return r;
}

template <typename TO>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(
    const __nv_bfloat16* __restrict__ D, int64_t M, int64_t N, int64_t ldd, const int32_t* __restrict__ entry_row,
    int32_t topk, const float* __restrict__ weights, const TO* residual, int64_t ldr,
    TO* out, int64_t ldo, unsigned int* status) {
  const int64_t t = blockIdx.x;
  for (int64_t n = threadIdx.x * 8; n < N; n += kCombineThreads * 8) {
    float acc[8] = {};
    if (residual) load8(residual + t * ldr + n, acc);
    for (int j = 0; j < topk; ++j) {
      const int32_t r = entry(entry_row, t * topk + j, M, status);
      if (r < 0) continue;
      const float w = weights ? weights[t * topk + j] : 1.0f;
      float f[8];
      load8(D + r * ldd + n, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += w * f[i];
    }
    store8(out + t * ldo + n, acc);
  }
}

// dD[row_tj] = w_tj dout_t,  dw_tj = <dout_t, D[row_tj]>; rows without a token are zero.  One CTA a token;
// the rows' zeros are written by the CTAs in turn.
template <typename TO>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_backward_kernel(
    const TO* __restrict__ dout, int64_t lddo, const __nv_bfloat16* __restrict__ D, int64_t M, int64_t N, int64_t ldd,
    const int32_t* __restrict__ entry_row, const int32_t* __restrict__ row_token, int64_t T, int32_t topk,
    const float* __restrict__ weights, __nv_bfloat16* __restrict__ dD, int64_t lddd, float* __restrict__ dweights,
    unsigned int* status) {
  __shared__ float red[2 * kCombineThreads / 32];
  int phase = 0;
  const int64_t t = blockIdx.x;
  if (t < T) {
    for (int j = 0; j < topk; ++j) {
      const int32_t r = entry(entry_row, t * topk + j, M, status);
      float dot[1] = {0.0f};
      if (r >= 0) {
        const float w = weights ? weights[t * topk + j] : 1.0f;
        for (int64_t n = threadIdx.x * 8; n < N; n += kCombineThreads * 8) {
          float f[8], g[8];
          load8(dout + t * lddo + n, g);
          if (dweights) {
            load8(D + r * ldd + n, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[0] += f[i] * g[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] *= w;
          store8(dD + r * lddd + n, g);
        }
      }
      if (dweights) {
        cta_sum<kCombineThreads / 32>(dot, red, phase++);
        if (threadIdx.x == 0) dweights[t * topk + j] = dot[0];
      }
    }
  }
  const float zero[8] = {};
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x)
    if (row_token[r] < 0)
      for (int64_t n = threadIdx.x * 8; n < N; n += kCombineThreads * 8) store8(dD + r * lddd + n, zero);
}

int64_t gate_ctas(int64_t T) {
  return std::min<int64_t>((T + kGateWarps - 1) / kGateWarps, kGateMaxCtas);
}
bool dtype_ok(int32_t d) { return d == FP8G_BF16 || d == FP8G_F32; }
uintptr_t dtype_size(int32_t d) { return d == FP8G_F32 ? 4 : 2; }

template <typename Kernel>
int allow_smem(Kernel kern, size_t bytes) {
  if (bytes <= 48 * 1024) return FP8G_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

template <typename TL>
int gate_launch(const void* logits, int64_t T, int32_t E, int64_t ldl, int32_t topk, int32_t renorm,
                const uint8_t* mask, float coef, int32_t* ids, float* weights, int32_t* counts, float* loss,
                void* workspace, cudaStream_t s) {
  const int64_t P = gate_ctas(T);
  float* part_p = static_cast<float*>(workspace);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + P * E);
  const size_t smem = static_cast<size_t>(2 * kGateWarps + 1) * E * 4;
  int st = allow_smem(moe_gate_kernel<TL>, smem);
  if (st != FP8G_OK) return st;
  moe_gate_kernel<TL><<<static_cast<unsigned>(P), kGateThreads, smem, s>>>(
      static_cast<const TL*>(logits), T, E, ldl, topk, renorm, mask, ids, weights, part_p, part_c);
  moe_gate_join_kernel<<<1, kGateThreads, 0, s>>>(part_p, part_c, static_cast<int32_t>(P), E, topk, coef, counts, loss);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

template <typename TL>
int gate_backward_launch(const void* logits, int64_t T, int32_t E, int64_t ldl, int32_t topk, int32_t renorm,
                         const uint8_t* mask, float coef, const int32_t* ids, const int32_t* counts,
                         const float* dweights, const float* dloss, void* dlogits, int64_t ldd, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(kGateWarps + 1) * E * 4;
  int st = allow_smem(moe_gate_backward_kernel<TL>, smem);
  if (st != FP8G_OK) return st;
  const int64_t ctas = std::min<int64_t>((T + kGateWarps - 1) / kGateWarps, 8 * kGateMaxCtas);
  moe_gate_backward_kernel<TL><<<static_cast<unsigned>(ctas), kGateThreads, smem, s>>>(
      static_cast<const TL*>(logits), T, E, ldl, topk, renorm, mask, coef, ids, counts, dweights, dloss,
      static_cast<TL*>(dlogits), ldd);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_moe_gate_workspace(int64_t T, int32_t E, int64_t* bytes) {
  if (T < 0 || T > 0x7FFFFFFF || E < 1 || E > kGateMaxExperts || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = gate_ctas(T) * E * 8;
  return FP8G_OK;
}

extern "C" int fp8g_moe_gate(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ldl, int32_t topk,
                             int32_t renormalize, const uint8_t* token_mask, float loss_coef, int32_t* topk_ids,
                             float* topk_weights, int32_t* counts, float* loss, void* workspace,
                             int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || T < 0 || T > 0x7FFFFFFF || E < 1 || E > kGateMaxExperts || ldl < E || topk < 1 ||
      topk > kGateMaxTopk || topk > E || (renormalize != 0 && renormalize != 1) || T * topk > 0x7FFFFFFF)
    return FP8G_ERR_INVALID_ARG;
  if (!counts || (T > 0 && (!logits || !topk_ids || !topk_weights))) return FP8G_ERR_INVALID_ARG;
  if (T > 0 && (!workspace || workspace_bytes < gate_ctas(T) * E * 8)) return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(logits, dtype_size(dtype)) || !aligned_to(topk_ids, 4) || !aligned_to(topk_weights, 4) ||
      !aligned_to(counts, 4) || !aligned_to(loss, 4) || !aligned16(workspace))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {  // no tokens: nothing chosen, no loss
    if (cudaMemsetAsync(counts, 0, static_cast<size_t>(E) * 4, s) != cudaSuccess ||
        (loss && cudaMemsetAsync(loss, 0, 4, s) != cudaSuccess)) {
      cudaGetLastError();
      return FP8G_ERR_CUDA;
    }
    return FP8G_OK;
  }
  auto go = dtype == FP8G_F32 ? gate_launch<float> : gate_launch<__nv_bfloat16>;
  return go(logits, T, E, ldl, topk, renormalize, token_mask, loss_coef, topk_ids, topk_weights, counts, loss,
            workspace, s);
}

extern "C" int fp8g_moe_gate_backward(const void* logits, int32_t dtype, int64_t T, int32_t E, int64_t ldl,
                                      int32_t topk, int32_t renormalize, const uint8_t* token_mask,
                                      float loss_coef, const int32_t* topk_ids, const int32_t* counts,
                                      const float* dweights, const float* dloss, void* dlogits, int64_t ldd,
                                      void* stream) {
  if (!dtype_ok(dtype) || T < 0 || T > 0x7FFFFFFF || E < 1 || E > kGateMaxExperts || ldl < E || ldd < E ||
      topk < 1 || topk > kGateMaxTopk || topk > E || (renormalize != 0 && renormalize != 1) ||
      T * topk > 0x7FFFFFFF)
    return FP8G_ERR_INVALID_ARG;
  if (T == 0) return FP8G_OK;
  if (!logits || !topk_ids || !counts || !dlogits) return FP8G_ERR_INVALID_ARG;
  if (!aligned_to(logits, dtype_size(dtype)) || !aligned_to(dlogits, dtype_size(dtype)) ||
      !aligned_to(topk_ids, 4) || !aligned_to(counts, 4) || !aligned_to(dweights, 4) || !aligned_to(dloss, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  auto go = dtype == FP8G_F32 ? gate_backward_launch<float> : gate_backward_launch<__nv_bfloat16>;
  return go(logits, T, E, ldl, topk, renormalize, token_mask, loss_coef, topk_ids, counts, dweights, dloss, dlogits,
            ldd, static_cast<cudaStream_t>(stream));
}

extern "C" int fp8g_moe_combine(const void* D, int64_t M, int64_t N, int64_t ldd, const int32_t* entry_row,
                                int64_t T, int32_t topk, const float* weights, const void* residual, int64_t ldr,
                                void* out, int32_t out_dtype, int64_t ldo, void* stream) {
  if (!dtype_ok(out_dtype) || M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || N % 8 != 0 || ldd < N ||
      T < 0 || T > 0x7FFFFFFF || topk < 1 || T * topk > 0x7FFFFFFF || ldo < N || (residual && ldr < N))
    return FP8G_ERR_INVALID_ARG;
  if (T == 0) return FP8G_OK;
  if ((M > 0 && !D) || !entry_row || !out) return FP8G_ERR_INVALID_ARG;
  if (!aligned16(D) || !aligned16(out) || !aligned16(residual) || ldd % 8 != 0 || ldo % 8 != 0 ||
      (residual && ldr % 8 != 0) || !aligned_to(entry_row, 4) || !aligned_to(weights, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (out_dtype == FP8G_F32)
    moe_combine_kernel<float><<<static_cast<unsigned>(T), kCombineThreads, 0, s>>>(
        static_cast<const __nv_bfloat16*>(D), M, N, ldd, entry_row, topk, weights,
        static_cast<const float*>(residual), ldr, static_cast<float*>(out), ldo, dev->status);
  else
    moe_combine_kernel<__nv_bfloat16><<<static_cast<unsigned>(T), kCombineThreads, 0, s>>>(
        static_cast<const __nv_bfloat16*>(D), M, N, ldd, entry_row, topk, weights,
        static_cast<const __nv_bfloat16*>(residual), ldr, static_cast<__nv_bfloat16*>(out), ldo, dev->status);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

extern "C" int fp8g_moe_combine_backward(const void* dout, int32_t dout_dtype, int64_t lddo, const void* D, int64_t M,
                                         int64_t N, int64_t ldd, const int32_t* entry_row,
                                         const int32_t* row_token, int64_t T, int32_t topk, const float* weights,
                                         void* dD, int64_t lddd, float* dweights, void* stream) {
  if (!dtype_ok(dout_dtype) || M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || N % 8 != 0 || lddd < N ||
      T < 0 || T > 0x7FFFFFFF || topk < 1 || T * topk > 0x7FFFFFFF || lddo < N || (dweights && ldd < N))
    return FP8G_ERR_INVALID_ARG;
  if (M == 0 && T == 0) return FP8G_OK;
  if ((M > 0 && (!dD || !row_token || (dweights && !D))) || (T > 0 && (!entry_row || !dout)))
    return FP8G_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(D) || !aligned16(dD) || lddo % 8 != 0 || (dweights && ldd % 8 != 0) ||
      lddd % 8 != 0 || !aligned_to(entry_row, 4) || !aligned_to(row_token, 4) || !aligned_to(weights, 4) ||
      !aligned_to(dweights, 4))
    return FP8G_ERR_ALIGNMENT;
  DeviceInfo* dev = nullptr;
  int st = current_device(&dev);
  if (st != FP8G_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(std::max<int64_t>(T, std::min<int64_t>(M, 1216)));
  if (dout_dtype == FP8G_F32)
    moe_combine_backward_kernel<float><<<grid, kCombineThreads, 0, s>>>(
        static_cast<const float*>(dout), lddo, static_cast<const __nv_bfloat16*>(D), M, N, ldd, entry_row, row_token, T,
        topk, weights, static_cast<__nv_bfloat16*>(dD), lddd, dweights, dev->status);
  else
    moe_combine_backward_kernel<__nv_bfloat16><<<grid, kCombineThreads, 0, s>>>(
        static_cast<const __nv_bfloat16*>(dout), lddo, static_cast<const __nv_bfloat16*>(D), M, N, ldd, entry_row,
        row_token, T, topk, weights, static_cast<__nv_bfloat16*>(dD), lddd, dweights, dev->status);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}
