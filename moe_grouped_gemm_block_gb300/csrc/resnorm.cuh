// resnorm.cuh -- what the forward and the backward kernels of the norms around a block (resnorm.cu, resnorm_grad.cu)
// share: how a row falls to threads, the copies that bring rows ahead of them, sums over a row.
#pragma once

#include <algorithm>
#include <cuda_runtime.h>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kResMaxThreads = 512;
constexpr int kResMaxStages = 3;

struct ResArgs {
  const void *x, *f, *w, *post, *gate, *dy, *dh;  // backward: x is h
  void *h, *y, *dx, *df;
  float *rstd, *rstd_f;  // results of the forward, inputs of the backward call
  float* parts;          // [CTAs][2][N]
  int64_t M, ldx, ldf, ldh, ldy, lddy, lddh, lddx, lddf;
  int32_t N, w_kind, norm_f, stages, keep;  // keep: the weights lie in shared memory
  float scale, eps, inv_n;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, of which `bytes` are read and the others are zero.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of this thread's groups of copies but the last `later` (0 .. kResMaxStages - 1) have landed.
__device__ __forceinline__ void cp_async_wait(int later) {
  if (later == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (later == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// How a row of N columns falls to its R threads, eight values at a time, V times.
//
// VEC: in vectors on the 16-byte grid.  Where rows start off it, row m does q = (m ld) mod 8 values after a vector's start,
// in all matrices alike (the host checks), and its first and last vectors reach into what lies beside it, which is read
// and left out (but nothing past the row's end is read).  q repeats every 8 rows, so a thread that steps by multiples
// of 8 rows keeps its columns, and with them its weights and column sums.  Else (rows that share no grid): value by value,
// neighbouring threads on neighbouring values.
//
// A thread's values of the rows to come are copied ahead of it into places of its own in shared memory (`slot`: of the
// CTA's threads' places of a matrix), and so are its weights, once: nobody waits for anybody else's, a thread orders its
// own reads and copies.  (bf16 value by value is too narrow for such copies: it is loaded when it is needed.  Weights read
// from L1 in every row, which the stages leave too little of, made 8192 x 7168 backward 379 us.)
template <bool VEC, int V>
struct Columns {
  int t, R, N, q;
  template <typename T>
  static constexpr bool staged() { return VEC || sizeof(T) == 4; }
  template <typename T>
  static __host__ __device__ constexpr int slot_bytes() { return staged<T>() ? V * 8 * static_cast<int>(sizeof(T)) : 0; }
  __device__ __forceinline__ int at(int v, int j) const { return VEC ? 8 * (t + v * R) + j - q : t + (8 * v + j) * R; }
  __device__ __forceinline__ bool has(int v, int j) const { return at(v, j) < N && (!VEC || at(v, j) >= 0); }
  // VEC: all eight are the row's
  __device__ __forceinline__ bool whole(int v) const { return at(v, 0) >= 0 && at(v, 7) < N; }
  template <typename T>
  __device__ __forceinline__ void copy(uint32_t slot, const T* row) const {
    const uint32_t to = slot + threadIdx.x * (VEC ? 16 : 4), step = blockDim.x * (VEC ? 16 : 4);
    if constexpr (VEC) {
      constexpr int kChunks = sizeof(T) / 2, kPer = 8 / kChunks;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (at(v, 7) < N) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) cp_async_16(to + (v * kChunks + c) * step, row + at(v, c * kPer));
        } else {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int first = at(v, c * kPer), n = min(kPer, N - first);
            if (n > 0) cp_async_16(to + (v * kChunks + c) * step, row + first, n * static_cast<int>(sizeof(T)));
          }
        }
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8 * V; ++i)
        if (has(i / 8, i % 8)) cp_async_4(to + i * step, row + at(i / 8, i % 8));
    }
  }
  // Eight values; 0 where there are none (`real`: the row exists).
  template <typename T>
  __device__ __forceinline__ void load(Raw8<T>& r, uint32_t slot, const T* row, int v, bool real) const {
    const uint32_t from = slot + threadIdx.x * (VEC ? 16 : 4), step = blockDim.x * (VEC ? 16 : 4);
    if constexpr (VEC) {
      if constexpr (sizeof(T) == 2) {
        const float4 a = ld_shared_v4f(from + v * step);
        r.v = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z), __float_as_uint(a.w));
      } else {
        r.a = ld_shared_v4f(from + 2 * v * step);
        r.b = ld_shared_v4f(from + (2 * v + 1) * step);
      }
      if (!real || !whole(v)) {
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) mask |= (real && has(v, j) ? 1u : 0u) << j;
        r.keep(mask);
      }
    } else {
      T f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] = from_f32<T>(0.0f);
        if (real && has(v, j)) {
          if constexpr (sizeof(T) == 4) f[j] = ld_shared_f32(from + (8 * v + j) * step);
          else f[j] = row[at(v, j)];
        }
      }
      r.set(f);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int v, const float2 (&f)[4]) const {
    if (VEC && whole(v)) {
      store8_stream(row + at(v, 0), {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y});
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (has(v, j)) row[at(v, j)] = from_f32<T>(j & 1 ? f[j / 2].y : f[j / 2].x);
    }
  }
  // This thread's weights, the product of two of them (null: 1) and a factor, into its places.
  static __host__ __device__ constexpr int weight_bytes() { return V * 32; }
  __device__ __forceinline__ void keep_weights(float* slot, const void* a, const void* b, int kind, float by) const {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float w = by;
        if (has(v, j)) {
          if (a) w *= load_any(a, kind, at(v, j));
          if (b) w *= load_any(b, kind, at(v, j));
        }
        slot[((2 * v + j / 4) * blockDim.x + threadIdx.x) * 4 + j % 4] = w;
      }
  }
  // f *= the weights: from this thread's places, or (slot null) from memory
  __device__ __forceinline__ void times(const float* slot, const void* a, const void* b, int kind, float by, int v,
                                        float2 (&f)[4]) const {
    if (slot) {
      const float4* p = reinterpret_cast<const float4*>(slot) + 2 * v * blockDim.x + threadIdx.x;
      const float4 x = p[0], y = p[blockDim.x];
      f[0] = __fmul2_rn(f[0], make_float2(x.x, x.y));
      f[1] = __fmul2_rn(f[1], make_float2(x.z, x.w));
      f[2] = __fmul2_rn(f[2], make_float2(y.x, y.y));
      f[3] = __fmul2_rn(f[3], make_float2(y.z, y.w));
      return;
    }
    if (a) from_memory(a, kind, v, f);
    if (b) from_memory(b, kind, v, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], make_float2(by, by));
  }
  __device__ __forceinline__ void from_memory(const void* w, int kind, int v, float2 (&f)[4]) const {
    if (VEC && q == 0 && whole(v) && (reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
      float2 g[4];
      if (kind == FP8G_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at(v, 0));
        const float4 x = __ldg(p), y = __ldg(p + 1);
        g[0] = make_float2(x.x, x.y), g[1] = make_float2(x.z, x.w), g[2] = make_float2(y.x, y.y), g[3] = make_float2(y.z, y.w);
      } else {
        Raw8<__nv_bfloat16> r;
        r.v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + at(v, 0)));
        r.get(g);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], g[i]);
      return;
    }
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = has(v, j) ? load_any(w, kind, at(v, j)) : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], make_float2(g[2 * i], g[2 * i + 1]));
  }
};
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The sum over the threads of a row: LPR lanes of a warp, or (LPR 0) the CTA, whose entries of `red` past its warps are 0.
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
    for (int i = 0; i < kResMaxThreads / 128; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(r + 4 * i);
      s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
    }
    return (s.x + s.y) + (s.z + s.w);
  }
}
__device__ __forceinline__ void res_sum_init(float (*red)[32]) {
  for (int i = threadIdx.x; i < 64; i += blockDim.x) (&red[0][0])[i] = 0.0f;
  __syncthreads();
}
__device__ __forceinline__ float root_inverse(float mean_square, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(mean_square + eps));
}

// The form of a row's length: LPR lanes of a warp (0: a CTA; -1: any length), V eights a thread.
struct ResForm {
  int lpr, v, threads, rows;  // rows a CTA at once
};
inline ResForm res_form(int64_t N, bool shifted, bool backward) {  // shifted: a row may take a vector more
  const int64_t eights = (N + (shifted ? 7 : 0) + 7) / 8;
  if (eights <= 8) return {8, 1, 256, 32};
  if (eights <= 16) return {16, 1, 256, 16};
  if (eights <= 32) return {32, 1, 256, 8};
  if (eights <= 64) return {32, 2, 256, 8};
  if (eights > 4 * kResMaxThreads) return {-1, 1, kResMaxThreads, 1};
  const int v = eights <= 512 && !backward ? 1 : eights <= 1024 ? 2 : 4;
  return {0, v, static_cast<int>(((eights + v - 1) / v + 31) / 32 * 32), 1};
}
// Shared memory of a CTA, where `per_sm` of them are to be resident: `weights` bytes of weights (left in memory where
// they would take too much) and up to kResMaxStages stages of `stage` bytes.
struct ResShared {
  int64_t bytes;
  int32_t stages, weights;  // stages 0: not even one fits (such rows are taken as rows of any length)
};
inline ResShared res_shared(int64_t stage, int64_t weights, int per_sm) {
  constexpr int64_t kMost = 220 * 1024;
  const int64_t each = std::max<int64_t>(kMost / per_sm - 1024, 0);
  const bool keep = weights + stage <= each;
  const int64_t left = each - (keep ? weights : 0);
  const int64_t n = std::min<int64_t>(kResMaxStages, stage ? left / stage : 1);
  return {n * stage + (keep ? weights : 0), static_cast<int32_t>(n), keep ? 1 : 0};
}

inline bool bad_type(int32_t t) { return t != FP8G_BF16 && t != FP8G_F32; }
inline int64_t type_size(int32_t t) { return t == FP8G_F32 ? 4 : 2; }
// How the rows of all matrices of a call lie: all on the 16-byte grid (aligned), all off it by the same in every row
// (shifted), or not so.
enum class ResGrid { kAligned, kShifted, kNone };
inline ResGrid res_grid(int64_t M, int64_t N, std::initializer_list<std::pair<const void*, int64_t>> matrices) {
  int64_t ld = -1;
  for (const auto& [p, l] : matrices) {
    if (!p) continue;
    if (!aligned16(p) || (M > 1 && ld >= 0 && (l - ld) % 8 != 0)) return ResGrid::kNone;
    ld = l;
  }
  return N % 8 == 0 && (M == 1 || ld % 8 == 0) ? ResGrid::kAligned : ResGrid::kShifted;
}

}  // namespace
}  // namespace fp8g
