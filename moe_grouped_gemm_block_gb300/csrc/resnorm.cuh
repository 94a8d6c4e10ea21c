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
constexpr int kResCluster = 2;  // CTAs of a row beyond 8192 values

struct ResArgs {
  const void *x, *f, *w, *post, *gate, *dy, *dh;  // backward: x is h
  void *h, *y, *dx, *df;
  float *rstd, *rstd_f;  // results of the forward, inputs of the backward call
  float* parts;          // [rows at once][2][N]
  int64_t M, ldx, ldf, ldh, ldy, lddy, lddh, lddx, lddf;
  int32_t N, w_kind, norm_f, stages, ranks;  // ranks: CTAs a row
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


// How a row falls to its threads: R threads of a CTA, which has the columns [lo, end) of it, take eight values at a time, V
// times.
//   kAligned  in vectors; every row lies on the 16-byte grid
//   kShifted  in vectors on the grid, but row m starts q = (m ld) mod 8 values after a vector's start, in all matrices
//             alike (the host checks): its first and last vectors reach into what lies beside it, which is read and left
//             out (nothing past the row's end is read).  q repeats every 8 rows, so a thread that steps by multiples of 8
//             rows keeps its columns, and with them its weights and column sums.
//   kSingle   rows that share no grid: value by value, neighbouring threads on neighbouring values
//
// A thread's values of the rows to come are copied ahead of it into places of its own in shared memory, and so are its
// weights, once: nobody waits for anybody else's, a thread orders its own reads and copies.  Places without a column, and
// those of a matrix that is not there, hold zeros from the start, so that no row asks what there is.  (bf16 value by value
// is too narrow for such copies: it is loaded when it is needed.)
enum ResMode { kAligned, kShifted, kSingle };
template <int MODE, int V>
struct Columns {
  int t, R, lo, end;
  __device__ __forceinline__ int at(int v, int j) const {
    return MODE == kSingle ? lo + t + (8 * v + j) * R : lo + 8 * (t + v * R) + j;
  }
  __device__ __forceinline__ bool has(int v, int j) const { return at(v, j) < end && (MODE != kShifted || at(v, j) >= 0); }
  __device__ __forceinline__ bool whole(int v) const {
    return MODE == kAligned ? at(v, 0) < end : at(v, 0) >= 0 && at(v, 7) < end;
  }
  // 8 V float32 weights, the product of two vectors (null: 1) and a factor, in places of 16 bytes a thread
  __device__ __forceinline__ void keep_weights(float4* to, const void* a, const void* b, int kind, float by) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float2 f[4] = {make_float2(by, by), make_float2(by, by), make_float2(by, by), make_float2(by, by)};
      if (a) from_memory(a, kind, v, f);
      if (b) from_memory(b, kind, v, f);
      to[2 * v * blockDim.x + threadIdx.x] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      to[(2 * v + 1) * blockDim.x + threadIdx.x] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
  }
  __device__ __forceinline__ void times(const float4* w, int v, float2 (&f)[4]) const {
    const float4 x = w[2 * v * blockDim.x + threadIdx.x], y = w[(2 * v + 1) * blockDim.x + threadIdx.x];
    f[0] = __fmul2_rn(f[0], make_float2(x.x, x.y));
    f[1] = __fmul2_rn(f[1], make_float2(x.z, x.w));
    f[2] = __fmul2_rn(f[2], make_float2(y.x, y.y));
    f[3] = __fmul2_rn(f[3], make_float2(y.z, y.w));
  }
  __device__ __forceinline__ void from_memory(const void* w, int kind, int v, float2 (&f)[4]) const {
    float g[8];
    if (MODE == kAligned && (reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
      if (!whole(v)) return;
      if (kind == FP8G_F32) load8(static_cast<const float*>(w) + at(v, 0), g);
      else load8(static_cast<const __nv_bfloat16*>(w) + at(v, 0), g);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = has(v, j) ? load_any(w, kind, at(v, j)) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(f[i], make_float2(g[2 * i], g[2 * i + 1]));
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int v, const float2 (&f)[4]) const {
    if (MODE != kSingle && whole(v)) {
      store8_stream(row + at(v, 0), {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y});
    } else if (MODE != kAligned) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (has(v, j)) row[at(v, j)] = from_f32<T>(j & 1 ? f[j / 2].y : f[j / 2].x);
    }
  }
};

// A thread's places of one matrix: stage s at slot + s stride.
template <typename T, int MODE, int V>
struct Source {
  static constexpr bool kStaged = MODE != kSingle || sizeof(T) == 4;
  static constexpr int kPlace = MODE == kSingle ? 4 : 16;  // bytes of a copy
  static constexpr int kCopies = kStaged ? V * 8 * static_cast<int>(sizeof(T)) / kPlace : 0;
  static __host__ __device__ constexpr int thread_bytes() { return kCopies * kPlace; }
  const T* row;   // the row to be copied next (loaded next, where it is not staged)
  int64_t step;   // elements to the one after it
  uint32_t slot, stride;
  // `matrix` null: the places at `slot` of one stage hold zeros
  __device__ __forceinline__ void init(const void* matrix, int64_t m, int64_t ld, int64_t rows, uint32_t at, uint32_t stage,
                                       int stages, const Columns<MODE, V>& col) {
    row = matrix ? static_cast<const T*>(matrix) + m * ld : nullptr;
    step = rows * ld;
    slot = at + threadIdx.x * kPlace;
    stride = matrix ? stage : 0u;
    for (int s = 0; s < (matrix ? stages : 1); ++s)
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const uint32_t to = slot + s * stride + i * blockDim.x * kPlace;
        if constexpr (MODE == kSingle) {
          if (!matrix || !col.has(i / 8, i % 8)) asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(0u) : "memory");
        } else {
          constexpr int kChunks = sizeof(T) / 2;
          if (!matrix || !col.whole(i / kChunks)) st_shared_v4(to, 0u, 0u, 0u, 0u);
        }
      }
  }
  __device__ __forceinline__ void copy(int s, const Columns<MODE, V>& col) const {
    if constexpr (!kStaged) return;
    if (!row) return;
    const uint32_t to = slot + s * stride, next = blockDim.x * kPlace;
    if constexpr (MODE == kSingle) {
#pragma unroll
      for (int i = 0; i < 8 * V; ++i)
        if (col.has(i / 8, i % 8)) cp_async_4(to + i * next, row + col.at(i / 8, i % 8));
    } else {
      constexpr int kChunks = sizeof(T) / 2, kPer = 8 / kChunks;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (MODE == kAligned ? col.whole(v) : col.at(v, 7) < col.end) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) cp_async_16(to + (v * kChunks + c) * next, row + col.at(v, c * kPer));
        } else if (MODE == kShifted) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int n = min(kPer, col.end - col.at(v, c * kPer));
            if (n > 0) cp_async_16(to + (v * kChunks + c) * next, row + col.at(v, c * kPer), n * static_cast<int>(sizeof(T)));
          }
        }
      }
    }
  }
  // Eight values of stage s; 0 where there are none.
  __device__ __forceinline__ void load(Raw8<T>& r, int s, int v, const Columns<MODE, V>& col) const {
    const uint32_t from = slot + s * stride, next = blockDim.x * kPlace;
    if constexpr (MODE != kSingle) {
      if constexpr (sizeof(T) == 2) {
        const float4 a = ld_shared_v4f(from + v * next);
        r.v = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(a.z), __float_as_uint(a.w));
      } else {
        r.a = ld_shared_v4f(from + 2 * v * next);
        r.b = ld_shared_v4f(from + (2 * v + 1) * next);
      }
      if (MODE == kShifted && !col.whole(v)) {
        uint32_t mask = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) mask |= (col.has(v, j) ? 1u : 0u) << j;
        r.keep(mask);
      }
    } else {
      T f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (kStaged) f[j] = ld_shared_f32(from + (8 * v + j) * next);
        else f[j] = row && col.has(v, j) ? row[col.at(v, j)] : from_f32<T>(0.0f);
      }
      r.set(f);
    }
  }
};

// The sum over the threads of a row: LPR lanes of a warp, or (LPR 0) the CTAs of a cluster, of which each warp tells all
// its sum; entries of `red` past the warps are 0.
template <int LPR>
__device__ __forceinline__ float res_sum(float v, float (*red)[32], int& phase, int ranks) {
  if constexpr (LPR > 0) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  } else {
    v = warp_sum(v);
    float* r = red[phase & 1];
    ++phase;
    const int warp = threadIdx.x >> 5;
    if (ranks == 1) {
      if ((threadIdx.x & 31) == 0) r[warp] = v;
      __syncthreads();
    } else {
      if ((threadIdx.x & 31) < ranks) {
        const uint32_t to = mapa_shared(smem_u32(r + static_cast<int>(cluster_ctarank()) * 16 + warp), threadIdx.x & 31);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
      }
      cluster_sync();
    }
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int quads = ranks == 1 ? 4 : 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= quads) break;
      const float4 q = *reinterpret_cast<const float4*>(r + 4 * i);
      s.x += q.x, s.y += q.y, s.z += q.z, s.w += q.w;
    }
    return (s.x + s.y) + (s.z + s.w);
  }
}
__device__ __forceinline__ void res_sum_init(float (*red)[32], int ranks) {
  for (int i = threadIdx.x; i < 64; i += blockDim.x) (&red[0][0])[i] = 0.0f;
  __syncthreads();
  if (ranks > 1) cluster_sync();
}
__device__ __forceinline__ float root_inverse(float mean_square, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(mean_square + eps));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The form of a row's length: LPR lanes of a warp (0: CTAs), V eights a thread, `ranks` CTAs a row; lpr -1: any length.
struct ResForm {
  int lpr, v, threads, rows, ranks;  // rows a CTA at once
};
inline ResForm res_form(int64_t N, ResMode mode, bool backward) {
  const int64_t eights = (N + (mode == kShifted ? 7 : 0) + 7) / 8;
  if (mode == kSingle && eights <= 64) return {32, eights <= 32 ? 1 : 2, 256, 8, 1};
  if (eights <= 8) return {8, 1, 256, 32, 1};
  if (eights <= 16) return {16, 1, 256, 16, 1};
  if (eights <= 64) return {32, eights <= 32 ? 1 : 2, 256, 8, 1};
  const int ranks = eights <= 2 * kResMaxThreads ? 1 : kResCluster;
  const int64_t mine = (eights + ranks - 1) / ranks;
  if (mine > 2 * kResMaxThreads) return {-1, 1, kResMaxThreads, 1, 1};
  const int v = mine <= kResMaxThreads && !backward && ranks == 1 ? 1 : 2;
  return {0, v, static_cast<int>(((mine + v - 1) / v + 31) / 32 * 32), 1, ranks};
}
// Shared memory of a CTA, where `per_sm` of them are to be resident: `weights` bytes of weights, `zeros` bytes of zeros, and
// up to kResMaxStages stages of `stage` bytes.  stages 0: not even one fits (such rows are taken as rows of any length).
struct ResShared {
  int64_t bytes;
  int32_t stages;
};
inline ResShared res_shared(int64_t stage, int64_t weights, int64_t zeros, int per_sm) {
  const int64_t each = 224 * 1024 / per_sm - 1024, left = each - weights - zeros;
  const int64_t n = left < 0 ? 0 : std::min<int64_t>(kResMaxStages, stage ? left / stage : 1);
  return {n * stage + weights + zeros, static_cast<int32_t>(n)};
}

inline bool bad_type(int32_t t) { return t != FP8G_BF16 && t != FP8G_F32; }
inline int64_t type_size(int32_t t) { return t == FP8G_F32 ? 4 : 2; }
// How the rows of all matrices of a call lie.
inline ResMode res_mode(int64_t M, int64_t N, std::initializer_list<std::pair<const void*, int64_t>> matrices) {
  int64_t ld = -1;
  for (const auto& [p, l] : matrices) {
    if (!p) continue;
    if (!aligned16(p) || (M > 1 && ld >= 0 && (l - ld) % 8 != 0)) return kSingle;
    ld = l;
  }
  return N % 8 == 0 && (M == 1 || ld % 8 == 0) ? kAligned : kShifted;
}
// bytes of a thread's places of a matrix whose values have `size` bytes
inline int64_t res_thread_bytes(ResMode mode, int v, int64_t size) { return mode == kSingle && size == 2 ? 0 : v * 8 * size; }

// Launches a kernel, as clusters where a row has several CTAs.
template <typename Kernel>
int res_launch(Kernel kernel, int64_t ctas, int threads, int64_t smem, int ranks, const ResArgs& a, cudaStream_t s) {
  const int st = allow_shared_memory(reinterpret_cast<const void*>(kernel), static_cast<size_t>(smem + 1024));  // (and what is static)
  if (st != FP8G_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

// What every row kernel starts with: its rows, its columns.
#define FP8G_RES_ROWS(ld)                                                                                              \
  constexpr int kRows = LPR ? 256 / (LPR ? LPR : 1) : 1;                                                               \
  const int mine = LPR ? static_cast<int>(threadIdx.x) / (LPR ? LPR : 1) : 0;                                          \
  const int rank = LPR == 0 && a.ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;                                  \
  const int64_t block = LPR == 0 ? blockIdx.x / a.ranks : blockIdx.x, blocks = LPR == 0 ? gridDim.x / a.ranks : gridDim.x; \
  const int64_t m_first = block * kRows, step = blocks * kRows;                                                        \
  const int shift = MODE == kShifted && a.M > 1 ? static_cast<int>((m_first + mine) % 8 * ((ld) & 7)) & 7 : 0;         \
  const int share = ((a.N + shift + 7) / 8 + a.ranks - 1) / a.ranks * 8;                                               \
  const Cols col{LPR ? static_cast<int>(threadIdx.x) % (LPR ? LPR : 1) : static_cast<int>(threadIdx.x),                \
                 LPR ? LPR : static_cast<int>(blockDim.x), rank * share - shift,                                       \
                 LPR ? a.N : min(a.N, (rank + 1) * share - shift)};

}  // namespace
}  // namespace fp8g
