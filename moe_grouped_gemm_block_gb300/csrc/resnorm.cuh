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
  float* parts;          // [rows at once][2][N]
  int64_t M, ldx, ldf, ldh, ldy, lddy, lddh, lddx, lddf;
  int32_t N, w_kind, norm_f, stages, stages_f, ranks;  // stages_f: of f, stages or one less; ranks: CTAs a row
  float scale, eps, inv_n;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All of this thread's groups of copies but the last `later` (at most 4) have landed.
__device__ __forceinline__ void cp_async_wait(int later) {
  if (later == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (later == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else if (later == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (later == 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
  else asm volatile("cp.async.wait_group 4;" ::: "memory");
}


// How a row falls to its threads: R threads of a CTA, which has the columns [lo, end) of it, take G values at a time, V
// times.  G is 8 where all matrices are bf16 and 4 where one is fp32, so that a warp's 16-byte accesses to the wider type
// lie side by side.
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
template <typename TS, typename TB>
__host__ __device__ constexpr int res_unit() { return sizeof(TS) == 4 || sizeof(TB) == 4 ? 4 : 8; }
// G values as they lie in memory.
template <typename T, int G>
struct Unit {
  static constexpr int kWords = G * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void get(float2 (&f)[G / 2]) const {
#pragma unroll
    for (int i = 0; i < G / 2; ++i)
      f[i] = sizeof(T) == 4 ? make_float2(__uint_as_float(w[2 * i % kWords]), __uint_as_float(w[(2 * i + 1) % kWords]))
                            : make_float2(__uint_as_float(w[i % kWords] << 16), __uint_as_float(w[i % kWords] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void set(int j, T v) {  // value j, of zeros
    if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(v);
    else w[j / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(v)) << (16 * (j & 1));
  }
  __device__ __forceinline__ void keep(int j, bool yes) {
    if constexpr (sizeof(T) == 4) w[j] = yes ? w[j] : 0u;
    else w[j / 2] &= yes ? 0xFFFFFFFFu : (j & 1 ? 0xFFFFu : 0xFFFF0000u);
  }
};
template <int MODE, int G, int V>
struct Columns {
  int t, R, lo, end;
  __device__ __forceinline__ int at(int v, int j) const {
    return MODE == kSingle ? lo + t + (G * v + j) * R : lo + G * (t + v * R) + j;
  }
  __device__ __forceinline__ bool has(int v, int j) const { return at(v, j) < end && (MODE != kShifted || at(v, j) >= 0); }
  __device__ __forceinline__ bool whole(int v) const {
    return MODE == kAligned ? at(v, 0) < end : at(v, 0) >= 0 && at(v, G - 1) < end;
  }
  // G V fp32 weights, the product of two vectors (null: 1) and a factor, in places of 16 bytes a thread
  __device__ __forceinline__ void keep_weights(float4* to, const void* a, const void* b, int kind, float by) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[G];
#pragma unroll
      for (int j = 0; j < G; ++j) f[j] = by;
      if (a) from_memory(a, kind, v, f);
      if (b) from_memory(b, kind, v, f);
#pragma unroll
      for (int c = 0; c < G / 4; ++c)
        to[(v * (G / 4) + c) * blockDim.x + threadIdx.x] = make_float4(f[4 * c], f[4 * c + 1], f[4 * c + 2], f[4 * c + 3]);
    }
  }
  __device__ __forceinline__ void from_memory(const void* w, int kind, int v, float (&f)[G]) const {
    if (MODE == kAligned && (reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
      if (!whole(v)) return;
      float2 g[G / 2];
      if (kind == FP8G_F32) {
#pragma unroll
        for (int c = 0; c < G / 4; ++c) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(w) + at(v, 4 * c)));
          g[2 * c] = make_float2(x.x, x.y), g[2 * c + 1] = make_float2(x.z, x.w);
        }
      } else {
        Unit<__nv_bfloat16, G> u;
#pragma unroll
        for (int c = 0; c < G / 4; ++c) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + at(v, 4 * c)));
          u.w[2 * c] = x.x, u.w[2 * c + 1] = x.y;
        }
        u.get(g);
      }
#pragma unroll
      for (int j = 0; j < G; ++j) f[j] *= j & 1 ? g[j / 2].y : g[j / 2].x;
    } else {
#pragma unroll
      for (int j = 0; j < G; ++j) f[j] *= has(v, j) ? load_any(w, kind, at(v, j)) : 0.0f;
    }
  }
  // the weights of unit v
  __device__ __forceinline__ void weights(const float4* w, int v, float2 (&f)[G / 2]) const {
#pragma unroll
    for (int c = 0; c < G / 4; ++c) {
      const float4 x = w[(v * (G / 4) + c) * blockDim.x + threadIdx.x];
      f[2 * c] = make_float2(x.x, x.y), f[2 * c + 1] = make_float2(x.z, x.w);
    }
  }
  __device__ __forceinline__ void times(const float4* w, int v, float2 (&f)[G / 2]) const {
    float2 g[G / 2];
    weights(w, v, g);
#pragma unroll
    for (int i = 0; i < G / 2; ++i) f[i] = __fmul2_rn(f[i], g[i]);
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int v, const float2 (&f)[G / 2]) const {
    if (MODE != kSingle && whole(v)) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int c = 0; c < G / 4; ++c)
          __stcs(reinterpret_cast<float4*>(row + at(v, 4 * c)), make_float4(f[2 * c].x, f[2 * c].y, f[2 * c + 1].x, f[2 * c + 1].y));
      } else if constexpr (G == 8) {
        __stcs(reinterpret_cast<uint4*>(row + at(v, 0)),
               make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y), pack2(f[3].x, f[3].y)));
      } else {
        __stcs(reinterpret_cast<uint2*>(row + at(v, 0)), make_uint2(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y)));
      }
    } else if (MODE != kAligned) {
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (has(v, j)) row[at(v, j)] = from_f32<T>(j & 1 ? f[j / 2].y : f[j / 2].x);
    }
  }
};

// A thread's places of one matrix: stage s at slot + s stride.
template <typename T, int MODE, int G, int V>
struct Source {
  using Cols = Columns<MODE, G, V>;
  static constexpr bool kStaged = MODE != kSingle || sizeof(T) == 4;
  static constexpr int kUnit = G * static_cast<int>(sizeof(T));                         // bytes of G values
  static constexpr int kPlace = MODE == kSingle ? 4 : kUnit < 16 ? kUnit : 16;          // bytes of a copy
  static constexpr int kCopies = kStaged ? V * kUnit / kPlace : 0, kChunks = kUnit / kPlace, kPer = G / kChunks;
  static __host__ __device__ constexpr int thread_bytes() { return kCopies * kPlace; }
  const T* row;   // the row to be copied next (loaded next, where it is not staged)
  int64_t step;   // elements to the one after it
  uint32_t slot, stride;
  static __device__ __forceinline__ void copy_place(uint32_t to, const T* from, int bytes) {
    if constexpr (kPlace == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    } else if constexpr (kPlace == 8) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    } else {
      cp_async_4(to, from);
    }
  }
  static __device__ __forceinline__ void copy_place(uint32_t to, const T* from) {
    if constexpr (kPlace == 16) cp_async_16(to, from);
    else if constexpr (kPlace == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
    else cp_async_4(to, from);
  }
  static __device__ __forceinline__ void zero_place(uint32_t to) {
#pragma unroll
    for (int b = 0; b < kPlace; b += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + b), "r"(0u) : "memory");
  }
  // `matrix` null: the places at `slot` of one stage hold zeros
  __device__ __forceinline__ void init(const void* matrix, int64_t m, int64_t ld, int64_t rows, uint32_t at, uint32_t stage,
                                       int stages, const Cols& col) {
    row = matrix ? static_cast<const T*>(matrix) + m * ld : nullptr;
    step = rows * ld;
    slot = at + threadIdx.x * kPlace;
    stride = matrix ? stage : 0u;
    for (int s = 0; s < (matrix ? stages : 1); ++s)
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        if (!matrix || !(MODE == kSingle ? col.has(i / G, i % G) : col.whole(i / kChunks)))
          zero_place(slot + s * stride + i * blockDim.x * kPlace);
  }
  __device__ __forceinline__ void copy(int s, const Cols& col) const {
    if constexpr (!kStaged) return;
    if (!row) return;
    const uint32_t to = slot + s * stride, next = blockDim.x * kPlace;
    if constexpr (MODE == kSingle) {
#pragma unroll
      for (int i = 0; i < G * V; ++i)
        if (col.has(i / G, i % G)) copy_place(to + i * next, row + col.at(i / G, i % G));
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (MODE == kAligned ? col.whole(v) : col.at(v, G - 1) < col.end) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) copy_place(to + (v * kChunks + c) * next, row + col.at(v, c * kPer));
        } else if (MODE == kShifted) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int n = min(kPer, col.end - col.at(v, c * kPer));
            if (n > 0) copy_place(to + (v * kChunks + c) * next, row + col.at(v, c * kPer), n * static_cast<int>(sizeof(T)));
          }
        }
      }
    }
  }
  // Unit v of stage s; 0 where there is nothing.
  __device__ __forceinline__ void load(Unit<T, G>& u, int s, int v, const Cols& col) const {
    const uint32_t from = slot + s * stride, next = blockDim.x * kPlace;
    if constexpr (MODE != kSingle) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint32_t p = from + (v * kChunks + c) * next;
        if constexpr (kPlace == 16)
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(u.w[4 * c % u.kWords]), "=r"(u.w[(4 * c + 1) % u.kWords]), "=r"(u.w[(4 * c + 2) % u.kWords]), "=r"(u.w[(4 * c + 3) % u.kWords])
                       : "r"(p) : "memory");
        else
          asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(u.w[0]), "=r"(u.w[1]) : "r"(p) : "memory");
      }
      if (MODE == kShifted && !col.whole(v)) {
#pragma unroll
        for (int j = 0; j < G; ++j) u.keep(j, col.has(v, j));
      }
    } else {
      u.zero();
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if constexpr (kStaged) u.set(j, ld_shared_f32(from + (G * v + j) * next));
        else if (row && col.has(v, j)) u.set(j, row[col.at(v, j)]);
      }
    }
  }
};

// The sum over the threads of a row: LPR lanes of a warp, or (LPR 0) the CTAs of a cluster, of which each warp tells all its
// sum; entries of `red` past the warps are 0.
template <int LPR>
__device__ __forceinline__ float res_sum(float v, float (*red)[32], int& phase, int ranks) {
  if constexpr (LPR > 0) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  } else {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_sum(v);
    float* r = red[phase & 1];
    ++phase;
    if (ranks == 1) {
      if (lane == 0) r[warp] = v;
      __syncthreads();
    } else {
      if (lane < ranks) {
        const uint32_t to = mapa_shared(smem_u32(r + static_cast<int>(cluster_ctarank()) * (32 / ranks) + warp), lane);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(v) : "memory");
      }
      cluster_sync();
    }
    return warp_sum(r[lane]);  // (32 entries, a lane each: the same order in every warp)
  }
}
__device__ __forceinline__ void res_sum_init(float (*red)[32], int ranks) {
  for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i >> 5][i & 31] = 0.0f;
  __syncthreads();
  if (ranks > 1) cluster_sync();
}
__device__ __forceinline__ float root_inverse(float mean_square, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(mean_square + eps));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The form of a row's length: LPR lanes of a warp (0: CTAs), V eights (of two units where G is 4) a thread, `ranks` CTAs a
// row; lpr -1: any length.
struct ResForm {
  int lpr, v, threads, rows, ranks;  // rows a CTA at once
};
inline ResForm res_form(int64_t N, ResMode mode, bool backward) {
  const int64_t eights = (N + (mode == kShifted ? 7 : 0) + 7) / 8;
  if (mode == kSingle && eights <= 64) return {32, eights <= 32 ? 1 : 2, 256, 8, 1};
  if (eights <= 8) return {8, 1, 256, 32, 1};
  if (eights <= 16) return {16, 1, 256, 16, 1};
  if (eights <= 64) return {32, eights <= 32 ? 1 : 2, 256, 8, 1};
  // Rows beyond 8192 values go to clusters of four CTAs of at most 256 threads, two on an SM, whose latencies lie under one
  // another's (4096 x 12288, fp32 stream, forward: 201 us; clusters of two, one CTA on an SM: 208).
  const int ranks = eights <= 2 * kResMaxThreads ? 1 : 4, most = 2 * (ranks == 4 ? 256 : kResMaxThreads);
  const int64_t mine = (eights + ranks - 1) / ranks;
  if (mine > most) return {-1, 1, kResMaxThreads, 1, 1};
  const int v = mine <= kResMaxThreads && !backward && ranks == 1 ? 1 : 2;
  return {0, v, static_cast<int>(((mine + v - 1) / v + 31) / 32 * 32), 1, ranks};
}
// Shared memory of a CTA, where `per_sm` of them are to be resident: `fixed` bytes (weights, zeros) and up to kResMaxStages
// stages of `stage` bytes and of `f` bytes, the latter one less where that lets another stage of the others in: a row that
// is worked on leaves memory idle for its latency unless more than one is on its way.  stages 0: not even one fits (such
// rows are taken as rows of any length).
struct ResShared {
  int64_t bytes;
  int32_t stages, stages_f;
};
inline ResShared res_shared(int64_t stage, int64_t f, int64_t fixed, int per_sm) {
  const int64_t left = 224 * 1024 / per_sm - 1024 - fixed;
  for (int n = kResMaxStages; n > 0; --n)
    for (int k = n; k >= std::max(1, n - 1); --k)
      if (n * stage + k * f <= left) return {n * stage + k * f + fixed, n, k};
  return {0, 0, 0};
}
// bytes of a thread's places of a matrix whose values have `size` bytes
inline int64_t res_thread_bytes(ResMode mode, int v, int64_t size) { return mode == kSingle && size == 2 ? 0 : v * 8 * size; }

// The forward call's form, shared memory and resident CTAs an SM: as many as keep 1024 threads there (two at least, and two
// clusters' CTAs), and fewer where their places do not fit beside one another.  stages 0: rows are taken as of any length.
struct ResPlan {
  ResForm form;
  ResShared shared;
  int per_sm;
};
inline ResPlan res_forward_plan(int64_t N, ResMode mode, int64_t stream_size, int64_t block_size, bool has_f) {
  ResPlan p{res_form(N, mode, false), {0, 0, 0}, 1};
  const ResForm& f = p.form;
  if (f.lpr < 0) return p;
  const int64_t stage = f.threads * res_thread_bytes(mode, f.v, stream_size);
  const int64_t stage_f = has_f ? f.threads * res_thread_bytes(mode, f.v, block_size) : 0;
  const int64_t weights = int64_t{4} * f.threads * f.v * 8 * (has_f ? 2 : 1);
  p.per_sm = f.ranks > 1 ? 2 : std::max(2, 1024 / f.threads);
  while ((p.shared = res_shared(stage, stage_f, weights, p.per_sm)).stages == 0 && p.per_sm > 1) --p.per_sm;
  return p;
}

// Columns a row may have: the kernels count them, and twice as many, in 32 bits.
constexpr int64_t kResMaxCols = int64_t{1} << 29;
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
