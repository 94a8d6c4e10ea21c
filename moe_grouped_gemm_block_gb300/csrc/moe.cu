// moe.cu -- the two ends of a MoE block around its grouped GEMMs: the gate (softmax, top-k, per-expert
// counts and the balance loss, with their gradient) and the combine (the experts' rows back to their tokens, with
// its gradient).

#include <algorithm>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

// ---------------------------------------------------------------- gate
//     p_t = softmax(l_t),  ids_t = the k largest logits (ties: the lowest index),  w_t = p_t[ids_t], over their sum
//     where renormalised;  c_e = how many unmasked (t, j) chose e;  Tv = the unmasked tokens
//     loss = coef E sum_e f_e P_e,   f_e = c_e / (k Tv),   P_e = (1 / Tv) sum over the unmasked t of p_te
//
// A row is held by LPR lanes of a warp, VPL consecutive logits each (a warp works on 32 / LPR rows at once, 32 for 8
// experts), so the whole of it stays in registers.  The k best are taken by merging the lanes' sorted lists: each
// round finds the largest head, whose lane drops it.  The kernel is bound by those instructions, not by memory:
// 65536 x 256 bf16 logits, top-8, 33 MB.
constexpr int kGateThreads = 256;
constexpr int kGateWarps = kGateThreads / 32;
constexpr int kGateMaxExperts = 2048;  // the routed layout's limit
constexpr int kGateMaxTopk = 32;
constexpr int kGateCluster = 8;        // CTAs that add their sums up before they write them
constexpr int kGateMaxClusters = 76;   // partial sums
constexpr int kGateBackwardCtas = 1216;

// The order of the selection as an unsigned integer: ascending in the value, NaN above everything (as a
// descending sort has it), -0 equal to +0 (the addition turns -0 into +0 and every NaN into the positive one).
// 0 is below every value's key: it stands for no logit.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  if constexpr (LPR == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  }
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A sorting network for eight (19 exchanges, descending).
template <typename Exchange>
__device__ __forceinline__ void sort8(Exchange ex) {
  ex(0, 2), ex(1, 3), ex(4, 6), ex(5, 7);
  ex(0, 4), ex(1, 5), ex(2, 6), ex(3, 7);
  ex(0, 1), ex(2, 3), ex(4, 5), ex(6, 7);
  ex(2, 4), ex(3, 5);
  ex(1, 4), ex(3, 6);
  ex(1, 2), ex(3, 4), ex(5, 6);
}

// The lane's logits by rank.  next(): the row's best that is left (its value and index, the same in all the row's
// lanes), taken out of the list of the lane that has it.
//
// More than 256 experts: the lane keeps its largest key and looks for the next one when it is taken.
template <typename TL, int VPL, int LPR>
struct Ranking {
  static_assert(LPR == 32, "rows of a whole warp");
  uint32_t key[VPL];
  uint32_t head;
  int base;
  __device__ __forceinline__ void find() {
    head = 0u;
#pragma unroll
    for (int i = 0; i < VPL; ++i) head = max(head, key[i]);
  }
  __device__ __forceinline__ void init(const float (&f)[VPL], int base_, int E) {
    base = base_;
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = base + i < E ? order_key(f[i]) : 0u;
    find();
  }
  __device__ __forceinline__ void next(float& v, int& id) {
    const uint32_t top = row_max<32>(head);
    const int from = __ffs(__ballot_sync(0xffffffffu, head == top)) - 1;
    int at = 0;
    if ((threadIdx.x & 31) == from) {
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i) at = key[i] == top ? i : at;
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = i == at ? 0u : key[i];
      find();
    }
    id = __shfl_sync(0xffffffffu, base + at, from);
    v = key_value(top);
  }
};

// bf16: the key's 16 bits and the index are one word, unlike any other of the row.
template <int LPR>
struct Ranking<__nv_bfloat16, 8, LPR> {
  uint32_t key[8];
  __device__ __forceinline__ void init(const float (&f)[8], int base, int E) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      key[i] = base + i < E ? (order_key(f[i]) & 0xFFFF0000u) | (0xFFFFu - static_cast<uint32_t>(base + i)) : 0u;
    sort8([&](int a, int b) {
      const uint32_t hi = max(key[a], key[b]), lo = min(key[a], key[b]);
      key[a] = hi;
      key[b] = lo;
    });
  }
  __device__ __forceinline__ void next(float& v, int& id) {
    const uint32_t top = row_max<LPR>(key[0]);
    if (key[0] == top) {
#pragma unroll
      for (int i = 0; i < 7; ++i) key[i] = key[i + 1];
      key[7] = 0u;
    }
    id = static_cast<int>(0xFFFFu - (top & 0xFFFFu));
    v = __uint_as_float(__float_as_uint(key_value(top & 0xFFFF0000u)) & 0xFFFF0000u);
  }
};

// fp32: keys sorted with their places; of equal keys the lower place comes first, of equal heads the lower lane.
template <int LPR>
struct Ranking<float, 8, LPR> {
  uint32_t key[8];
  uint32_t places;  // a hexadecimal digit each, the head's lowest
  int base;
  __device__ __forceinline__ void init(const float (&f)[8], int base_, int E) {
    base = base_;
    uint32_t at[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      key[i] = base + i < E ? order_key(f[i]) : 0u;
      at[i] = i;
    }
    sort8([&](int a, int b) {
      const bool swap = key[a] < key[b] || (key[a] == key[b] && at[a] > at[b]);
      const uint32_t k = key[a], p = at[a];
      key[a] = swap ? key[b] : k;
      key[b] = swap ? k : key[b];
      at[a] = swap ? at[b] : p;
      at[b] = swap ? p : at[b];
    });
    places = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) places |= at[i] << (4 * i);
  }
  __device__ __forceinline__ void next(float& v, int& id) {
    const int lane = threadIdx.x & 31;
    const uint32_t top = row_max<LPR>(key[0]);
    int from = lane;
    if constexpr (LPR > 1) {
      const uint32_t row = (LPR == 32 ? 0xffffffffu : (1u << (LPR & 31)) - 1u) << (lane & ~(LPR - 1) & 31);
      from = __ffs(__ballot_sync(0xffffffffu, key[0] == top) & row) - 1;
    }
    id = base + static_cast<int>(places & 7u);
    if constexpr (LPR > 1) id = __shfl_sync(0xffffffffu, id, from);
    v = key_value(top);
    if (lane == from) {
#pragma unroll
      for (int i = 0; i < 7; ++i) key[i] = key[i + 1];
      key[7] = 0u;
      places >>= 4;
    }
  }
};

// Logits base .. base + VPL - 1 of a row; -inf past its end.  vec: the row's groups of 8 lie on 16-byte boundaries and
// E is a multiple of 8.
template <int VPL, typename TL>
__device__ __forceinline__ void load_logits(const TL* row, int base, int E, bool vec, float (&f)[VPL]) {
#pragma unroll
  for (int v = 0; v < VPL; v += 8) {
    if (vec && base + v < E) {
      float g[8];
      load8(row + base + v, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[v + i] = g[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[v + i] = base + v + i < E ? to_f32(row[base + v + i]) : -INFINITY;
    }
  }
}

struct GateArgs {
  const void* logits;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  float* part_p;    // [clusters][E]
  int32_t* part_c;  // [clusters][E]
  int32_t* counts;
  float* loss;
  int64_t T, ldl;
  int32_t E, topk, renorm, vec;
  float coef;
};

// The balance loss from v = (sum_e c_e sum_t p_te, sum_e c_e).
__device__ __forceinline__ float balance_loss(float cp, float c, int E, int topk, float coef) {
  const float k = static_cast<float>(topk), tv = c / k;
  return tv > 0.0f ? coef * static_cast<float>(E) * (cp / (k * tv * tv)) : 0.0f;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

// Shared memory of the forward kernel: [E] sums of p and [E] counts of the CTA, then per warp its rows' selection
// (ids, exponentials) and factors; the warps' sums of p [WARPS][E] take that room at the end.
template <int LPR>
__host__ __device__ constexpr int gate_warp_words(int topk) { return (32 / LPR) * (2 * topk + 1); }
template <int LPR>
size_t gate_smem(int E, int topk) {
  return 4 * (2 * static_cast<size_t>(E) + std::max(kGateWarps * E, kGateWarps * gate_warp_words<LPR>(topk)));
}

// A warp's rows, and so each partial sum's terms and their order, follow from the grid alone.
template <typename TL, int VPL, int LPR>
__global__ void __launch_bounds__(kGateThreads) moe_gate_kernel(const GateArgs a) {
  constexpr int G = 32 / LPR;  // rows a warp at once
  extern __shared__ float smem[];
  __shared__ float2 s_loss[kGateCluster];
  __shared__ float red[2 * 2 * kGateWarps];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, grp = lane / LPR, base = sub * VPL;
  const int E = a.E, topk = a.topk;
  float* sum_p = smem;
  int32_t* cnt = reinterpret_cast<int32_t*>(smem + E);
  float* rest = smem + 2 * E;
  int32_t* sel_id = reinterpret_cast<int32_t*>(rest + warp * gate_warp_words<LPR>(topk));
  float* sel_e = reinterpret_cast<float*>(sel_id + G * topk);
  float* factor = sel_e + G * topk;
  for (int e = threadIdx.x; e < E; e += kGateThreads) cnt[e] = 0;
  __syncthreads();
  const TL* logits = static_cast<const TL*>(a.logits);
  const float inv_k = 1.0f / static_cast<float>(topk);
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps * G;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGateWarps + warp) * G; t0 < a.T; t0 += stride) {
    const int64_t t = t0 + grp;
    const bool in = t < a.T;
    const bool real = in && (!a.mask || a.mask[t]);
    float f[VPL];
    load_logits(logits + (in ? t : t0) * a.ldl, base, E, a.vec, f);
    Ranking<TL, VPL, LPR> rank;
    rank.init(f, base, E);
    float mx = 0.0f, picked = 0.0f;
    for (int j = 0; j < topk; ++j) {
      float v;
      int id;
      rank.next(v, id);
      if (j == 0) mx = v == -INFINITY ? 0.0f : v;  // every expert ruled out: the exponentials are all 0
      const float e = __expf(v - mx);
      picked += e;
      if (sub == 0) {
        sel_id[grp * topk + j] = id;
        sel_e[grp * topk + j] = e;
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      f[i] = __expf(f[i] - mx);
      s += f[i];
    }
    s = row_sum<LPR>(s);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
    if (real) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(f[i], inv, acc[i]);
    }
    if (sub == 0) factor[grp] = !real ? -1.0f : a.renorm ? (picked == 0.0f ? 0.0f : 1.0f / picked) : inv;
    __syncwarp();
    // the warp's rows are neighbours: their results go out in one piece
    for (int q = lane; q < G * topk; q += 32) {
      const int g = G == 1 ? 0 : static_cast<int>((static_cast<float>(q) + 0.5f) * inv_k);
      if (t0 + g >= a.T) break;
      const int id = sel_id[q];
      const float w = factor[g];
      a.ids[t0 * topk + q] = id;
      a.weights[t0 * topk + q] = w == -1.0f ? 0.0f : sel_e[q] * w;
      if (w != -1.0f) atomicAdd(cnt + id, 1);  // whole numbers: the order does not matter
    }
    __syncwarp();
  }
  // the CTA's sums: over the rows that a warp's lanes shared, then over the warps
#pragma unroll
  for (int i = 0; i < VPL; ++i)
#pragma unroll
    for (int off = 16; off >= LPR; off >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
  __syncthreads();
  if (lane < LPR) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (base + i < E) rest[warp * E + base + i] = acc[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kGateThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kGateWarps; ++w) s += rest[w * E + e];
    sum_p[e] = s;
  }
  // the cluster's: each CTA takes a share of the experts
  const int ranks = static_cast<int>(cluster_size()), me = static_cast<int>(cluster_ctarank());
  const int each = (E + ranks - 1) / ranks, lo = me * each, hi = min(E, lo + each);
  cluster_sync();
  const bool single = static_cast<int>(gridDim.x) == ranks;
  const int64_t part = static_cast<int64_t>(blockIdx.x / ranks) * E;
  float v[2] = {0.0f, 0.0f};
  for (int e = lo + static_cast<int>(threadIdx.x); e < hi; e += kGateThreads) {
    float p = 0.0f;
    int32_t c = 0;
    for (int r = 0; r < ranks; ++r) {
      p += ld_cluster(mapa_shared(smem_u32(sum_p + e), r));
      c += __float_as_int(ld_cluster(mapa_shared(smem_u32(cnt + e), r)));
    }
    if (single) {
      a.counts[e] = c;
      v[0] += static_cast<float>(c) * p;
      v[1] += static_cast<float>(c);
    } else {
      a.part_p[part + e] = p;
      a.part_c[part + e] = c;
    }
  }
  if (single) {
    cta_sum<kGateWarps>(v, red, 0);
    if (threadIdx.x == 0) {
      const uint32_t to = mapa_shared(smem_u32(&s_loss[me]), 0);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(v[0]), "f"(v[1]) : "memory");
    }
  }
  cluster_sync();  // (and nobody leaves while its sums may still be read)
  if (single && me == 0 && threadIdx.x == 0 && a.loss) {
    float cp = 0.0f, c = 0.0f;
    for (int r = 0; r < ranks; ++r) {
      cp += s_loss[r].x;
      c += s_loss[r].y;
    }
    *a.loss = balance_loss(cp, c, E, topk, a.coef);
  }
}

// Counts and loss from the clusters' partial sums, in their order: 32 experts a warp, the warps beside each other
// taking a share of the partial sums.
constexpr int kGateJoinThreads = 1024;
__global__ void __launch_bounds__(kGateJoinThreads) moe_gate_join_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int32_t P, int32_t E, int32_t topk,
    float coef, int32_t* __restrict__ counts, float* __restrict__ loss) {
  constexpr int W = kGateJoinThreads / 32;
  __shared__ float s_p[W][32];
  __shared__ int32_t s_c[W][32];
  __shared__ float red[2 * 2 * W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cols = min(W, (E + 31) / 32), slices = W / cols;  // columns of 32 experts at once, warps for each
  const int col = warp % cols, slice = warp / cols;
  float v[2] = {0.0f, 0.0f};  // sum_e c_e sum_t p_te, sum_e c_e
  griddep_wait();
  for (int e0 = 0; e0 < E; e0 += 32 * cols) {
    const int e = e0 + 32 * col + lane;
    float p = 0.0f;
    int32_t c = 0;
    if (slice < slices && e < E) {
      const int lo = P * slice / slices, hi = P * (slice + 1) / slices;
#pragma unroll 4
      for (int i = lo; i < hi; ++i) {
        p += __ldcg(part_p + static_cast<int64_t>(i) * E + e);
        c += __ldcg(part_c + static_cast<int64_t>(i) * E + e);
      }
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    __syncthreads();
    if (slice == 0 && e < E) {
      for (int i = 1; i < slices; ++i) {
        p += s_p[col + i * cols][lane];
        c += s_c[col + i * cols][lane];
      }
      counts[e] = c;
      v[0] += static_cast<float>(c) * p;
      v[1] += static_cast<float>(c);
    }
    __syncthreads();
  }
  cta_sum<W>(v, red, 0);
  if (threadIdx.x == 0 && loss) *loss = balance_loss(v[0], v[1], E, topk, coef);
}

// dl_te = p_te (G_te - sum_e G_te p_te),  G_te = g_e + sum_j [ids_tj = e] dp_tj,
// g_e = dloss coef E c_e / (k Tv^2),  dp_tj = dw_tj, or (dw_tj - sum_i dw_ti w_ti) / S_t where renormalised
// (S_t = the selected probabilities' sum).  Masked tokens get zeros.  Rows as in the forward kernel; the selected
// experts' dw come to their lanes through a row of shared memory, where this pattern (a NaN that no arithmetic makes)
// marks an expert that was not selected.
constexpr uint32_t kNotSelected = 0xFFFFDEADu;

struct GateGrad {
  const void* logits;
  const uint8_t* mask;
  const int32_t* ids;
  const int32_t* counts;
  const float* dweights;
  const float* dloss;
  void* dlogits;
  int64_t T, ldl, ldd;
  int32_t E, topk, renorm, vec;
  float coef;
};

template <typename TL, int VPL, int LPR>
__global__ void __launch_bounds__(kGateThreads) moe_gate_backward_kernel(const GateGrad a) {
  constexpr int G = 32 / LPR;
  __shared__ float red[2 * kGateWarps];
  extern __shared__ float smem[];  // per warp: G rows of LPR * VPL
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, grp = lane / LPR, base = sub * VPL;
  const int E = a.E, topk = a.topk;
  float* row = smem + warp * (32 * VPL);
  float n[1] = {0.0f};
  for (int e = threadIdx.x; e < E; e += kGateThreads) n[0] += static_cast<float>(a.counts[e]);
  cta_sum<kGateWarps>(n, red, 0);
  const float k = static_cast<float>(topk), tv = n[0] / k, inv_k = 1.0f / k;
  const float scale = a.dloss && tv > 0.0f ? *a.dloss * a.coef * static_cast<float>(E) / (k * tv * tv) : 0.0f;
  float g[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) g[i] = base + i < E ? scale * static_cast<float>(a.counts[base + i]) : 0.0f;
  const TL* logits = static_cast<const TL*>(a.logits);
  TL* dlogits = static_cast<TL*>(a.dlogits);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps * G;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGateWarps + warp) * G; t0 < a.T; t0 += stride) {
    const int64_t t = t0 + grp;
    const bool in = t < a.T;
    const bool real = in && (!a.mask || a.mask[t]);
    float f[VPL], d[VPL];
    load_logits(logits + (in ? t : t0) * a.ldl, base, E, a.vec, f);
    if (a.dweights) {
      uint4* mine = reinterpret_cast<uint4*>(row + lane * VPL);
#pragma unroll
      for (int i = 0; i < VPL / 4; ++i) mine[i] = make_uint4(kNotSelected, kNotSelected, kNotSelected, kNotSelected);
      __syncwarp();
      for (int q = lane; q < G * topk; q += 32) {
        const int r = G == 1 ? 0 : static_cast<int>((static_cast<float>(q) + 0.5f) * inv_k);
        if (t0 + r >= a.T) break;
        const int id = a.ids[t0 * topk + q];
        if (id >= 0 && id < E) row[r * (LPR * VPL) + id] = a.dweights[t0 * topk + q];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < VPL; ++i) d[i] = row[lane * VPL + i];
      __syncwarp();
    }
    float mx = f[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) mx = fmaxf(mx, f[i]);
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (mx == -INFINITY) mx = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      f[i] = __expf(f[i] - mx);
      s += f[i];
    }
    s = row_sum<LPR>(s);
    const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < VPL; ++i) f[i] *= inv;
    float G_[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) G_[i] = g[i];
    if (a.dweights) {
      float total = 0.0f, dot = 0.0f;
      if (a.renorm) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (__float_as_uint(d[i]) != kNotSelected) {
            total += f[i];
            dot = fmaf(d[i], f[i], dot);
          }
        total = row_sum<LPR>(total);
        dot = row_sum<LPR>(dot);
        total = total == 0.0f ? 0.0f : 1.0f / total;
        dot *= total;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (__float_as_uint(d[i]) != kNotSelected) G_[i] += a.renorm ? (d[i] - dot) * total : d[i];
    }
    float inner = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) inner = fmaf(G_[i], f[i], inner);
    inner = row_sum<LPR>(inner);
#pragma unroll
    for (int i = 0; i < VPL; ++i) f[i] = real ? f[i] * (G_[i] - inner) : 0.0f;
    if (!in) continue;
    TL* out = dlogits + t * a.ldd;
#pragma unroll
    for (int v = 0; v < VPL; v += 8) {
      if (a.vec && base + v < E) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f[v + i];
        store8(out + base + v, o);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (base + v + i < E) out[base + v + i] = from_f32<TL>(f[v + i]);
      }
    }
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

// The clusters of a forward call, at most (each writes a row of partial sums).
int64_t gate_clusters(int64_t T) {
  return std::min<int64_t>(kGateMaxClusters, (T + kGateCluster * kGateWarps - 1) / (kGateCluster * kGateWarps));
}

template <typename TL, int VPL, int LPR>
int gate_launch(const GateArgs& a, cudaStream_t s) {
  auto kern = moe_gate_kernel<TL, VPL, LPR>;
  const size_t smem = gate_smem<LPR>(a.E, a.topk);
  int st = allow_smem(kern, smem);
  if (st != FP8G_OK) return st;
  // one CTA for a few rounds of its warps' rows (its latency is below a cluster's), else clusters
  const int64_t at_once = kGateWarps * (32 / LPR);
  const int cluster = a.T <= 2 * at_once ? 1 : kGateCluster;
  const int64_t clusters =
      cluster == 1 ? 1 : std::min<int64_t>(kGateMaxClusters, (a.T + cluster * at_once - 1) / (cluster * at_once));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster));
  cfg.blockDim = dim3(kGateThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  if (clusters == 1) return FP8G_OK;  // the cluster has finished the counts and the loss itself
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kGateJoinThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  if (cudaLaunchKernelEx(&cfg, moe_gate_join_kernel, static_cast<const float*>(a.part_p),
                         static_cast<const int32_t*>(a.part_c), static_cast<int32_t>(clusters), a.E, a.topk, a.coef,
                         a.counts, a.loss) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

template <typename TL, int VPL, int LPR>
int gate_backward_launch(const GateGrad& a, cudaStream_t s) {
  auto kern = moe_gate_backward_kernel<TL, VPL, LPR>;
  const size_t smem = static_cast<size_t>(kGateWarps) * 32 * VPL * 4;
  int st = allow_smem(kern, smem);
  if (st != FP8G_OK) return st;
  const int64_t at_once = kGateWarps * (32 / LPR);
  const int64_t ctas = std::min<int64_t>((a.T + at_once - 1) / at_once, kGateBackwardCtas);
  kern<<<static_cast<unsigned>(ctas), kGateThreads, smem, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

// A row's lanes: as many as hold it at 8 logits each, beyond 256 experts all 32 with more.
template <typename TL>
auto gate_form(int E) {
  return E <= 8     ? gate_launch<TL, 8, 1>
         : E <= 16  ? gate_launch<TL, 8, 2>
         : E <= 32  ? gate_launch<TL, 8, 4>
         : E <= 64  ? gate_launch<TL, 8, 8>
         : E <= 128 ? gate_launch<TL, 8, 16>
         : E <= 256 ? gate_launch<TL, 8, 32>
         : E <= 512 ? gate_launch<TL, 16, 32>
                    : gate_launch<TL, 64, 32>;
}
template <typename TL>
auto gate_backward_form(int E) {
  return E <= 8     ? gate_backward_launch<TL, 8, 1>
         : E <= 16  ? gate_backward_launch<TL, 8, 2>
         : E <= 32  ? gate_backward_launch<TL, 8, 4>
         : E <= 64  ? gate_backward_launch<TL, 8, 8>
         : E <= 128 ? gate_backward_launch<TL, 8, 16>
         : E <= 256 ? gate_backward_launch<TL, 8, 32>
         : E <= 512 ? gate_backward_launch<TL, 16, 32>
                    : gate_backward_launch<TL, 64, 32>;
}
// Whether rows of E logits can be taken eight at a time.
bool logit_vectors(const void* p, int64_t ld, int32_t E, int32_t dtype) {
  return E % 8 == 0 && aligned16(p) && (ld * static_cast<int64_t>(dtype_size(dtype))) % 16 == 0;
}

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_moe_gate_workspace(int64_t T, int32_t E, int64_t* bytes) {
  if (T < 0 || T > 0x7FFFFFFF || E < 1 || E > kGateMaxExperts || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = gate_clusters(T) * E * 8;
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
  if (T > 0 && (!workspace || workspace_bytes < gate_clusters(T) * E * 8)) return FP8G_ERR_INVALID_ARG;
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
  GateArgs a{};
  a.logits = logits, a.mask = token_mask, a.ids = topk_ids, a.weights = topk_weights, a.counts = counts, a.loss = loss;
  a.part_p = static_cast<float*>(workspace);
  a.part_c = reinterpret_cast<int32_t*>(a.part_p + gate_clusters(T) * E);
  a.T = T, a.ldl = ldl, a.E = E, a.topk = topk, a.renorm = renormalize, a.coef = loss_coef;
  a.vec = logit_vectors(logits, ldl, E, dtype);
  return (dtype == FP8G_F32 ? gate_form<float>(E) : gate_form<__nv_bfloat16>(E))(a, s);
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
  GateGrad a{};
  a.logits = logits, a.mask = token_mask, a.ids = topk_ids, a.counts = counts, a.dweights = dweights, a.dloss = dloss;
  a.dlogits = dlogits, a.T = T, a.ldl = ldl, a.ldd = ldd;
  a.E = E, a.topk = topk, a.renorm = renormalize, a.coef = loss_coef;
  a.vec = logit_vectors(logits, ldl, E, dtype) && logit_vectors(dlogits, ldd, E, dtype);
  return (dtype == FP8G_F32 ? gate_backward_form<float>(E) : gate_backward_form<__nv_bfloat16>(E))(
      a, static_cast<cudaStream_t>(stream));
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
