// moe.cu -- the two ends of a MoE block around its grouped GEMMs: the gate (softmax, top-k, per-expert
// counts and the balance loss, with their gradient) and the combine (the experts' rows back to their tokens, with
// its gradient).

#include <algorithm>
#include <cuda_runtime.h>
#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"
#include "topk.cuh"
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
// round finds the largest head, whose lane goes on to its next one.
//
// The kernels are bound by their instructions, not by memory: 362 of a warp for a bf16 row of 256 with 8 picks, most
// of them on the ALU, which takes one every second cycle (the sort's minima and maxima, the keys, the picks).
// 65536 x 256, 8 picks: forward bf16 38 us, fp32 47 (15% and 22% of the copy rate), of which the joined sums take 5;
// backward bf16 26 us (40%).  Few tokens (64 x 32): 7 us, a launch.
constexpr int kGateThreads = 256;
constexpr int kGateWarps = kGateThreads / 32;
constexpr int kGateMaxExperts = 2048;  // the routed layout's limit
constexpr int kGateMaxTopk = 32;
constexpr int kGateCluster = 8;        // CTAs of a small call, which finish it together
constexpr int kGateMaxParts = 608;     // CTAs, and partial sums, of a larger one

// Four sums at once: each half of the row's lanes goes on with two of them, each quarter with one (10 shuffles of a
// whole warp's row instead of 20).
template <int LPR>
__device__ __forceinline__ float4 row_sum4(float a, float b, float c, float d) {
  if constexpr (LPR < 8) {
    return make_float4(row_sum<LPR>(a), row_sum<LPR>(b), row_sum<LPR>(c), row_sum<LPR>(d));
  } else {
    const int lane = threadIdx.x & 31;
    const bool half = lane & (LPR / 2), quarter = lane & (LPR / 4);
    float v = (half ? c : a) + __shfl_xor_sync(0xffffffffu, half ? a : c, LPR / 2);
    const float w = (half ? d : b) + __shfl_xor_sync(0xffffffffu, half ? b : d, LPR / 2);
    v = (quarter ? w : v) + __shfl_xor_sync(0xffffffffu, quarter ? v : w, LPR / 4);
    v = row_sum<LPR / 4>(v);
    return make_float4(__shfl_sync(0xffffffffu, v, 0, LPR), __shfl_sync(0xffffffffu, v, LPR / 4, LPR),
                       __shfl_sync(0xffffffffu, v, LPR / 2, LPR), __shfl_sync(0xffffffffu, v, 3 * LPR / 4, LPR));
  }
}

// The lane's logits by rank.  next(): the row's best that is left (the same in all the row's lanes), taken out of the
// list of the lane that has it; value() and id() of what next() gave.  `list`: kListWords words of shared memory of
// the lane's own, of which words 8 and 9 are 0.
//
// The general form, beyond 256 experts: the lane keeps its largest key and looks for the next one when it is taken.
struct Pick {
  uint32_t key;
  int id;
};
constexpr int kListWords = 12;  // eight keys, two for the end; lanes 12 words apart write 16 bytes without conflicts
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
  __device__ __forceinline__ void init(const Logits<TL, VPL>& l, int base_, int E, uint32_t*) {
    base = base_;
    float2 f[VPL / 2];
    l.get(f);
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = base + i < E ? order_key(i & 1 ? f[i / 2].y : f[i / 2].x) : 0u;
    find();
  }
  __device__ __forceinline__ Pick next() {
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
    return {top, __shfl_sync(0xffffffffu, base + at, from)};
  }
  static __device__ __forceinline__ float value(const Pick& p) { return key_value(p.key); }
  static __device__ __forceinline__ int id(const Pick& p) { return p.id; }
};

// bf16: the key's 16 bits and the index are one word, unlike any other of the row.  The sorted list lies in shared
// memory, its next two in registers (a round need not wait for the load of the one before).
template <int LPR>
struct Ranking<__nv_bfloat16, 8, LPR> {
  uint32_t head, second;
  const uint32_t* at;
  __device__ __forceinline__ void init(const Logits<__nv_bfloat16, 8>& l, int base, int E, uint32_t* list) {
    const uint32_t w[4] = {l.raw[0].v.x, l.raw[0].v.y, l.raw[0].v.z, l.raw[0].v.w};
    uint32_t key[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t k = order_key2(w[i]), c = 0xFFFFu - static_cast<uint32_t>(base + 2 * i);
      key[2 * i] = __byte_perm(k, c, 0x1054);          // the low key over the place
      key[2 * i + 1] = __byte_perm(k, c - 1u, 0x3254);  // the high one
    }
    if (base + 8 > E) {
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = base + i < E ? key[i] : 0u;
    }
    sort8([&](int a, int b) {
      const uint32_t hi = max(key[a], key[b]), lo = min(key[a], key[b]);
      key[a] = hi;
      key[b] = lo;
    });
    head = key[0];
    second = key[1];
    at = list + 1;
    reinterpret_cast<uint4*>(list)[0] = make_uint4(key[0], key[1], key[2], key[3]);
    reinterpret_cast<uint4*>(list)[1] = make_uint4(key[4], key[5], key[6], key[7]);
  }
  __device__ __forceinline__ Pick next() {
    const uint32_t top = row_max<LPR>(head);
    if (head == top) {
      head = second;
      second = *++at;
    }
    return {top, 0};
  }
  __device__ __forceinline__ void next(uint32_t* to) {  // which the lane that has it writes
    const uint32_t top = row_max<LPR>(head);
    if (head == top) {
      *to = top;
      head = second;
      second = *++at;
    }
  }
  static __device__ __forceinline__ float value(const Pick& p) {
    return __uint_as_float(__float_as_uint(key_value(p.key & 0xFFFF0000u)) & 0xFFFF0000u);
  }
  static __device__ __forceinline__ int id(const Pick& p) { return static_cast<int>(0xFFFFu - (p.key & 0xFFFFu)); }
};

// fp32: keys sorted with their places; of equal keys the lower place comes first, of equal heads the lower lane.
template <int LPR>
struct Ranking<float, 8, LPR> {
  uint32_t head, second;
  uint32_t places;  // a hexadecimal digit each, the head's lowest
  const uint32_t* at;
  int base;
  __device__ __forceinline__ void init(const Logits<float, 8>& l, int base_, int E, uint32_t* list) {
    base = base_;
    float2 f[4];
    l.get(f);
    uint32_t key[8], place[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      key[i] = order_key(i & 1 ? f[i / 2].y : f[i / 2].x);
      place[i] = i;
    }
    if (base + 8 > E) {
#pragma unroll
      for (int i = 0; i < 8; ++i) key[i] = base + i < E ? key[i] : 0u;
    }
    sort8([&](int a, int b) {
      const bool swap = key[a] < key[b] || (key[a] == key[b] && place[a] > place[b]);
      const uint32_t k = key[a], p = place[a];
      key[a] = swap ? key[b] : k;
      key[b] = swap ? k : key[b];
      place[a] = swap ? place[b] : p;
      place[b] = swap ? p : place[b];
    });
    places = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) places |= place[i] << (4 * i);
    head = key[0];
    second = key[1];
    at = list + 1;
    reinterpret_cast<uint4*>(list)[0] = make_uint4(key[0], key[1], key[2], key[3]);
    reinterpret_cast<uint4*>(list)[1] = make_uint4(key[4], key[5], key[6], key[7]);
  }
  __device__ __forceinline__ Pick next() {
    const int lane = threadIdx.x & 31;
    const uint32_t top = row_max<LPR>(head);
    int from = lane, id = base + static_cast<int>(places & 7u);
    if constexpr (LPR > 1) {
      const uint32_t row = (LPR == 32 ? 0xffffffffu : (1u << (LPR & 31)) - 1u) << (lane & ~(LPR - 1) & 31);
      from = __ffs(__ballot_sync(0xffffffffu, head == top) & row) - 1;
      id = __shfl_sync(0xffffffffu, id, from);
    }
    if (lane == from) {
      head = second;
      second = *++at;
      places >>= 4;
    }
    return {top, id};
  }
  static __device__ __forceinline__ float value(const Pick& p) { return key_value(p.key); }
  static __device__ __forceinline__ int id(const Pick& p) { return p.id; }
};

struct GateArgs {
  const void* logits;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  float* part_p;    // [CTAs][E]
  int32_t* part_c;  // [CTAs][E]
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

// Shared memory of the forward kernel: [E] sums of p and [E] counts of the CTA, then per warp the lanes' lists and its
// rows' picks (keys, ids, weights) and factors; the warps' sums of p [WARPS][E] take that room at the end.
template <int LPR>
__host__ __device__ constexpr int gate_warp_words(int topk) {
  return 32 * kListWords + ((32 / LPR) * (3 * topk + 1) + 3) / 4 * 4;
}
template <int LPR>
size_t gate_smem(int E, int topk, int warps) {
  return 4 * (2 * static_cast<size_t>((E + 3) / 4 * 4) + warps * std::max(E, gate_warp_words<LPR>(topk)));
}

// CTAs that are resident on an SM at once.
__host__ __device__ constexpr int gate_per_sm(int vpl) { return vpl == 8 ? 4 : vpl == 16 ? 2 : 1; }

// A warp's rows, and so each partial sum's terms and their order, follow from the grid alone.
template <typename TL, int VPL, int LPR, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, gate_per_sm(VPL) * kGateWarps / WARPS)
    moe_gate_kernel(const GateArgs a) {
  constexpr int kThreads = 32 * WARPS;
  constexpr int G = 32 / LPR;  // rows a warp at once
  using Rank = Ranking<TL, VPL, LPR>;
  constexpr bool kOneWord = std::is_same_v<TL, __nv_bfloat16> && VPL == 8;  // a pick's key holds its index
  extern __shared__ __align__(16) float smem[];
  __shared__ float2 s_loss[kGateCluster];
  __shared__ float red[2 * 2 * WARPS];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, grp = lane / LPR, base = sub * VPL;
  const int E = a.E, topk = a.topk, padded = (E + 3) / 4 * 4;
  float* sum_p = smem;
  int32_t* cnt = reinterpret_cast<int32_t*>(smem + padded);
  float* rest = smem + 2 * padded;
  uint32_t* list = reinterpret_cast<uint32_t*>(rest) + warp * gate_warp_words<LPR>(topk) + lane * kListWords;
  uint32_t* pick_key = reinterpret_cast<uint32_t*>(rest) + warp * gate_warp_words<LPR>(topk) + 32 * kListWords;
  int32_t* pick_id = reinterpret_cast<int32_t*>(pick_key + G * topk);
  float* pick_w = reinterpret_cast<float*>(pick_id + G * topk);
  float* factor = pick_w + G * topk;
  list[8] = list[9] = 0u;  // the end of every list
  for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  const TL* logits = static_cast<const TL*>(a.logits);
  const float inv_k = 1.0f / static_cast<float>(topk);
  float2 acc[VPL / 2];
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * WARPS * G;
  int64_t t0 = (static_cast<int64_t>(blockIdx.x) * WARPS + warp) * G;
  Logits<TL, VPL> next;
  bool next_real = false;
  auto fetch = [&](int64_t at) {
    const int64_t t = at + grp < a.T ? at + grp : a.T - 1;
    next_real = at + grp < a.T && (!a.mask || a.mask[t]);
    next.load(logits + t * a.ldl, base, E, a.vec);
  };
  if (t0 < a.T) fetch(t0);
  for (; t0 < a.T; t0 += stride) {
    Logits<TL, VPL> l = next;
    const bool real = next_real;
    if (t0 + stride < a.T) fetch(t0 + stride);
    Rank rank;
    rank.init(l, base, E, list);
    // the row's picks go to a lane each (of a whole warp's row), or through shared memory to the row's lanes in turn
    Pick mine = rank.next();
    float mx = Rank::value(mine);
    if (mx == -INFINITY) mx = 0.0f;  // every expert ruled out: the exponentials are all 0
    if constexpr (G == 1 && kOneWord) {
      if (lane == 0) pick_key[0] = mine.key;
#pragma unroll 2
      for (int j = 1; j < topk; ++j) rank.next(pick_key + j);
      __syncwarp();
      if (lane < topk) mine.key = pick_key[lane];
      __syncwarp();
    } else if constexpr (G == 1) {
#pragma unroll 2
      for (int j = 1; j < topk; ++j) {
        const Pick p = rank.next();
        if (lane == j) mine = p;
      }
    } else {
      for (int j = 0;;) {
        if (sub == 0) {
          pick_key[grp * topk + j] = mine.key;
          if constexpr (!kOneWord) pick_id[grp * topk + j] = mine.id;
        }
        if (++j == topk) break;
        mine = rank.next();
      }
      __syncwarp();
    }
    float picked = 0.0f;
    if constexpr (G == 1) {
      if (lane < topk) picked = exp_below(Rank::value(mine), mx);
    } else {
      for (int j = sub; j < topk; j += LPR) {
        const Pick p{pick_key[grp * topk + j], 0};
        const float e = exp_below(Rank::value(p), mx);
        picked += e;
        if constexpr (kOneWord) pick_id[grp * topk + j] = Rank::id(p);
        pick_w[grp * topk + j] = e;
      }
    }
    const float own = picked;
    picked = row_sum<LPR>(picked);
    float2 f[VPL / 2];
    l.get(f);
    const float s = row_sum<LPR>(exp_below(f, mx));
    const float inv = s == 0.0f ? 0.0f : recip_approx(s);
    if (real) {
#pragma unroll
      for (int i = 0; i < VPL / 2; ++i) acc[i] = __ffma2_rn(f[i], make_float2(inv, inv), acc[i]);
    }
    const float scale = a.renorm ? (picked == 0.0f ? 0.0f : recip_approx(picked)) : inv;
    if constexpr (G == 1) {
      if (lane < topk) {
        const int id = Rank::id(mine);
        a.ids[t0 * topk + lane] = id;
        a.weights[t0 * topk + lane] = real ? own * scale : 0.0f;
        if (real) atomicAdd(cnt + id, 1);  // whole numbers: the order does not matter
      }
    } else {
      if (sub == 0) factor[grp] = real ? scale : -1.0f;
      __syncwarp();
      // the warp's rows are neighbours: their results go out in one piece
      for (int q = lane; q < G * topk; q += 32) {
        const int g = static_cast<int>((static_cast<float>(q) + 0.5f) * inv_k);
        if (t0 + g >= a.T) break;
        const int id = pick_id[q];
        const float w = factor[g];
        a.ids[t0 * topk + q] = id;
        a.weights[t0 * topk + q] = w == -1.0f ? 0.0f : pick_w[q] * w;
        if (w != -1.0f) atomicAdd(cnt + id, 1);
      }
      __syncwarp();
    }
  }
  // the CTA's sums: over the rows that a warp's lanes shared, then over the warps
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i)
#pragma unroll
    for (int off = 16; off >= LPR; off >>= 1) {
      acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, off);
      acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, off);
    }
  __syncthreads();
  if (lane < LPR) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (base + i < E) rest[warp * E + base + i] = i & 1 ? acc[i / 2].y : acc[i / 2].x;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) s += rest[w * E + e];
    sum_p[e] = s;
  }
  // a cluster's: each CTA takes a share of the experts
  const int ranks = static_cast<int>(cluster_size()), me = static_cast<int>(cluster_ctarank());
  const int each = (E + ranks - 1) / ranks, lo = me * each, hi = min(E, lo + each);
  cluster_sync();
  const bool single = static_cast<int>(gridDim.x) == ranks;
  const int64_t part = static_cast<int64_t>(blockIdx.x / ranks) * E;
  float v[2] = {0.0f, 0.0f};
  for (int e = lo + static_cast<int>(threadIdx.x); e < hi; e += kThreads) {
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
    cta_sum<WARPS>(v, red, 0);
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

// Counts and loss from the CTAs' partial sums, in their order.  One cluster; a CTA takes 32 experts at a time, its
// warps a share of the partial sums each.
constexpr int kGateJoinThreads = 1024;
__global__ void __launch_bounds__(kGateJoinThreads) moe_gate_join_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int32_t P, int32_t E, int32_t topk,
    float coef, int32_t* __restrict__ counts, float* __restrict__ loss) {
  constexpr int W = kGateJoinThreads / 32;
  constexpr int kLoads = 10;  // a warp's share, 19 rows at most, in two trips to L2
  __shared__ float s_p[W][32];
  __shared__ int32_t s_c[W][32];
  __shared__ float2 s_loss[kGateCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ranks = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
  float v[2] = {0.0f, 0.0f};  // warp 0: sum_e c_e sum_t p_te, sum_e c_e
  cluster_sync();             // every CTA runs before it is written to
  griddep_wait();
  for (int e0 = 32 * me; e0 < E; e0 += 32 * ranks) {
    const int e = e0 + lane;
    float p = 0.0f;
    int32_t c = 0;
    if (e < E) {
      const int lo = P * warp / W, hi = P * (warp + 1) / W;
      for (int i0 = lo; i0 < hi; i0 += kLoads) {
        float pi[kLoads];
        int32_t ci[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          pi[i] = i0 + i < hi ? __ldcg(part_p + static_cast<int64_t>(i0 + i) * E + e) : 0.0f;
          ci[i] = i0 + i < hi ? __ldcg(part_c + static_cast<int64_t>(i0 + i) * E + e) : 0;
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          p += pi[i];
          c += ci[i];
        }
      }
    }
    s_p[warp][lane] = p;
    s_c[warp][lane] = c;
    __syncthreads();
    if (warp == 0 && e < E) {
#pragma unroll
      for (int i = 1; i < W; ++i) {
        p += s_p[i][lane];
        c += s_c[i][lane];
      }
      counts[e] = c;
      v[0] += static_cast<float>(c) * p;
      v[1] += static_cast<float>(c);
    }
    __syncthreads();
  }
  if (warp == 0) {
    const float cp = warp_sum(v[0]), c = warp_sum(v[1]);
    if (lane == 0)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(smem_u32(&s_loss[me]), 0)), "f"(cp),
                   "f"(c)
                   : "memory");
  }
  cluster_sync();
  if (me == 0 && threadIdx.x == 0 && loss) {
    float cp = 0.0f, c = 0.0f;
    for (int r = 0; r < ranks; ++r) {
      cp += s_loss[r].x;
      c += s_loss[r].y;
    }
    *loss = balance_loss(cp, c, E, topk, coef);
  }
}

// dl_te = p_te (G_te - sum_e G_te p_te),  G_te = g_e + sum_j [ids_tj = e] dp_tj,
// g_e = dloss coef E c_e / (k Tv^2),  dp_tj = dw_tj, or (dw_tj - sum_i dw_ti w_ti) / S_t where renormalised
// (S_t = the selected probabilities' sum).  Masked tokens get zeros.  Rows as in the forward kernel.  Every lane writes
// p (g - inner product) for its logits; the selected experts' values, a few a row, are worked out by a lane each (it
// reads their logits again) and written over them.
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

// CTAs that are resident on an SM at once: all that are launched (65536 x 64 fp32: 12.4 us, with 4 an SM 14.4).
__host__ __device__ constexpr int gate_grad_per_sm(int vpl, int lpr) {
  return vpl == 64 ? 1 : vpl == 16 || (lpr > 1 && lpr < 16) ? 3 : 4;
}
template <typename TL, int VPL, int LPR>
__global__ void __launch_bounds__(kGateThreads, gate_grad_per_sm(VPL, LPR))
    moe_gate_backward_kernel(const GateGrad a) {
  constexpr int G = 32 / LPR;
  // a lane's selected experts, at most
  constexpr int kPicks = LPR >= kGateMaxTopk ? 1 : LPR * 8 >= kGateMaxTopk ? kGateMaxTopk / LPR : 8;
  __shared__ float red[2 * kGateWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, grp = lane / LPR, base = sub * VPL;
  const int E = a.E, topk = a.topk;
  float n[1] = {0.0f};
  for (int e = threadIdx.x; e < E; e += kGateThreads) n[0] += static_cast<float>(a.counts[e]);
  cta_sum<kGateWarps>(n, red, 0);
  const float k = static_cast<float>(topk), tv = n[0] / k;
  const float scale = a.dloss && tv > 0.0f ? *a.dloss * a.coef * static_cast<float>(E) / (k * tv * tv) : 0.0f;
  float2 g[VPL / 2];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    (i & 1 ? g[i / 2].y : g[i / 2].x) = base + i < E ? scale * static_cast<float>(a.counts[base + i]) : 0.0f;
  const TL* logits = static_cast<const TL*>(a.logits);
  TL* dlogits = static_cast<TL*>(a.dlogits);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateWarps * G;
  // the next row's logits and this lane's (first) selected expert and gradient are on their way meanwhile
  Logits<TL, VPL> next;
  bool next_real = false;
  int next_id = -1;
  float next_dw = 0.0f;
  auto fetch = [&](int64_t t) {  // t < a.T, or a row past the end, of which nothing is used
    const int64_t r = min(t, a.T - 1);
    next_real = t < a.T && (!a.mask || a.mask[r]);
    next.load(logits + r * a.ldl, base, E, a.vec);
    if (a.dweights && sub < topk) {
      next_id = a.ids[r * topk + sub];
      next_dw = a.dweights[r * topk + sub];
    }
  };
  int64_t t = (static_cast<int64_t>(blockIdx.x) * kGateWarps + warp) * G + grp;
  if (t - grp < a.T) fetch(t);
  for (; t - grp < a.T; t += stride) {
    const Logits<TL, VPL> l = next;
    const bool real = next_real;
    const int id0 = next_id;
    const float dw0 = next_dw;
    if (t - grp + stride < a.T) fetch(t + stride);
    const TL* row = logits + min(t, a.T - 1) * a.ldl;
    // the lane's selected experts, the row's sub, sub + LPR, ...: their logits, or id -1 for none
    int id[kPicks];
    float dw[kPicks], e[kPicks];
#pragma unroll
    for (int j = 0; j < kPicks; ++j) {
      const int q = j * LPR + sub;
      id[j] = -1;
      dw[j] = 0.0f;
      e[j] = -INFINITY;
      if (a.dweights && q < topk) {
        id[j] = j == 0 ? id0 : a.ids[min(t, a.T - 1) * topk + q];
        dw[j] = j == 0 ? dw0 : a.dweights[min(t, a.T - 1) * topk + q];
        if (id[j] >= 0 && id[j] < E) e[j] = to_f32(row[id[j]]);
        else id[j] = -1;
      }
    }
    float2 f[VPL / 2];
    l.get(f);
    float mx = fmaxf(f[0].x, f[0].y);
#pragma unroll
    for (int i = 1; i < VPL / 2; ++i) mx = fmaxf(mx, fmaxf(f[i].x, f[i].y));
    mx = row_max<LPR>(mx);
    if (mx == -INFINITY) mx = 0.0f;
    // sums over the exponentials f = s p: all of them, with g, the selected ones, and with their dw
    const float own_s = exp_below(f, mx);
    float2 own_g = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) own_g = __ffma2_rn(g[i], f[i], own_g);
    float sel = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < kPicks; ++j) {
      if (j * LPR >= topk) break;
      e[j] = exp_below(e[j], mx);
      sel += e[j];
      if (id[j] >= 0) dot = fmaf(dw[j], e[j], dot);
    }
    const float4 sums = row_sum4<LPR>(own_s, own_g.x + own_g.y, sel, dot);
    const float s = sums.x, sum_g = sums.y;
    sel = sums.z;
    dot = sums.w;
    const float inv = !real || s == 0.0f ? 0.0f : recip_approx(s);
    const float inv_sel = sel == 0.0f ? 0.0f : recip_approx(sel);
    // renormalised, the weights' gradient has no component along the weights: the inner product is g's alone
    const float inner = inv * (a.renorm ? sum_g : sum_g + dot);
    const float per = a.renorm ? s * inv_sel : 1.0f;         // 1 / S_t
    const float mean = a.renorm ? dot * inv_sel : 0.0f;      // sum_i dw_i w_i
    TL* out = dlogits + t * a.ldd;
    if (t < a.T) {
#pragma unroll
      for (int i = 0; i < VPL / 2; ++i) {
        const float2 p = __fmul2_rn(f[i], make_float2(inv, inv));
        f[i] = real ? __fmul2_rn(p, __fadd2_rn(g[i], make_float2(-inner, -inner))) : make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int v = 0; v < VPL; v += 8) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = i & 1 ? f[(v + i) / 2].y : f[(v + i) / 2].x;
        if (a.vec && base + v + 8 <= E) {
          store8(out + base + v, o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (base + v + i < E) out[base + v + i] = from_f32<TL>(o[i]);
        }
      }
    }
    if (!a.dweights) continue;
    __syncwarp();  // over what the row's lanes have written
#pragma unroll
    for (int j = 0; j < kPicks; ++j) {
      if (j * LPR >= topk) break;
      if (real && id[j] >= 0) {
        const float own = fmaf(per, dw[j] - mean, scale * static_cast<float>(a.counts[id[j]]));
        out[id[j]] = from_f32<TL>(e[j] * inv * (own - inner));
      }
    }
  }
}

// ---------------------------------------------------------------- combine
//     out_t = residual_t + sum_j w_tj D[row_tj]
// Both directions are bound by memory: 16-byte loads, the rows of several entries in flight per thread.  4096 tokens
// of 2 x 4096, fp32 with a residual: 35 us (85% of the copy rate); 8192 of 8 x 2048, bf16: 56 us (88%); backward
// 4001 of 4 x 7168: 91 us (92%), 8192 of 8 x 2048: 101 us (93%).
constexpr int kCombineThreads = 128;
constexpr int kCombineSpan = kCombineThreads * 8;  // columns a CTA takes at once

// The row of an entry, or -1 where it is dropped or out of range (the latter is flagged).
__device__ __forceinline__ int32_t entry(const int32_t* __restrict__ entry_row, int64_t i, int64_t M,
                                         unsigned int* status) {
  const int32_t r = __ldg(entry_row + i);
  if (r >= M) {
    record_status(status, FP8G_ERR_DEVICE_ASSERT);
    return -1;
  }
  return r;
}

// A CTA (blockIdx.x, blockIdx.y) takes token blockIdx.x and every gridDim.y-th span of columns; JN entries' rows are in
// flight at once.
template <typename TO, int JN>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(
    const __nv_bfloat16* __restrict__ D, int64_t M, int32_t N, int64_t ldd, const int32_t* __restrict__ entry_row,
    int32_t topk, const float* __restrict__ weights, const TO* residual, int64_t ldr, TO* out, int64_t ldo,
    unsigned int* status) {
  const int64_t t = blockIdx.x;
  for (int64_t n = static_cast<int64_t>(blockIdx.y) * kCombineSpan + threadIdx.x * 8; n < N;
       n += static_cast<int64_t>(gridDim.y) * kCombineSpan) {
    Raw8<TO> res;
    if (residual) res.load_stream(residual + t * ldr + n);
    float acc[8] = {};
    for (int j0 = 0; j0 < topk; j0 += JN) {
      uint4 raw[JN];
      float w[JN];
      int32_t r[JN];
#pragma unroll
      for (int u = 0; u < JN; ++u) {
        r[u] = j0 + u < topk ? entry(entry_row, t * topk + j0 + u, M, status) : -1;
        w[u] = r[u] >= 0 && weights ? __ldg(weights + t * topk + j0 + u) : 1.0f;
      }
#pragma unroll
      for (int u = 0; u < JN; ++u)
        if (r[u] >= 0) raw[u] = __ldg(reinterpret_cast<const uint4*>(D + static_cast<int64_t>(r[u]) * ldd + n));
#pragma unroll
      for (int u = 0; u < JN; ++u) {
        if (r[u] < 0) continue;
        const uint32_t q[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] = fmaf(w[u], __uint_as_float(q[i] << 16), acc[2 * i]);
          acc[2 * i + 1] = fmaf(w[u], __uint_as_float(q[i] & 0xFFFF0000u), acc[2 * i + 1]);
        }
      }
    }
    if (residual) {
      float2 f[4];
      res.get(f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += f[i].x;
        acc[2 * i + 1] += f[i].y;
      }
    }
    store8_stream(out + t * ldo + n, acc);
  }
}

// dD[row_tj] = w_tj dout_t,  dw_tj = <dout_t, D[row_tj]>; rows without a token are zero.  The first `zero_ctas` CTAs
// write those: a warp looks at 32 rows at a time, far apart so that the runs of padding rows spread over the warps.
// Each of the others takes a token, JN of its entries at a time: its dout is read once for them.
template <typename TO, int JN, int THREADS>
__global__ void __launch_bounds__(THREADS) moe_combine_backward_kernel(
    const TO* __restrict__ dout, int64_t lddo, const __nv_bfloat16* __restrict__ D, int64_t M, int32_t N, int64_t ldd,
    const int32_t* __restrict__ entry_row, const int32_t* __restrict__ row_token, int32_t zero_ctas, int32_t topk,
    const float* __restrict__ weights, __nv_bfloat16* __restrict__ dD, int64_t lddd, float* __restrict__ dweights,
    unsigned int* status) {
  constexpr int kWarps = THREADS / 32;
  __shared__ float red[2 * kWarps * JN];
  if (static_cast<int>(blockIdx.x) < zero_ctas) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(zero_ctas) * kWarps;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32; r0 < M; r0 += 32 * warps) {
      const int64_t r = r0 + lane * warps;
      unsigned empty = __ballot_sync(0xffffffffu, r < M && __ldg(row_token + r) < 0);
      for (; empty; empty &= empty - 1) {
        __nv_bfloat16* p = dD + (r0 + (__ffs(empty) - 1) * warps) * lddd;
        for (int64_t n = lane * 8; n < N; n += 256) __stcs(reinterpret_cast<uint4*>(p + n), make_uint4(0u, 0u, 0u, 0u));
      }
    }
    return;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) - zero_ctas;
  int phase = 0;
  for (int j0 = 0; j0 < topk; j0 += JN) {
    int32_t r[JN];
    float w[JN], dot[JN];
#pragma unroll
    for (int j = 0; j < JN; ++j) {
      r[j] = j0 + j < topk ? entry(entry_row, t * topk + j0 + j, M, status) : -1;
      w[j] = r[j] >= 0 && weights ? __ldg(weights + t * topk + j0 + j) : 1.0f;
      dot[j] = 0.0f;
    }
    for (int64_t n = threadIdx.x * 8; n < N; n += THREADS * 8) {
      Raw8<TO> graw;
      Raw8<__nv_bfloat16> d[JN];
      graw.load(dout + t * lddo + n);
      if (dweights) {
#pragma unroll
        for (int j = 0; j < JN; ++j)
          if (r[j] >= 0) d[j].load_stream(D + static_cast<int64_t>(r[j]) * ldd + n);
      }
      float2 g[4];
      graw.get(g);
#pragma unroll
      for (int j = 0; j < JN; ++j) {
        if (r[j] < 0) continue;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack2(w[j] * g[i].x, w[j] * g[i].y);
        __stcs(reinterpret_cast<uint4*>(dD + static_cast<int64_t>(r[j]) * lddd + n),
               make_uint4(o[0], o[1], o[2], o[3]));
        if (dweights) {
          float2 f[4], s = make_float2(0.0f, 0.0f);
          d[j].get(f);
#pragma unroll
          for (int i = 0; i < 4; ++i) s = __ffma2_rn(f[i], g[i], s);
          dot[j] += s.x + s.y;
        }
      }
    }
    if (dweights) {
      cta_sum<kWarps>(dot, red, phase++);
#pragma unroll
      for (int j = 0; j < JN; ++j)
        if (static_cast<int>(threadIdx.x) == j && j0 + j < topk) dweights[t * topk + j0 + j] = dot[j];
    }
  }
}

bool dtype_ok(int32_t d) { return d == FP8G_BF16 || d == FP8G_F32; }
uintptr_t dtype_size(int32_t d) { return d == FP8G_F32 ? 4 : 2; }

// Rows that a CTA has at once, by the lanes a row takes.
int64_t gate_rows(int E) {
  int lpr = 1;
  while (lpr < 32 && lpr * 8 < E) lpr *= 2;
  return kGateWarps * (32 / lpr);
}
// Whether a call is finished by one CTA or cluster, without partial sums.
bool gate_few(int64_t T, int E) { return T <= 2 * kGateCluster * gate_rows(E); }
// The CTAs of a larger call, at most (each writes a row of partial sums).
int64_t gate_parts(int64_t T, int E) {
  return gate_few(T, E) ? 0 : std::min<int64_t>(kGateMaxParts, (T + gate_rows(E) - 1) / gate_rows(E));
}

template <typename TL, int VPL, int LPR>
int gate_launch(const GateArgs& a, const DeviceInfo* dev, cudaStream_t s) {
  // A CTA or a cluster of them for few rows: it finishes the counts and the loss itself.  More rows go to as many CTAs
  // as are resident at once (in clusters of 8, which do not fill every SM, 65536 x 256 took 54 us instead of 38), one
  // of 32 warps an SM where the registers allow it and there are rows for all of them (fewer partial sums: 65536 x 256
  // fp32 47 us, with four CTAs of 8 warps 51; bf16 38 with either).
  constexpr int kLarge = VPL == 8 ? 32 : kGateWarps;
  const int64_t G = 32 / LPR;
  const bool few = gate_few(a.T, a.E), large = !few && a.T >= dev->sm_count * kLarge * G;
  const int warps = large ? kLarge : kGateWarps;
  const int cluster = a.T <= 2 * kGateWarps * G || !few ? 1 : kGateCluster;
  const int64_t ctas = few ? cluster
                           : std::min({gate_parts(a.T, a.E), (a.T + warps * G - 1) / (warps * G),
                                       int64_t{gate_per_sm(VPL)} * kGateWarps / warps * dev->sm_count});
  const size_t smem = gate_smem<LPR>(a.E, a.topk, warps);
  auto kern = large ? moe_gate_kernel<TL, VPL, LPR, kLarge> : moe_gate_kernel<TL, VPL, LPR, kGateWarps>;
  const int st = allow_shared_memory(reinterpret_cast<const void*>(kern), smem);
  if (st != FP8G_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  if (few) return FP8G_OK;
  const int joins = std::min(kGateCluster, (a.E + 31) / 32);
  cfg.gridDim = dim3(static_cast<unsigned>(joins));
  cfg.blockDim = dim3(kGateJoinThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].val.clusterDim.x = static_cast<unsigned>(joins);
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, moe_gate_join_kernel, static_cast<const float*>(a.part_p),
                         static_cast<const int32_t*>(a.part_c), static_cast<int32_t>(ctas), a.E, a.topk, a.coef,
                         a.counts, a.loss) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

template <typename TL, int VPL, int LPR>
int gate_backward_launch(const GateGrad& a, const DeviceInfo* dev, cudaStream_t s) {
  auto kern = moe_gate_backward_kernel<TL, VPL, LPR>;
  const int64_t at_once = kGateWarps * (32 / LPR);
  const int64_t ctas = std::min<int64_t>((a.T + at_once - 1) / at_once, gate_grad_per_sm(VPL, LPR) * dev->sm_count);
  kern<<<static_cast<unsigned>(ctas), kGateThreads, 0, s>>>(a);
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
// Whether rows of logits can be taken eight at a time.
bool logit_vectors(const void* p, int64_t ld, int32_t dtype) {
  return aligned16(p) && (ld * static_cast<int64_t>(dtype_size(dtype))) % 16 == 0;
}

template <typename TO>
int combine_backward_launch(const void* dout, int64_t lddo, const __nv_bfloat16* D, int64_t M, int32_t N, int64_t ldd,
                            const int32_t* entry_row, const int32_t* row_token, int64_t T, int32_t topk,
                            const float* weights, __nv_bfloat16* dD, int64_t lddd, float* dweights,
                            const DeviceInfo* dev, cudaStream_t s) {
  // more threads a token where there are few tokens
  const bool few = T < 2 * dev->sm_count && N > 2048;
  auto kern = few          ? (topk <= 2   ? moe_combine_backward_kernel<TO, 2, 512>
                              : topk <= 4 ? moe_combine_backward_kernel<TO, 4, 512>
                                          : moe_combine_backward_kernel<TO, 8, 512>)
              : topk <= 2 ? moe_combine_backward_kernel<TO, 2, 128>
              : topk <= 4 ? moe_combine_backward_kernel<TO, 4, 128>
                          : moe_combine_backward_kernel<TO, 8, 128>;
  const int threads = few ? 512 : 128;
  // CTAs for the zero rows: down to a row a warp, two CTAs an SM at most
  const int warps = threads / 32;
  const int64_t zero = std::min<int64_t>((M + warps - 1) / warps, 2 * static_cast<int64_t>(dev->sm_count));
  kern<<<static_cast<unsigned>(zero + T), threads, 0, s>>>(static_cast<const TO*>(dout), lddo, D, M, N, ldd, entry_row,
                                                          row_token, static_cast<int32_t>(zero), topk, weights, dD,
                                                          lddd, dweights, dev->status);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

}  // namespace
}  // namespace fp8g

using namespace fp8g;

extern "C" int fp8g_moe_gate_workspace(int64_t T, int32_t E, int64_t* bytes) {
  if (T < 0 || T > 0x7FFFFFFF || E < 1 || E > kGateMaxExperts || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = gate_parts(T, E) * E * 8;
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
  const int64_t scratch = gate_parts(T, E) * E * 8;
  if (scratch > 0 && (!workspace || workspace_bytes < scratch)) return FP8G_ERR_INVALID_ARG;
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
  a.part_c = reinterpret_cast<int32_t*>(a.part_p + gate_parts(T, E) * E);
  a.T = T, a.ldl = ldl, a.E = E, a.topk = topk, a.renorm = renormalize, a.coef = loss_coef;
  a.vec = logit_vectors(logits, ldl, dtype);
  return (dtype == FP8G_F32 ? gate_form<float>(E) : gate_form<__nv_bfloat16>(E))(a, dev, s);
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
  a.vec = logit_vectors(logits, ldl, dtype) && logit_vectors(dlogits, ldd, dtype);
  return (dtype == FP8G_F32 ? gate_backward_form<float>(E) : gate_backward_form<__nv_bfloat16>(E))(
      a, dev, static_cast<cudaStream_t>(stream));
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
  // A CTA a token; few tokens are split by columns too, so that every SM has a few CTAs (64 tokens of 8 x 7168: 33 us
  // in whole rows).
  const int64_t spans = (N + kCombineSpan - 1) / kCombineSpan;
  const dim3 grid(static_cast<unsigned>(T),
                  static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(spans, 8 * dev->sm_count / T))));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto kern, auto type) {
    using TO = decltype(type);
    kern<<<grid, kCombineThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(D), M, static_cast<int32_t>(N), ldd,
                                          entry_row, topk, weights, static_cast<const TO*>(residual), ldr,
                                          static_cast<TO*>(out), ldo, dev->status);
  };
  if (out_dtype == FP8G_F32)
    launch(topk <= 2 ? moe_combine_kernel<float, 2> : moe_combine_kernel<float, 4>, float());
  else
    launch(topk <= 2 ? moe_combine_kernel<__nv_bfloat16, 2> : moe_combine_kernel<__nv_bfloat16, 4>, __nv_bfloat16());
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

extern "C" int fp8g_moe_combine_backward(const void* dout, int32_t dout_dtype, int64_t lddo, const void* D, int64_t M,
                                         int64_t N, int64_t ldd, const int32_t* entry_row,
                                         const int32_t* row_token, int64_t T, int32_t topk, const float* weights,
                                         void* dD, int64_t lddd, float* dweights, void* stream) {
  if (!dtype_ok(dout_dtype) || M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || N % 8 != 0 || lddd < N ||
      T < 0 || T > 0x7FFFFFFF - 4096 /* beside the CTAs of the zero rows */ || topk < 1 || T * topk > 0x7FFFFFFF ||
      lddo < N || (dweights && ldd < N))
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
  return (dout_dtype == FP8G_F32 ? combine_backward_launch<float> : combine_backward_launch<__nv_bfloat16>)(
      dout, lddo, static_cast<const __nv_bfloat16*>(D), M, static_cast<int32_t>(N), ldd, entry_row, row_token, T, topk,
      weights, static_cast<__nv_bfloat16*>(dD), lddd, dweights, dev, static_cast<cudaStream_t>(stream));
}
