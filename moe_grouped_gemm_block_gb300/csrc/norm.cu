// norm.cu -- layer norm over the rows of a matrix and its gradients.
//
//     mu_m = mean_n x,   r_m = 1 / sqrt(mean_n (x - mu)^2 + eps),   y = (x - mu) r w + b
//     with h = (x - mu) r and g = dy w:
//     dx = r (g - mean_n g - h mean_n (g h)),   dw = sum_m dy h,   db = sum_m dy
//
// All sums are taken in fp32.  The variance is the mean of the squared differences from the mean (a second pass over
// the values in registers), or in the ring from a value near it with a bound on what cancels; never the difference
// of two large sums.
//
// Forms, by the row's length (rows go in vectors of 8 values on the 16-byte grid, see RowShape):
//   warp     short rows: a row (or 2, 4 at once) per warp, all in registers, no barriers
//   ring     longer rows: resident CTAs (clusters of two beyond 8192 values) walk over their rows, which bulk copies
//            bring into a ring of shared-memory stages ahead of them; some warps form a row's sums, the others the
//            results, with the weights and (backward) the weight gradients' sums in registers
//   cta      forward, rows longer than the ring takes: a CTA per row, the row in registers
//   scalar   rows that share no grid: a CTA per row (backward: resident), value by value in registers
//   any      rows longer than those hold
// The form follows from N, the types, the alignment and the strides, not from M, but that a single row has no stride.  So
// on the 16-byte grid (N and the strides multiples of 8) a row's bits do not depend on how many rows the call has; off
// it they also follow from where the row starts, (m ld) mod 8, and a row alone may take another form than among others.
// (A CTA per row with all its threads on the sums, for few rows, would save less than a microsecond of the kernel:
// 64 x 7168 bf16.)
//
// Bound by memory, and below some tens of MB by a call's fixed part (launch, weights, first rows, the last stores:
// about 8 us of a ring, 11 backward with the joined sums).  Device times, and the share of the copy rate:
//   ring     16384 x 8192 fp32 rows, bf16 y: forward 135 us (88%), backward 212 (93%)
//            4096 x 7168 bf16: forward 25 us (69%), backward 41 (63%)
//            4096 x 12288 bf16, clusters: forward 44 us (67%), backward 75 (59%)
//   warp     16384 x 512 bf16: forward 10.4 us (48%), backward 16.4 (45%)
//   scalar and any are there for every other row, not for speed

#include <algorithm>
#include <cuda_runtime.h>
#include <initializer_list>

#include "common.cuh"
#include "ptx.cuh"
#include "rows.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kNormThreads = 256;

// ---------------------------------------------------------------- rows in registers
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, const float2 (&f)[4]) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y), pack2(f[3].x, f[3].y)));
}
__device__ __forceinline__ void store_pairs(float* p, const float2 (&f)[4]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
  __stcs(reinterpret_cast<float4*>(p + 4), make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The values of a vector that the mask has.
template <bool SHIFT, typename T>
__device__ __forceinline__ void store_masked(T* p, const float2 (&f)[4], uint32_t mask) {
  if (!SHIFT || mask == 0xFFu) {
    store_pairs(p, f);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (mask >> j & 1u) p[j] = from_f32<T>(j & 1 ? f[j / 2].y : f[j / 2].x);
}

// A vector of a row, read once: 16-byte loads where all of it may be read (`inside`, see vector_inside), value by value
// where it would reach past the matrix's end.
template <bool SHIFT, typename T>
__device__ __forceinline__ void load_vector(Raw8<T>& r, const T* p, uint32_t mask, bool inside) {
  if constexpr (!SHIFT) {  // a vector is there or not
    if (mask) r.load_stream(p);
    else r.zero();
  } else if (mask == 0xFFu || (mask && inside)) {
    r.load_stream(p);
    if (mask != 0xFFu) r.keep(mask);
  } else {
    r.gather(p, mask);
  }
}

// Eight weights (or biases) from column n on, where the mask has them; `fill` where there are none.  w_kind: the
// type, and kWeightVectors where the weights lie on 16-byte boundaries (and n is a multiple of 8).
constexpr int32_t kWeightVectors = 2;
__device__ __forceinline__ void weights8(const void* w, int32_t w_kind, int n, uint32_t mask, float fill,
                                         float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = both(fill);
  if (!w || !mask) return;
  if (w_kind == (FP8G_F32 | kWeightVectors)) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + n);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  } else if (w_kind == (FP8G_BF16 | kWeightVectors)) {
    Raw8<__nv_bfloat16> r;
    r.v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + n));
    r.get(f);
  } else {
    // eight loads at once, without branches: where a value does not exist, of one that does
    float t[8];
    const int some = n + __ffs(mask) - 1;
    if ((w_kind & ~kWeightVectors) == FP8G_F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = __ldg(static_cast<const float*>(w) + (mask >> j & 1u ? n + j : some));
    } else {
      unsigned short h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = __ldg(static_cast<const unsigned short*>(w) + (mask >> j & 1u ? n + j : some));
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = __uint_as_float(static_cast<uint32_t>(h[j]) << 16);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (mask >> j & 1u) (j & 1 ? f[j / 2].y : f[j / 2].x) = t[j];
  }
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The sum of a pair over the CTA, the same in every thread; `red` holds two rounds of 32 pairs (round `phase`),
// so one barrier a call is enough.
__device__ __forceinline__ float2 block_sum(float2 v, float2 (*red)[32], int phase) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = make_float2(warp_sum(v.x), warp_sum(v.y));
  if (warps == 1) return v;
  if (lane == 0) red[phase & 1][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? red[phase & 1][lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}
__device__ __forceinline__ float block_sum(float v, float2 (*red)[32], int phase) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  v = warp_sum(v);
  if (warps == 1) return v;
  if (lane == 0) red[phase & 1][threadIdx.x >> 5].x = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[phase & 1][lane].x : 0.0f);
}

// The sum of (x - mu)^2 over the existing values of NV vectors.
template <bool SHIFT, typename T, int NV>
__device__ __forceinline__ float spread_sum(const Raw8<T> (&raw)[NV], const uint32_t (&mask)[NV], float mu) {
  float2 s = both(0.0f);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!mask[v]) continue;
    float2 f[4];
    raw[v].get(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 d = __fadd2_rn(f[i], both(-mu));
      if (SHIFT && mask[v] != 0xFFu)
        d = make_float2(mask[v] >> (2 * i) & 1u ? d.x : 0.0f, mask[v] >> (2 * i + 1) & 1u ? d.y : 0.0f);
      s = __ffma2_rn(d, d, s);
    }
  }
  return s.x + s.y;
}
template <typename T, int NV>
__device__ __forceinline__ float value_sum(const Raw8<T> (&raw)[NV]) {
  float2 s = both(0.0f);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float2 f[4];
    raw[v].get(f);
    s = __fadd2_rn(s, __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3])));
  }
  return s.x + s.y;
}

// ---------------------------------------------------------------- the ring of row stages
// Roles of a CTA's warps: column warps own kRingVecs vectors a thread of every row, sum warps take whole rows in
// turn and form their sums, one thread of the last warp issues the copies.  A row's stage goes full (its copies have
// landed) -> ready (its sums are in `slot`; the column warps wait for this alone, as a sum warp of their CTA gave it
// after it had seen the stage full: a second wait made 16384 x 4096 bf16 7% slower) -> empty (every column warp has
// read it); nothing else orders the warps, so the latencies of one row's sums lie under the columns' work on others.
// (With all warps of the CTA taking a row together, sums through a barrier, a row cost about 2000 cycles of latency:
// 4096 x 7168 bf16 rows took 42 us forward and 43 us backward, and 29 and 36 us with two to four rows at a time.)
constexpr int kRingMaxStages = 16;
constexpr int kRingVecs = 2;
constexpr int kRingMaxColumnWarps = 16;
// With 16 column warps: forward 24 warps of 80 registers, backward 20 warps of 96.
constexpr int kRingThreads = 32 * 24, kRingGradThreads = 32 * 20;

struct RingShared {
  uint64_t full[kRingMaxStages], ready[kRingMaxStages], empty[kRingMaxStages];
  uint64_t peer[kRingMaxStages];   // a cluster's: the other CTA has read its slot
  float4 slot[kRingMaxStages][2];  // a row's sums from each CTA of the cluster
  int dead;
};

// Waits for a barrier's phase, at most `budget` cycles; past that it records the status and nobody in the CTA waits
// any more (the results are void, the kernel ends).  False: the phase is not complete.  CLUSTER: what the other CTA wrote
// before it arrived is seen too.
template <bool CLUSTER = false>
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, long long budget, unsigned int* status,
                                          volatile int* dead) {
  const uint32_t b = smem_u32(bar);
  auto done = [&] { return CLUSTER ? mbar_try_wait_cluster(b, parity) : mbar_try_wait(b, parity); };
  if (done()) return true;
  const long long t0 = clock64();
  while (!done()) {
    if (*dead) return false;
    if (clock64() - t0 > budget) {
      *dead = 1;
      record_status(status, FP8G_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// Whether a wait has run out, the same answer in all of a warp.  The sum warps leave then: no barrier is told twice in
// a phase what to expect.
__device__ __forceinline__ bool ring_dead(const RingShared& sm) {
  return __any_sync(0xffffffffu, *const_cast<const volatile int*>(&sm.dead));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// Written to a CTA of the cluster; its barrier `bar` counts the 16 bytes when they are there.
__device__ __forceinline__ void st_async4(uint32_t addr, float4 v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   addr),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}

// Vector v of the share from its stage.  The values that do not exist are zero (ZERO), or anything: those of the
// neighbouring rows, which the column warps leave out of all that they store.
template <bool SHIFT, bool ZERO, typename T>
__device__ __forceinline__ void stage_vector(Raw8<T>& r, const T* stage, int v, uint32_t mask, bool last_row,
                                             const T* row) {
  if (SHIFT && mask != 0xFFu && last_row) {
    r.gather(row + v * 8, mask);  // row: the share's first vector in memory
  } else {
    r.load(stage + v * 8);
    if (SHIFT && ZERO && mask != 0xFFu) r.keep(mask);
  }
}

constexpr int kSumUnroll = 4;  // vectors in flight per lane of a sum warp

// The rows of sum warp w: those in the stages w, w + warps, ... in every round, so that it sees each round of its
// stages' barriers (a wait tells the round only by its parity).
struct SumRows {
  int stage, round, w, warps, stages;
  __device__ __forceinline__ SumRows(int w_, int warps_, int stages_)
      : stage(w_), round(0), w(w_), warps(warps_), stages(stages_) {}
  __device__ __forceinline__ int64_t row() const { return static_cast<int64_t>(round) * stages + stage; }
  __device__ __forceinline__ void next() {
    stage += warps;
    if (stage >= stages) {
      stage = w;
      ++round;
    }
  }
};

template <int CL>
__device__ __forceinline__ void ring_init(RingShared& sm, int stages, int column_warps) {
  if (threadIdx.x == 0) {
    sm.dead = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.ready[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), column_warps);
      mbar_init(smem_u32(&sm.peer[s]), 1);
    }
    fence_mbar_init();
  }
}

// In a cluster: tells the other CTA that its last row's sums have been read from this CTA's slot s.  Who does is a
// matter of time, as an arrival at another CTA waits for what its warp has on its way.  The column warps have stores
// (4096 x 12288 bf16 backward took 93 us).  The copying thread knows first, but then copies late: it does where the
// stages are few (16384 fp32 columns backward, 3 stages: 274 us, by the sum warps 352).  Else a sum warp does when it
// finds its stage full again (12288 bf16 columns forward, 16 stages: 44 us, by the copying thread 52).
constexpr int kRingFewStages = 4;
__device__ __forceinline__ void ring_tell(RingShared& sm, int s, int rank) {
  mbar_arrive_cluster(mapa_shared(smem_u32(&sm.peer[s]), rank ^ 1));
}

// The copying thread: row after row into the ring, each stage once it is empty.  `load` copies row i into stage s and
// returns nothing.  In the end, and where a wait has run out, it waits (with the same limit) for the copies on their way:
// none may land once the CTA has left.  `skip`: see NormArgs.
template <int CL, typename Load>
__device__ __forceinline__ void ring_copies(RingShared& sm, int rows, int stages, int rank, int skip, long long budget,
                                            unsigned int* status, Load load) {
  int s = 0, i = 0;
  uint32_t parity = 1;  // the first round of `empty` counts as complete
  for (; i < rows; ++i) {
    if (i >= stages) {
      ring_wait(&sm.empty[s], parity, budget, status, &sm.dead);
      if (*const_cast<volatile int*>(&sm.dead)) break;
      if (CL > 1 && stages <= kRingFewStages) ring_tell(sm, s, rank);
    }
    if (i != skip) load(i, s);
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
  }
  const long long t0 = clock64();
  for (int k = max(0, i - stages); k < i; ++k)
    while (!mbar_try_wait(smem_u32(&sm.full[k % stages]), (k / stages) & 1) && clock64() - t0 <= budget) {
    }
}
// The end of a cluster's CTA: neither leaves while the other may still write to it.  Where a wait has run out, sums may be
// on their way that nobody waits for (their arrival can be seen by their receiver alone): they get 2^17 cycles, some 60
// us, to land.
__device__ __forceinline__ void ring_leave_cluster(const RingShared& sm) {
  if (ring_dead(sm)) {
    const long long t0 = clock64();
    while (clock64() - t0 < (1 << 17)) {
    }
  }
  cluster_sync();
}

// A sum warp hands its row, of the ring's round `round`, on: its sums to every CTA of the cluster.
template <int CL>
__device__ __forceinline__ void ring_ready(RingShared& sm, int s, int round, int rank, float4 v, long long budget,
                                           unsigned int* status) {
  const int lane = threadIdx.x & 31;
  if constexpr (CL == 1) {
    if (lane == 0) {
      sm.slot[s][0] = v;
      mbar_arrive(smem_u32(&sm.ready[s]));
    }
  } else {
    if (lane == 0) mbar_arrive_expect_tx(true, smem_u32(&sm.ready[s]), CL * 16);
    if (round > 0 && !__all_sync(0xffffffffu, ring_wait<true>(&sm.peer[s], (round - 1) & 1, budget, status, &sm.dead)))
      return;
    if (lane < CL)
      st_async4(mapa_shared(smem_u32(&sm.slot[s][rank]), lane), v, mapa_shared(smem_u32(&sm.ready[s]), lane));
  }
}
// A column warp has read the stage and the slot.  (Where a wait has run out the column warps go through their remaining
// rows, whose values are void, without waiting: leaving the loop would take an answer that a whole warp agrees on in every
// row, and that holds up the lanes that have done with their last row for those that still store its ragged vectors:
// 8000 x 12001 bf16 forward 84 us, 88 so.)
__device__ __forceinline__ void ring_empty(RingShared& sm, int s) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&sm.empty[s]));
}

// ---------------------------------------------------------------- forward
// (y may be x itself: a row is read before it is written)
struct NormArgs {
  const void* x;
  void* y;
  const void* w;
  const void* b;
  float* mean;  // mean and rstd may be null
  float* rstd;
  int64_t M, ldx, ldy;
  int32_t N, w_kind;
  float eps;
  // Test hook, -1 normally: the ring's copying thread leaves out its row number `skip`, so that the waits for it run out.
  int32_t skip;
  unsigned int* status;
  long long budget;
};

__device__ __forceinline__ void norm_vector(float2 (&f)[4], float mu, float r, const float2 (&w)[4],
                                            const float2 (&b)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(f[i], both(-mu)), both(r)), w[i], b[i]);
}

// warp form: LPR lanes a row, lane l of a row holds the vectors l, l + LPR, ...  The next row is on its way while one
// is worked on.
template <typename TX, typename TY, int LPR, int NV, bool SHIFT>
__global__ void __launch_bounds__(kNormThreads) layer_norm_warp_kernel(const NormArgs a) {
  constexpr int kRows = kNormThreads / LPR;  // rows a CTA at once: a multiple of 8
  const int sub = threadIdx.x % LPR;
  const TX* x = static_cast<const TX*>(a.x);
  TY* y = static_cast<TY*>(a.y);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  // the loop runs for whole warps (m0 is the warp's first row): the sums are taken by all its lanes
  int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows + (threadIdx.x & ~31) / LPR;
  const int64_t off = (threadIdx.x & 31) / LPR;
  const RowShape<SHIFT> shape(a.N, m0 + off, a.ldx);
  uint32_t mask[NV];
  float2 wf[NV][4], bf[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    mask[v] = shape.mask(v * LPR + sub);
    weights8(a.w, a.w_kind, shape.col(v * LPR + sub), mask[v], 1.0f, wf[v]);
    weights8(a.b, a.w_kind, shape.col(v * LPR + sub), mask[v], 0.0f, bf[v]);
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  Raw8<TX> next[NV];
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = shape.col(v * LPR + sub);
      load_vector<SHIFT>(next[v], x + m * a.ldx + c, m < a.M ? mask[v] : 0u, vector_inside(m, a.M, a.ldx, a.N, c));
    }
  };
  fetch(m0 + off);
  for (; m0 < a.M; m0 += stride) {
    const int64_t m = m0 + off;
    Raw8<TX> raw[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) raw[v] = next[v];
    if (m0 + stride < a.M) fetch(m + stride);
    const float mu = lanes_sum<LPR>(value_sum(raw)) * inv_n;
    const float var = lanes_sum<LPR>(spread_sum<SHIFT>(raw, mask, mu)) * inv_n;
    const float r = 1.0f / sqrtf(var + a.eps);
    if (m >= a.M) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!mask[v]) continue;
      float2 f[4];
      raw[v].get(f);
      norm_vector(f, mu, r, wf[v], bf[v]);
      store_masked<SHIFT>(y + m * a.ldy + shape.col(v * LPR + sub), f, mask[v]);
    }
    if (sub == 0) {
      if (a.mean) a.mean[m] = mu;
      if (a.rstd) a.rstd[m] = r;
    }
  }
}

// The sums of a warp's values: their sum and, about their own mean, their squared differences.  `count`: the values
// that the warp holds.
template <bool SHIFT, typename T, int NV>
__device__ __forceinline__ float2 warp_moments(const Raw8<T> (&raw)[NV], const uint32_t (&mask)[NV], float inv_count) {
  const float s = warp_sum(value_sum(raw));
  return make_float2(s, warp_sum(spread_sum<SHIFT>(raw, mask, s * inv_count)));
}
// A row's mean and 1 / sqrt(variance + eps) from its warps' sums, lane i holding warp i's: the squared differences
// about the row's mean are those about each warp's own plus count (difference of the means)^2.
__device__ __forceinline__ float2 join_moments(float2 v, float count, float inv_count, float inv_n, float eps) {
  const float mu = warp_sum(v.x) * inv_n;
  const float d = v.x * inv_count - mu;
  const float var = warp_sum(fmaf(count * d, d, v.y)) * inv_n;
  return make_float2(mu, 1.0f / sqrtf(var + eps));
}
// The values that the calling warp's masks have.
template <int NV>
__device__ __forceinline__ int warp_count(const uint32_t (&mask)[NV]) {
  int n = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) n += __popc(mask[v]);
  return __reduce_add_sync(0xffffffffu, n);
}

// cta form: a CTA a row, thread t holds the vectors t, t + blockDim.x, ...
template <typename TX, typename TY, int NV, bool SHIFT>
__global__ void __launch_bounds__(1024) layer_norm_cta_kernel(const NormArgs a) {
  __shared__ float2 red[32];
  __shared__ float cnt[32];
  const int64_t m = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, threads = blockDim.x;
  const RowShape<SHIFT> shape(a.N, m, a.ldx);
  Raw8<TX> raw[NV];
  uint32_t mask[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = v * threads + static_cast<int>(threadIdx.x);
    mask[v] = shape.mask(i);
    load_vector<SHIFT>(raw[v], static_cast<const TX*>(a.x) + m * a.ldx + shape.col(i), mask[v],
                       vector_inside(m, a.M, a.ldx, a.N, shape.col(i)));
  }
  const int n = warp_count(mask);
  const float2 own = warp_moments<SHIFT>(raw, mask, n ? 1.0f / static_cast<float>(n) : 0.0f);
  if (lane == 0) {
    red[warp] = own;
    cnt[warp] = static_cast<float>(n);
  }
  __syncthreads();
  const bool in = lane < threads / 32;
  const float c = in ? cnt[lane] : 0.0f;
  const float2 st = join_moments(in ? red[lane] : both(0.0f), c, c > 0.0f ? 1.0f / c : 0.0f,
                                 1.0f / static_cast<float>(a.N), a.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!mask[v]) continue;
    const int col = shape.col(v * threads + static_cast<int>(threadIdx.x));
    float2 f[4], wf[4], bf[4];
    weights8(a.w, a.w_kind, col, mask[v], 1.0f, wf);
    weights8(a.b, a.w_kind, col, mask[v], 0.0f, bf);
    raw[v].get(f);
    norm_vector(f, st.x, st.y, wf, bf);
    store_masked<SHIFT>(static_cast<TY*>(a.y) + m * a.ldy + col, f, mask[v]);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[m] = st.x;
    if (a.rstd) a.rstd[m] = st.y;
  }
}

// ring form.  A sum warp takes the differences from K, the mean of the row's first whole vectors (of its CTA's share; 32,
// or 30 at the least): variance = mean (x - K)^2 - (mean (x - K))^2 then loses little to cancellation, as (K - mean)^2 is
// at most N / 240 variances whatever the values.  Nothing but the row's own values may enter K: a neighbour's could be
// anything.  The root is rsqrtf's, two units in the last place at most, which is less than the sums' own roundings (with
// IEEE roots 8000 x 12001 bf16 takes 88 us instead of 84).
template <typename TX, typename TY, int CL, bool SHIFT>
__global__ void __launch_bounds__(kRingThreads, 1) layer_norm_ring_kernel(const NormArgs a, int32_t stages,
                                                                             int32_t stage_bytes, int32_t column_warps,
                                                                             int32_t sum_warps) {
  constexpr int NV = kRingVecs;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ RingShared sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, columns = column_warps * 32;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int P = static_cast<int>(gridDim.x) / CL, first = static_cast<int>(blockIdx.x) / CL;
  const int rows = static_cast<int>((a.M - first + P - 1) / P);  // rows first, first + P, ...
  const RowShape<SHIFT> shape(a.N, first, a.ldx);
  const Share share(shape, rank, CL);
  const TX* x = static_cast<const TX*>(a.x) + shape.col(share.first);
  ring_init<CL>(sm, stages, column_warps);
  if constexpr (CL == 1) __syncthreads();
  else cluster_sync();  // every CTA of the cluster runs before it is written to
  if (warp == column_warps + sum_warps) {
    if (lane == 0)
      ring_copies<CL>(sm, rows, stages, rank, a.skip, a.budget, a.status, [&](int i, int s) {
        const int64_t m = first + static_cast<int64_t>(i) * P;
        const uint32_t bar = smem_u32(&sm.full[s]);
        const uint32_t bytes = static_cast<uint32_t>(copied(shape, share, m + 1 == a.M)) * 8 * sizeof(TX);
        mbar_arrive_expect_tx(true, bar, bytes);
        if (bytes) bulk_load(smem_u32(ring) + s * stage_bytes, x + m * a.ldx, bytes, bar);
      });
  } else if (warp >= column_warps) {
    // the values that the share holds
    const int held = min(a.N, shape.col(share.first + share.count)) - max(0, shape.col(share.first));
    const float n = static_cast<float>(held), inv_n = 1.0f / n;
    const Inner<SHIFT> in(share);
    const int heads = in.heads();
    const float inv_heads = 1.0f / static_cast<float>(8 * heads);
    for (SumRows it(warp - column_warps, sum_warps, stages); it.row() < rows; it.next()) {
      const int s = it.stage;
      const int64_t m = first + it.row() * P;
      ring_wait(&sm.full[s], it.round & 1, a.budget, a.status, &sm.dead);
      if (ring_dead(sm)) break;
      if (CL > 1 && it.round > 0 && lane == 0 && stages > kRingFewStages) ring_tell(sm, s, rank);
      const TX* stage = reinterpret_cast<const TX*>(ring + s * stage_bytes);
      float2 f[4], d1 = both(0.0f), d2 = both(0.0f), e1 = both(0.0f), e2 = both(0.0f);
      Raw8<TX> r[kSumUnroll];
      if (lane < heads) r[0].load(stage + (in.lo + lane) * 8);
      else r[0].zero();
      r[0].get(f);
      const float2 t = __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3]));
      const float K = warp_sum(t.x + t.y) * inv_heads;
      auto add = [&](const Raw8<TX>& raw) {
        raw.get(f);
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float2 p = __fadd2_rn(f[k], both(-K)), q = __fadd2_rn(f[k + 1], both(-K));
          d1 = __fadd2_rn(d1, p);
          d2 = __ffma2_rn(p, p, d2);
          e1 = __fadd2_rn(e1, q);
          e2 = __ffma2_rn(q, q, e2);
        }
      };
      int v = in.lo + lane;
      for (; v + 32 * (kSumUnroll - 1) < in.hi; v += 32 * kSumUnroll) {
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u) r[u].load(stage + (v + 32 * u) * 8);
#pragma unroll
        for (int u = 0; u < kSumUnroll; ++u) add(r[u]);
      }
      for (; v < in.hi; v += 32) {
        r[0].load(stage + v * 8);
        add(r[0]);
      }
      if (SHIFT && lane < 2) {  // the first and the last vector
        v = lane == 0 ? 0 : share.count - 1;
        const uint32_t mask = shape.mask(share.first + v);
        stage_vector<SHIFT, true>(r[0], stage, v, mask, m + 1 == a.M, x + m * a.ldx);
        r[0].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = mask >> j & 1u ? (j & 1 ? f[j / 2].y : f[j / 2].x) - K : 0.0f;
          d1.x += d;
          d2.x = fmaf(d, d, d2.x);
        }
      }
      d1 = __fadd2_rn(d1, e1);
      d2 = __fadd2_rn(d2, e2);
      const float s1 = warp_sum(d1.x + d1.y), s2 = warp_sum(d2.x + d2.y);
      float4 st = make_float4(fmaf(s1, inv_n, K), fmaf(-s1 * inv_n, s1, s2), n, 0.0f);
      if (st.y < 0.0f) st.y = 0.0f;  // a NaN stays one
      if constexpr (CL == 1) {
        st.y = rsqrtf(st.y * inv_n + a.eps);
        if (lane == 0) {
          if (a.mean) a.mean[m] = st.x;
          if (a.rstd) a.rstd[m] = st.y;
        }
      }
      ring_ready<CL>(sm, s, it.round, rank, st, a.budget, a.status);
    }
  } else {
    TY* y = static_cast<TY*>(a.y) + shape.col(share.first);
    uint32_t mask[NV];
    float2 wf[NV][4], bf[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * columns + tid;
      mask[v] = i < share.count ? shape.mask(share.first + i) : 0u;
      weights8(a.w, a.w_kind, shape.col(share.first + i), mask[v], 1.0f, wf[v]);
      weights8(a.b, a.w_kind, shape.col(share.first + i), mask[v], 0.0f, bf[v]);
    }
    const float inv_n = 1.0f / static_cast<float>(a.N);
    int s = 0;
    uint32_t parity = 0;
    for (int i = 0; i < rows; ++i) {
      const int64_t m = first + static_cast<int64_t>(i) * P;
      ring_wait<(CL > 1)>(&sm.ready[s], parity, a.budget, a.status, &sm.dead);
      const TX* stage = reinterpret_cast<const TX*>(ring + s * stage_bytes);
      const float4 st = sm.slot[s][0];
      float mu = st.x, r = st.y;
      if constexpr (CL == 2) {  // the two halves' means and spreads, each about its own mean
        const float4 su = sm.slot[s][1];
        const float d = su.x - st.x;
        mu = (st.x * st.z + su.x * su.z) * inv_n;
        r = rsqrtf(fmaf(d * d, st.z * su.z * inv_n, st.y + su.y) * inv_n + a.eps);
        if (rank == 0 && tid == 0) {
          if (a.mean) a.mean[m] = mu;
          if (a.rstd) a.rstd[m] = r;
        }
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        Raw8<TX> raw;
        if (mask[v]) stage_vector<SHIFT, false>(raw, stage, v * columns + tid, mask[v], m + 1 == a.M, x + m * a.ldx);
        if (v == NV - 1) ring_empty(sm, s);
        if (!mask[v]) continue;
        float2 f[4];
        raw.get(f);
        norm_vector(f, mu, r, wf[v], bf[v]);
        store_masked<SHIFT>(y + m * a.ldy + (v * columns + tid) * 8, f, mask[v]);
      }
      if (++s == stages) {
        s = 0;
        parity ^= 1u;
      }
    }
  }
  if constexpr (CL > 1) ring_leave_cluster(sm);
}

// scalar form: thread t holds the values t, t + blockDim.x, ...
template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(1024) layer_norm_scalar_kernel(
    const TX* x, int32_t N, int64_t ldx, const void* __restrict__ w, const void* __restrict__ b,
    int32_t w_kind, float eps, TY* y, int64_t ldy, float* __restrict__ mean,
    float* __restrict__ rstd) {
  __shared__ float2 red[2][32];
  const int64_t m = blockIdx.x;
  float f[NV];
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
    f[v] = col < N ? to_f32(x[m * ldx + col]) : 0.0f;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) s += f[v];
  const float inv_n = 1.0f / static_cast<float>(N);
  const float mu = block_sum(s, red, 0) * inv_n;
  s = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const float d = f[v] - mu;
    if (v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x) < N) s = fmaf(d, d, s);
  }
  const float r = 1.0f / sqrtf(block_sum(s, red, 1) * inv_n + eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
    if (col >= N) continue;
    const float wn = w ? load_any(w, w_kind, col) : 1.0f, bn = b ? load_any(b, w_kind, col) : 0.0f;
    y[m * ldy + col] = from_f32<TY>(fmaf((f[v] - mu) * r, wn, bn));
  }
  if (threadIdx.x == 0) {
    if (mean) mean[m] = mu;
    if (rstd) rstd[m] = r;
  }
}

// any form: one CTA a row, any length and alignment: the row is read three times (from L1 / L2 after the first).
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads) layer_norm_any_kernel(
    const TX* x, int64_t N, int64_t ldx, const void* __restrict__ w, const void* __restrict__ b,
    int32_t w_kind, float eps, TY* y, int64_t ldy, float* __restrict__ mean,
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
    const float wn = w ? load_any(w, w_kind, n) : 1.0f, bn = b ? load_any(b, w_kind, n) : 0.0f;
    yr[n] = from_f32<TY>((to_f32(xr[n]) - mu) * r * wn + bn);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[m] = mu;
    if (rstd) rstd[m] = r;
  }
}

// ---------------------------------------------------------------- backward
struct NormGrad {  // arguments of every backward form
  const void* dy;
  const void* x;
  void* dx;
  const void* w;
  const float* mean;
  const float* rstd;
  float* parts;  // each CTA's or cluster's sums of dy h and of dy (see Parts); null where none are wanted
  int64_t M, lddy, ldx, lddx;
  int32_t N, w_kind;
  int32_t skip;  // see NormArgs
  unsigned int* status;
  long long budget;
};

// One vector of a row: h = (x - mu) r and g = dy w ...
__device__ __forceinline__ void grad_hg(const float2 (&xf)[4], const float2 (&yf)[4], const float2 (&wf)[4], float mu,
                                        float r, float2 (&h)[4], float2 (&g)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = __fmul2_rn(__fadd2_rn(xf[i], both(-mu)), both(r));
    g[i] = __fmul2_rn(yf[i], wf[i]);
  }
}
// ... the row's sums of g and g h, and the weight gradients' terms ...
__device__ __forceinline__ void grad_sums(const float2 (&h)[4], const float2 (&g)[4], const float2 (&yf)[4], float2& s1,
                                          float2& s2, float2 (&dw)[4], float2 (&db)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s1 = __fadd2_rn(s1, g[i]);
    s2 = __ffma2_rn(g[i], h[i], s2);
    dw[i] = __ffma2_rn(yf[i], h[i], dw[i]);
    db[i] = __fadd2_rn(db[i], yf[i]);
  }
}
// ... and dx = r (g - c1 - h c2), with rc = r c.
__device__ __forceinline__ void grad_dx(const float2 (&h)[4], const float2 (&g)[4], float rc1, float rc2, float r,
                                        float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __ffma2_rn(g[i], both(r), __ffma2_rn(h[i], both(-rc2), both(-rc1)));
}
// How the partial sums lie: [P][2][pitch], column n of row k at n + ((k shift) mod 8).  The ring's rows are shifted as
// the matrix's, so that its vectors lie on the 16-byte grid here too (value by value, 3 x 5670 bf16 took 16 us instead
// of 12).
struct Parts {
  int64_t P, pitch;
  int32_t shift;
};
__host__ __device__ __forceinline__ int64_t shifted_pitch(int64_t n) { return (n + 15) / 8 * 8; }
__device__ __forceinline__ void store_part(float* p, const float2 (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}

// warp form, as forward.  One CTA an SM, of as many warps as its registers hold, so that there are few partial sums:
// the warps add theirs up in shared memory, kSumBuffers of them at a time.
constexpr int kSumBuffers = 4;
template <typename TX, typename TY, int NV, bool SHIFT>
__host__ __device__ constexpr int grad_warps() {
  return NV == 4 ? 8 : NV == 2 ? (sizeof(TX) + sizeof(TY) > 4 ? 12 : 16) : SHIFT ? 16 : 20;
}
template <typename TX, typename TY, int LPR, int NV, bool SHIFT>
__global__ void __launch_bounds__(32 * grad_warps<TX, TY, NV, SHIFT>(), 1)
    layer_norm_grad_warp_kernel(const NormGrad a) {
  constexpr int kNormGradThreads = 32 * grad_warps<TX, TY, NV, SHIFT>();
  constexpr int kRows = kNormGradThreads / LPR;  // (times a grid that is a multiple of 8, or the whole matrix)
  constexpr int kCols = LPR * NV * 8;
  __shared__ __align__(16) float sums[kSumBuffers][2 * kCols];
  griddep_launch_dependents();
  const int sub = threadIdx.x % LPR;
  const TX* x = static_cast<const TX*>(a.x);
  const TY* dy = static_cast<const TY*>(a.dy);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t m0 = static_cast<int64_t>(blockIdx.x) * kRows + (threadIdx.x & ~31) / LPR;
  const int64_t off = (threadIdx.x & 31) / LPR;
  const RowShape<SHIFT> shape(a.N, m0 + off, a.ldx);
  uint32_t mask[NV];
  float2 wf[NV][4], dw[NV][4], db[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    mask[v] = shape.mask(v * LPR + sub);
    weights8(a.w, a.w_kind, shape.col(v * LPR + sub), mask[v], 1.0f, wf[v]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[v][i] = db[v][i] = both(0.0f);
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  Raw8<TX> nx[NV];
  Raw8<TY> ny[NV];
  float nmu = 0.0f, nr = 0.0f;
  auto fetch = [&](int64_t m) {  // what lies past a row's or the matrix's end is zero and adds nothing
    const bool in = m < a.M;
    nmu = in ? a.mean[m] : 0.0f;
    nr = in ? a.rstd[m] : 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = shape.col(v * LPR + sub);
      load_vector<SHIFT>(nx[v], x + m * a.ldx + c, in ? mask[v] : 0u, vector_inside(m, a.M, a.ldx, a.N, c));
      load_vector<SHIFT>(ny[v], dy + m * a.lddy + c, in ? mask[v] : 0u, vector_inside(m, a.M, a.lddy, a.N, c));
    }
  };
  fetch(m0 + off);
  for (; m0 < a.M; m0 += stride) {
    const int64_t m = m0 + off;
    const float mu = nmu, r = nr;
    float2 h[NV][4], g[NV][4], s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 xf[4], yf[4];
      nx[v].get(xf);
      ny[v].get(yf);
      grad_hg(xf, yf, wf[v], mu, r, h[v], g[v]);
      grad_sums(h[v], g[v], yf, s1, s2, dw[v], db[v]);
    }
    if (m0 + stride < a.M) fetch(m + stride);
    const float rc1 = lanes_sum<LPR>(s1.x + s1.y) * inv_n * r, rc2 = lanes_sum<LPR>(s2.x + s2.y) * inv_n * r;
    if (m >= a.M) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!mask[v]) continue;
      float2 f[4];
      grad_dx(h[v], g[v], rc1, rc2, r, f);
      store_masked<SHIFT>(static_cast<TX*>(a.dx) + m * a.lddx + shape.col(v * LPR + sub), f, mask[v]);
    }
  }
  if (!a.parts) return;
  // over the rows that the warp's lanes shared (rows of one shape each), then over the warps
  if constexpr (!SHIFT) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1) {
          dw[v][i].x += __shfl_xor_sync(0xffffffffu, dw[v][i].x, o);
          dw[v][i].y += __shfl_xor_sync(0xffffffffu, dw[v][i].y, o);
          db[v][i].x += __shfl_xor_sync(0xffffffffu, db[v][i].x, o);
          db[v][i].y += __shfl_xor_sync(0xffffffffu, db[v][i].y, o);
        }
  }
  for (int n = threadIdx.x; n < kSumBuffers * 2 * kCols; n += kNormGradThreads) sums[0][n] = 0.0f;
  __syncthreads();
  // on the grid a warp's lanes hold each column once; off it every row group has columns of its own
  constexpr int kGroups = SHIFT ? kNormGradThreads / LPR : kNormGradThreads / 32;
  const int own = SHIFT ? static_cast<int>(threadIdx.x) / LPR
                        : (threadIdx.x & 31) < LPR ? static_cast<int>(threadIdx.x) / 32 : -1;
  for (int t = 0; t < kGroups; t += kSumBuffers) {
    if (own >= t && own < t + kSumBuffers) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float* sw = sums[own - t] + shape.col(v * LPR + sub);
        if (!SHIFT || mask[v] == 0xFFu) {
          if (!mask[v]) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sw[j] += j & 1 ? dw[v][j / 2].y : dw[v][j / 2].x;
            sw[kCols + j] += j & 1 ? db[v][j / 2].y : db[v][j / 2].x;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (mask[v] >> j & 1u) {
              sw[j] += j & 1 ? dw[v][j / 2].y : dw[v][j / 2].x;
              sw[kCols + j] += j & 1 ? db[v][j / 2].y : db[v][j / 2].x;
            }
        }
      }
    }
    __syncthreads();
  }
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * 2 * a.N;
  for (int n = threadIdx.x; n < a.N; n += kNormGradThreads) {
    part[n] = (sums[0][n] + sums[1][n]) + (sums[2][n] + sums[3][n]);
    part[a.N + n] = (sums[0][kCols + n] + sums[1][kCols + n]) + (sums[2][kCols + n] + sums[3][kCols + n]);
  }
}

// ring form, as forward with the x and dy rows in a stage.  The sum warps read the weights from shared memory, in the
// order of the row's vectors: the first four values of every vector, then the other four (16-byte reads without
// bank conflicts).
template <typename TX, typename TY, int CL, bool SHIFT>
__global__ void __launch_bounds__(kRingGradThreads, 1) layer_norm_grad_ring_kernel(
    const NormGrad a, int32_t stages, int32_t stage_bytes, int32_t x_bytes, int32_t column_warps, int32_t sum_warps) {
  constexpr int NV = kRingVecs;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ RingShared sm;
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, columns = column_warps * 32;
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int P = static_cast<int>(gridDim.x) / CL, first = static_cast<int>(blockIdx.x) / CL;
  const int rows = static_cast<int>((a.M - first + P - 1) / P);  // rows first, first + P, ...
  const RowShape<SHIFT> shape(a.N, first, a.ldx);
  const Share share(shape, rank, CL);
  const TX* x = static_cast<const TX*>(a.x) + shape.col(share.first);
  const TY* dy = static_cast<const TY*>(a.dy) + shape.col(share.first);
  float4* ws = reinterpret_cast<float4*>(ring + stages * stage_bytes);  // [2][share.count]
  ring_init<CL>(sm, stages, column_warps);
  if constexpr (CL == 1) __syncthreads();
  else cluster_sync();  // every CTA of the cluster runs before it is written to
  const float inv_n = 1.0f / static_cast<float>(a.N);
  if (warp == column_warps + sum_warps) {
    if (lane == 0)
      ring_copies<CL>(sm, rows, stages, rank, a.skip, a.budget, a.status, [&](int i, int s) {
        const int64_t m = first + static_cast<int64_t>(i) * P;
        const uint32_t bar = smem_u32(&sm.full[s]), dst = smem_u32(ring) + s * stage_bytes;
        const uint32_t n = static_cast<uint32_t>(copied(shape, share, m + 1 == a.M)) * 8;
        mbar_arrive_expect_tx(true, bar, n * (sizeof(TX) + sizeof(TY)));
        if (n) {
          bulk_load(dst, x + m * a.ldx, n * sizeof(TX), bar);
          bulk_load(dst + x_bytes, dy + m * a.lddy, n * sizeof(TY), bar);
        }
      });
  } else if (warp >= column_warps) {
    // the weights, in the order of the row's vectors; the first copies are already under way
    for (int v = tid - columns; v < share.count; v += sum_warps * 32) {
      float2 f[4];
      weights8(a.w, a.w_kind, shape.col(share.first + v), shape.mask(share.first + v), 1.0f, f);
      ws[v] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      ws[share.count + v] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
    asm volatile("bar.sync 1, %0;" ::"r"(sum_warps * 32) : "memory");  // the sum warps among themselves
    SumRows it(warp - column_warps, sum_warps, stages);
    float nmu = 0.0f, nr = 0.0f;  // the next row's statistics
    auto stats = [&] {
      if (it.row() >= rows) return;
      nmu = a.mean[first + it.row() * P];
      nr = a.rstd[first + it.row() * P];
    };
    stats();
    while (it.row() < rows) {
      const int s = it.stage, round = it.round;
      const int64_t m = first + it.row() * P;
      const float mu = nmu, r = nr;
      it.next();
      stats();
      ring_wait(&sm.full[s], round & 1, a.budget, a.status, &sm.dead);
      if (ring_dead(sm)) break;
      if (CL > 1 && round > 0 && lane == 0 && stages > kRingFewStages) ring_tell(sm, s, rank);
      const TX* xs = reinterpret_cast<const TX*>(ring + s * stage_bytes);
      const TY* ys = reinterpret_cast<const TY*>(ring + s * stage_bytes + x_bytes);
      const Inner<SHIFT> in(share);
      float2 s1[2] = {both(0.0f), both(0.0f)}, s2[2] = {both(0.0f), both(0.0f)};
      auto add = [&](const Raw8<TX>& rx, const Raw8<TY>& ry, const float4& wa, const float4& wb) {
        const float2 w[4] = {make_float2(wa.x, wa.y), make_float2(wa.z, wa.w), make_float2(wb.x, wb.y),
                             make_float2(wb.z, wb.w)};
        float2 xf[4], yf[4];
        rx.get(xf);
        ry.get(yf);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 g = __fmul2_rn(yf[k], w[k]);
          s1[k & 1] = __fadd2_rn(s1[k & 1], g);
          s2[k & 1] = __ffma2_rn(g, __fadd2_rn(xf[k], both(-mu)), s2[k & 1]);
        }
      };
      constexpr int U = kSumUnroll / 2;
      int v = in.lo + lane;
      for (; v + 32 * (U - 1) < in.hi; v += 32 * U) {
        Raw8<TX> rx[U];
        Raw8<TY> ry[U];
        float4 wa[U], wb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          rx[u].load(xs + (v + 32 * u) * 8);
          ry[u].load(ys + (v + 32 * u) * 8);
          wa[u] = ws[v + 32 * u];
          wb[u] = ws[share.count + v + 32 * u];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) add(rx[u], ry[u], wa[u], wb[u]);
      }
      Raw8<TX> rx;
      Raw8<TY> ry;
      for (; v < in.hi; v += 32) {
        rx.load(xs + v * 8);
        ry.load(ys + v * 8);
        add(rx, ry, ws[v], ws[share.count + v]);
      }
      if (SHIFT && lane < 2) {  // the first and the last vector; dy is zero where they do not exist
        v = lane == 0 ? 0 : share.count - 1;
        const uint32_t mask = shape.mask(share.first + v);
        stage_vector<SHIFT, true>(rx, xs, v, mask, m + 1 == a.M, x + m * a.ldx);
        stage_vector<SHIFT, true>(ry, ys, v, mask, m + 1 == a.M, dy + m * a.lddy);
        add(rx, ry, ws[v], ws[share.count + v]);
      }
      s1[0] = __fadd2_rn(s1[0], s1[1]);
      s2[0] = __fadd2_rn(s2[0], s2[1]);
      const float c1 = warp_sum(s1[0].x + s1[0].y) * inv_n * r;
      const float c2 = warp_sum(s2[0].x + s2[0].y) * inv_n * r * r;
      ring_ready<CL>(sm, s, round, rank, make_float4(mu, r, c1, c2), a.budget, a.status);
    }
  } else {
    TX* out = static_cast<TX*>(a.dx) + shape.col(share.first);
    uint32_t mask[NV];
    float2 wf[NV][4], dw[NV][4], db[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = v * columns + tid;
      mask[v] = i < share.count ? shape.mask(share.first + i) : 0u;
      weights8(a.w, a.w_kind, shape.col(share.first + i), mask[v], 1.0f, wf[v]);
#pragma unroll
      for (int k = 0; k < 4; ++k) dw[v][k] = db[v][k] = both(0.0f);
    }
    int s = 0;
    uint32_t parity = 0;
    for (int i = 0; i < rows; ++i) {
      const int64_t m = first + static_cast<int64_t>(i) * P;
      ring_wait<(CL > 1)>(&sm.ready[s], parity, a.budget, a.status, &sm.dead);
      const TX* xs = reinterpret_cast<const TX*>(ring + s * stage_bytes);
      const TY* ys = reinterpret_cast<const TY*>(ring + s * stage_bytes + x_bytes);
      float4 st = sm.slot[s][0];
      if constexpr (CL == 2) {
        const float4 su = sm.slot[s][1];
        st.z += su.z;
        st.w += su.w;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        Raw8<TX> rx;
        Raw8<TY> ry;
        if (mask[v]) {
          stage_vector<SHIFT, false>(rx, xs, v * columns + tid, mask[v], m + 1 == a.M, x + m * a.ldx);
          stage_vector<SHIFT, false>(ry, ys, v * columns + tid, mask[v], m + 1 == a.M, dy + m * a.lddy);
        }
        if (v == NV - 1) ring_empty(sm, s);
        if (!mask[v]) continue;
        float2 xf[4], yf[4], h[4], g[4], f[4];
        rx.get(xf);
        ry.get(yf);
        grad_hg(xf, yf, wf[v], st.x, st.y, h, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dw[v][k] = __ffma2_rn(yf[k], h[k], dw[v][k]);
          db[v][k] = __fadd2_rn(db[v][k], yf[k]);
        }
        grad_dx(h, g, st.z, st.w, st.y, f);
        store_masked<SHIFT>(out + m * a.lddx + (v * columns + tid) * 8, f, mask[v]);
      }
      if (++s == stages) {
        s = 0;
        parity ^= 1u;
      }
    }
    if (a.parts) {
      const int64_t pitch = SHIFT ? shifted_pitch(a.N) : a.N;
      float* part = a.parts + first * 2 * pitch + static_cast<int64_t>(share.first + tid) * 8;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!mask[v]) continue;
        store_part(part + v * columns * 8, dw[v]);
        store_part(part + pitch + v * columns * 8, db[v]);
      }
    }
  }
  if constexpr (CL > 1) ring_leave_cluster(sm);
}

// scalar form: resident CTAs, thread t holds the columns t, t + blockDim.x, ...
template <typename TX, typename TY, int NV>
__global__ void __launch_bounds__(512) layer_norm_grad_scalar_kernel(const NormGrad a) {
  __shared__ float2 red[2][32];
  griddep_launch_dependents();
  const int tid = threadIdx.x, threads = blockDim.x;
  const TX* x = static_cast<const TX*>(a.x);
  const TY* dy = static_cast<const TY*>(a.dy);
  float w[NV], dw[NV], db[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * threads + tid;
    w[v] = a.w && col < a.N ? load_any(a.w, a.w_kind, col) : 1.0f;
    dw[v] = db[v] = 0.0f;
  }
  const float inv_n = 1.0f / static_cast<float>(a.N);
  int phase = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const float mu = a.mean[m], r = a.rstd[m];
    float h[NV], g[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = v * threads + tid;
      h[v] = col < a.N ? to_f32(x[m * a.ldx + col]) : mu;
      g[v] = col < a.N ? to_f32(dy[m * a.lddy + col]) : 0.0f;
    }
    float2 s = both(0.0f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[v] = (h[v] - mu) * r;
      dw[v] = fmaf(g[v], h[v], dw[v]);
      db[v] += g[v];
      g[v] *= w[v];
      s.x += g[v];
      s.y = fmaf(g[v], h[v], s.y);
    }
    s = block_sum(s, red, phase++);
    const float c1 = s.x * inv_n, c2 = s.y * inv_n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = v * threads + tid;
      if (col < a.N) static_cast<TX*>(a.dx)[m * a.lddx + col] = from_f32<TX>(fmaf(h[v], -c2, g[v] - c1) * r);
    }
  }
  if (!a.parts) return;
  float* part = a.parts + blockIdx.x * 2 * static_cast<int64_t>(a.N);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = v * threads + tid;
    if (col < a.N) {
      part[col] = dw[v];
      part[a.N + col] = db[v];
    }
  }
}

// any form: the data gradient, one CTA a row, any length and alignment.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kNormThreads) layer_norm_dx_any_kernel(
    const TY* __restrict__ dy, int64_t lddy, const TX* __restrict__ x, int64_t ldx, const void* __restrict__ w,
    int32_t w_kind, const float* __restrict__ mean, const float* __restrict__ rstd, int64_t N,
    TX* __restrict__ dx, int64_t lddx) {
  __shared__ float red[2 * 2 * kNormThreads / 32];
  const int64_t m = blockIdx.x;
  const float mu = mean[m], r = rstd[m];
  const TX* xr = x + m * ldx;
  const TY* dyr = dy + m * lddy;
  float s[2] = {0.0f, 0.0f};
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float g = to_f32(dyr[n]) * (w ? load_any(w, w_kind, n) : 1.0f);
    s[0] += g;
    s[1] += g * ((to_f32(xr[n]) - mu) * r);
  }
  cta_sum<kNormThreads / 32>(s, red, 0);
  const float c1 = s[0] / static_cast<float>(N), c2 = s[1] / static_cast<float>(N);
  for (int64_t n = threadIdx.x; n < N; n += kNormThreads) {
    const float g = to_f32(dyr[n]) * (w ? load_any(w, w_kind, n) : 1.0f);
    dx[m * lddx + n] = from_f32<TX>((g - c1 - (to_f32(xr[n]) - mu) * r * c2) * r);
  }
}

// Partial sums of the weight gradients, any length and alignment: thread = column, blockIdx.y = a range of rows.
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

// dw and db (either may be null) from the P partial rows [2][N].  A CTA takes 32 columns, its warps an equal share of
// the rows each: the additions' order follows from P alone.  The sums are short and the rows' addresses far apart, so
// the time is the loads' latency: eight in flight per lane, and many warps (P = 152, N = 7168: 6.3 us with 8 warps,
// 5 with 19).
constexpr int kJoinMaxWarps = 32;
constexpr int kJoinUnroll = 8;
__global__ void __launch_bounds__(32 * kJoinMaxWarps) layer_norm_join_kernel(const float* __restrict__ parts, Parts l,
                                                                             int64_t N, float* __restrict__ dw,
                                                                             float* __restrict__ db) {
  __shared__ float sums[kJoinMaxWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  griddep_wait();
  const int lo = static_cast<int>(l.P * warp / warps), hi = static_cast<int>(l.P * (warp + 1) / warps);
  float s = 0.0f;
  if (i < 2 * N) {
    const float* p = parts + (i < N ? i : i - N + l.pitch);
    for (int k = lo; k < hi; k += kJoinUnroll) {
      float v[kJoinUnroll];
#pragma unroll
      for (int u = 0; u < kJoinUnroll; ++u)
        v[u] = k + u < hi ? __ldcg(p + (k + u) * 2 * l.pitch + ((k + u) * l.shift & 7)) : 0.0f;
      s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || i >= 2 * N) return;
  float t = 0.0f;
  for (int w = 0; w < warps; ++w) t += sums[w][lane];
  if (i < N) {
    if (dw) dw[i] = t;
  } else if (db) {
    db[i - N] = t;
  }
}

bool dtype_ok(int32_t d) { return d == FP8G_BF16 || d == FP8G_F32; }
int dtype_size(int32_t d) { return d == FP8G_F32 ? 4 : 2; }

// ---------------------------------------------------------------- launches
// The warp form's vectors a row, at most, on the 16-byte grid and off it.  Beyond them a lane's registers (weights,
// next row, backward the sums) leave too few warps an SM: 16384 x 1000 bf16 forward 30 us against 21 in the ring,
// backward 29 against 33; 16384 x 501 forward 30 against 21, backward 41 against 31.
constexpr int64_t kWarpVectors = 64, kWarpGradVectors = 128, kWarpShiftVectors = 32;
constexpr int64_t kRingMaxN = 8192;      // ring form: a CTA's columns; twice that in clusters of two
constexpr int64_t kCtaMaxN = 32768;      // cta form: up to 4 vectors a thread
constexpr int64_t kScalarMaxN = 16384;   // scalar form: up to 16 values a thread, forward ...
constexpr int64_t kGradScalarMaxN = 8192;  // ... and backward
// Shared memory of the stages (and weights) of one of `per_sm` CTAs an SM: its 228 KB but 1 KB a CTA and RingShared.
constexpr int ring_bytes(int per_sm) { return 228 * 1024 / per_sm - 1024 - 1280; }
static_assert(sizeof(RingShared) <= 1280 - 128, "with the stages' alignment");
constexpr int64_t kNormMaxParts = 912;   // rows of partial sums

// Rows of partial sums that the workspace has room for: the largest grid of any backward form.
int64_t norm_parts(int64_t M) { return std::min<int64_t>(M, kNormMaxParts); }

enum Grid { kNone, kGrid, kShifted };  // see RowShape
struct Rows {
  const void* p;
  int64_t ld;
};
// How the rows of all a call's matrices fall on the 16-byte grid: all on it, all equally off it, or neither.
Grid row_grid(int64_t M, int64_t N, std::initializer_list<Rows> all) {
  bool on = N % 8 == 0, same = true;
  const int64_t ld0 = all.begin()->ld & 7;
  for (const Rows& r : all) {
    if (!aligned16(r.p)) return kNone;
    on &= M == 1 || (r.ld & 7) == 0;
    same &= M == 1 || (r.ld & 7) == ld0;
  }
  return on ? kGrid : same ? kShifted : kNone;
}
// The weights' type as the kernels take it.
int32_t weight_kind(const void* w, const void* b, int32_t dtype, Grid grid) {
  return dtype | (aligned16(w) && aligned16(b) && grid == kGrid ? kWeightVectors : 0);
}
// Threads for `items` items a row at `each` a thread.
int row_threads(int64_t items, int each) { return static_cast<int>((items + each * 32 - 1) / (each * 32) * 32); }
// Vectors a row takes, at most.
int64_t row_vectors(int64_t N, Grid grid) { return (N + (grid == kShifted ? 7 : 0) + 7) / 8; }

struct RingPlan {
  int cluster, column_warps, sum_warps, stages, threads;
  int32_t each, stage_bytes;  // vectors a CTA holds of a row, at most; bytes of a stage
  int64_t rows_at_once;       // CTAs or clusters
};
// A ring for rows of `vecs` vectors, `size` bytes a value over all matrices of a stage; `extra` bytes of shared memory
// a vector beside the stages (backward).  As many CTAs an SM as its registers hold: short rows take several.
RingPlan ring_plan(int64_t M, int64_t vecs, int size, int extra, int max_threads, Grid grid, int sms) {
  RingPlan p;
  p.cluster = vecs * 8 <= kRingMaxN ? 1 : 2;
  p.each = static_cast<int32_t>((vecs + p.cluster - 1) / p.cluster);
  p.column_warps = row_threads(p.each, kRingVecs) / 32;
  const int warps = max_threads / 32;  // what an SM's registers hold
  // about a sum warp for two column warps, as far as there is room for them
  p.sum_warps = std::max(2, std::min(warps - 1 - p.column_warps, (p.column_warps + 2) / 2));
  // Short rows take several CTAs an SM.  Backward each of them writes its partial sums: with 16384 rows of 2048 bf16
  // values two are 20% faster than one (48 against 58 us), with 2560 (fp32 rows) 13% slower (84 against 74).
  int per_sm = std::max(1, warps / (p.column_warps + p.sum_warps + 1));
  if (extra && p.column_warps > 4) per_sm = 1;
  p.stage_bytes = p.each * 8 * size;
  p.stages = static_cast<int>(
      std::min<int64_t>(kRingMaxStages, (ring_bytes(per_sm) - static_cast<int64_t>(p.each) * extra) / p.stage_bytes));
  p.sum_warps = std::min(p.sum_warps, p.stages);  // (a sum warp has stages of its own)
  p.threads = 32 * (p.column_warps + p.sum_warps + 1);
  p.rows_at_once = std::min<int64_t>(static_cast<int64_t>(sms) * per_sm / p.cluster, kNormMaxParts);
  if (grid == kShifted) p.rows_at_once = p.rows_at_once / 8 * 8;  // a CTA's rows are multiples of 8 apart
  p.rows_at_once = std::min(M, p.rows_at_once);
  return p;
}
template <typename Kernel, typename... Args>
int ring_launch(Kernel kern, const RingPlan& p, int64_t smem, cudaStream_t s, Args... args) {
  const int st = allow_shared_memory(reinterpret_cast<const void*>(kern), ring_bytes(1));
  if (st != FP8G_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows_at_once * p.cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(p.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}

template <typename TX, typename TY, bool SHIFT>
int layer_norm_vectors(const NormArgs& a, Grid grid, const DeviceInfo* dev, cudaStream_t s) {
  const int64_t M = a.M, vecs = row_vectors(a.N, grid);
  const int sms = dev->sm_count;
  if (vecs <= (SHIFT ? kWarpShiftVectors : kWarpVectors)) {
    auto go = vecs <= 8    ? layer_norm_warp_kernel<TX, TY, 8, 1, SHIFT>
              : vecs <= 16 ? layer_norm_warp_kernel<TX, TY, 16, 1, SHIFT>
              : vecs <= 32 ? layer_norm_warp_kernel<TX, TY, 32, 1, SHIFT>
                           : layer_norm_warp_kernel<TX, TY, 32, 2, false>;
    const int64_t per = kNormThreads / (vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32);
    // three CTAs an SM, with several rows to a warp: 16384 x 512 bf16 10.4 us, x 128 6.7; with eight 12.4 and 8.2
    const int64_t ctas = std::min<int64_t>((M + per - 1) / per, 3 * static_cast<int64_t>(sms));
    go<<<static_cast<unsigned>(ctas), kNormThreads, 0, s>>>(a);
  } else if (vecs * 8 <= 2 * kRingMaxN) {
    const RingPlan p = ring_plan(M, vecs, sizeof(TX), 0, kRingThreads, grid, sms);
    auto go = p.cluster == 1 ? layer_norm_ring_kernel<TX, TY, 1, SHIFT> : layer_norm_ring_kernel<TX, TY, 2, SHIFT>;
    return ring_launch(go, p, static_cast<int64_t>(p.stages) * p.stage_bytes, s, a, p.stages, p.stage_bytes,
                       p.column_warps, p.sum_warps);
  } else {
    layer_norm_cta_kernel<TX, TY, 4, SHIFT><<<static_cast<unsigned>(M), row_threads(vecs, 4), 0, s>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

template <typename TX, typename TY>
int layer_norm_launch(NormArgs a, const DeviceInfo* dev, cudaStream_t s) {
  const Grid grid = row_grid(a.M, a.N, {{a.x, a.ldx}, {a.y, a.ldy}});
  const int32_t dtype = a.w_kind;
  a.w_kind = weight_kind(a.w, a.b, dtype, grid);
  if (grid != kNone && row_vectors(a.N, grid) * 8 <= kCtaMaxN)
    return grid == kGrid ? layer_norm_vectors<TX, TY, false>(a, grid, dev, s)
                         : layer_norm_vectors<TX, TY, true>(a, grid, dev, s);
  const TX* x = static_cast<const TX*>(a.x);
  TY* y = static_cast<TY*>(a.y);
  const unsigned rows = static_cast<unsigned>(a.M);
  if (a.N <= kScalarMaxN) {
    const int nv = a.N <= 1024 ? 4 : a.N <= 4096 ? 8 : 16;
    auto go = nv == 4   ? layer_norm_scalar_kernel<TX, TY, 4>
              : nv == 8 ? layer_norm_scalar_kernel<TX, TY, 8>
                        : layer_norm_scalar_kernel<TX, TY, 16>;
    go<<<rows, row_threads(a.N, nv), 0, s>>>(x, a.N, a.ldx, a.w, a.b, dtype, a.eps, y, a.ldy, a.mean, a.rstd);
  } else {
    layer_norm_any_kernel<TX, TY><<<rows, kNormThreads, 0, s>>>(x, a.N, a.ldx, a.w, a.b, dtype, a.eps, y, a.ldy, a.mean,
                                                                a.rstd);
  }
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}

// The backward forms; *l is how their partial sums lie.
template <typename TX, typename TY, bool SHIFT>
int layer_norm_grad_vectors(const NormGrad& a, Grid grid, Parts* l, const DeviceInfo* dev, cudaStream_t s) {
  const int64_t M = a.M, vecs = row_vectors(a.N, grid);
  const int sms = dev->sm_count;
  if (vecs <= (SHIFT ? kWarpShiftVectors : kWarpGradVectors)) {
    auto go = vecs <= 8    ? layer_norm_grad_warp_kernel<TX, TY, 8, 1, SHIFT>
              : vecs <= 16 ? layer_norm_grad_warp_kernel<TX, TY, 16, 1, SHIFT>
              : vecs <= 32 ? layer_norm_grad_warp_kernel<TX, TY, 32, 1, SHIFT>
              : vecs <= 64 ? layer_norm_grad_warp_kernel<TX, TY, 32, 2, false>
                           : layer_norm_grad_warp_kernel<TX, TY, 32, 4, false>;
    const int threads = 32 * (vecs <= 32   ? grad_warps<TX, TY, 1, SHIFT>()
                              : vecs <= 64 ? grad_warps<TX, TY, 2, false>()
                                           : grad_warps<TX, TY, 4, false>());
    const int64_t per = threads / (vecs <= 8 ? 8 : vecs <= 16 ? 16 : 32);
    l->P = std::min<int64_t>((M + per - 1) / per, std::min<int64_t>(sms, kNormMaxParts) / 8 * 8);
    go<<<static_cast<unsigned>(l->P), threads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
  }
  const RingPlan p = ring_plan(M, vecs, sizeof(TX) + sizeof(TY), 32, kRingGradThreads, grid, sms);
  l->P = p.rows_at_once;
  if (SHIFT) {
    l->pitch = shifted_pitch(a.N);
    l->shift = static_cast<int32_t>(a.ldx & 7);
  }
  auto go = p.cluster == 1 ? layer_norm_grad_ring_kernel<TX, TY, 1, SHIFT>
                           : layer_norm_grad_ring_kernel<TX, TY, 2, SHIFT>;
  return ring_launch(go, p, static_cast<int64_t>(p.stages) * p.stage_bytes + static_cast<int64_t>(p.each) * 32, s, a,
                     p.stages, p.stage_bytes, static_cast<int32_t>(p.each * 8 * sizeof(TX)), p.column_warps,
                     p.sum_warps);
}

template <typename TX, typename TY>
int layer_norm_backward_launch(NormGrad a, float* dw, float* db, const DeviceInfo* dev, cudaStream_t s) {
  const int64_t M = a.M, N = a.N;
  const int sms = dev->sm_count;
  const Grid grid = row_grid(M, N, {{a.x, a.ldx}, {a.dy, a.lddy}, {a.dx, a.lddx}});
  const int32_t dtype = a.w_kind;
  a.w_kind = weight_kind(a.w, nullptr, dtype, grid);
  Parts l{0, N, 0};
  if (grid != kNone && row_vectors(N, grid) * 8 <= 2 * kRingMaxN) {
    const int st = grid == kGrid ? layer_norm_grad_vectors<TX, TY, false>(a, grid, &l, dev, s)
                                 : layer_norm_grad_vectors<TX, TY, true>(a, grid, &l, dev, s);
    if (st != FP8G_OK) return st;
  } else if (N <= kGradScalarMaxN) {
    a.w_kind = dtype;
    const int nv = N <= 1024 ? 4 : N <= 4096 ? 8 : 16;
    const int threads = row_threads(N, nv);
    l.P = std::min<int64_t>({M, static_cast<int64_t>(sms) * std::max(1, std::min(4, 1024 / threads)), norm_parts(M)});
    auto go = nv == 4   ? layer_norm_grad_scalar_kernel<TX, TY, 4>
              : nv == 8 ? layer_norm_grad_scalar_kernel<TX, TY, 8>
                        : layer_norm_grad_scalar_kernel<TX, TY, 16>;
    go<<<static_cast<unsigned>(l.P), threads, 0, s>>>(a);
  } else {
    layer_norm_dx_any_kernel<TX, TY><<<static_cast<unsigned>(M), kNormThreads, 0, s>>>(
        static_cast<const TY*>(a.dy), a.lddy, static_cast<const TX*>(a.x), a.ldx, a.w, dtype, a.mean, a.rstd, N,
        static_cast<TX*>(a.dx), a.lddx);
    if (a.parts) {
      l.P = norm_parts(M);
      const dim3 ctas(static_cast<unsigned>((N + kNormThreads - 1) / kNormThreads), static_cast<unsigned>(l.P));
      layer_norm_dw_any_kernel<TX, TY><<<ctas, kNormThreads, 0, s>>>(
          static_cast<const TY*>(a.dy), a.lddy, static_cast<const TX*>(a.x), a.ldx, a.mean, a.rstd, M, N, a.parts);
    }
  }
  if (cudaGetLastError() != cudaSuccess) return FP8G_ERR_CUDA;
  if (!a.parts) return FP8G_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((2 * N + 31) / 32));
  const int64_t join_warps = std::min<int64_t>(kJoinMaxWarps, (l.P + kJoinUnroll - 1) / kJoinUnroll);
  cfg.blockDim = dim3(32 * static_cast<unsigned>(join_warps));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, layer_norm_join_kernel, static_cast<const float*>(a.parts), l, N,
                         dw, db) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
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
  NormArgs a{};
  a.x = x, a.y = y, a.w = weight, a.b = bias, a.mean = mean, a.rstd = rstd;
  a.M = M, a.ldx = ldx, a.ldy = ldy;
  a.N = static_cast<int32_t>(N), a.w_kind = w_dtype, a.eps = eps;
  a.status = dev->status, a.budget = wait_budget_cycles(), a.skip = test_skip_stage();
  return go(a, dev, static_cast<cudaStream_t>(stream));
}

extern "C" int fp8g_layer_norm_backward_workspace(int64_t M, int64_t N, int64_t* bytes) {
  if (M < 0 || M > 0x7FFFFFFF || N < 1 || N > 0x7FFFFFFF || !bytes) return FP8G_ERR_INVALID_ARG;
  *bytes = norm_parts(M) * 2 * shifted_pitch(N) * 4;
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
  if ((dweight || dbias) && M > 0 && (!workspace || workspace_bytes < norm_parts(M) * 2 * shifted_pitch(N) * 4))
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
  NormGrad a{};
  a.dy = dy, a.x = x, a.dx = dx, a.w = weight, a.mean = mean, a.rstd = rstd;
  a.parts = dweight || dbias ? static_cast<float*>(workspace) : nullptr;
  a.M = M, a.lddy = lddy, a.ldx = ldx, a.lddx = lddx;
  a.N = static_cast<int32_t>(N), a.w_kind = w_dtype;
  a.status = dev->status, a.budget = wait_budget_cycles(), a.skip = test_skip_stage();
  return go(a, dweight, dbias, dev, s);
}
