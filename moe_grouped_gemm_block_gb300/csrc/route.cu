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
#include "shares.cuh"
#include "topk.cuh"
#include "vec.cuh"

namespace fp8g {
namespace {

constexpr int kRouteMaxExperts = 2048;
constexpr int kRouteMaxTopk = 32;
constexpr int kRouteMaxGroups = 32;
constexpr int kRouteWarps = 4;
// Picks of a row whose contenders are looked for, with scores and where the logits decide alone.  4096 x 1024, us, all in 64 bits
// and contenders first: 17 picks 333 and 56, 24 336 and 118, 28 338 and 243, 32 340 and 370 (contenders are too many then);
// by the logits 17 58 and 42, 24 70 and 49, 28 76 and 84.
constexpr int kRouteFewTopk = 28, kRouteFewLogits = 24;

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
  int32_t E, topk, groups, kept, log_groups, softmax, renorm, vec, single;
  float scale;
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The order of doubles as an unsigned integer (this GPU compares those many times faster): what is not a number stands as
// infinity, and so ranks first; 0 is below every value's key.
__device__ __forceinline__ uint64_t order_key(double v) {
  if (!(v == v)) v = INFINITY;
  const int64_t u = __double_as_longlong(v + 0.0);
  return static_cast<uint64_t>(u) ^ (static_cast<uint64_t>(u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t key) {
  return __longlong_as_double(static_cast<int64_t>(key & 0x8000000000000000ull ? key ^ 0x8000000000000000ull : ~key));
}
constexpr uint64_t kRuledOut = 0x000FFFFFFFFFFFFFull;  // the key of -inf

// e^x for x <= 0, in 64 bits without a branch (0 below 2^-1022): 2^n e^r with |r| <= ln 2 / 2, the series of e^r up to
// r^13 / 13! (the next term is below 2^-57).  ln 2 in two parts (Cody and Waite), the first its 42 leading bits, so that n
// times it, of at most 11 bits, is exact.
__device__ __forceinline__ double exp_series(double x) {
  const double n = rint(x * 1.4426950408889634);
  const double r = fma(n, -0x1.ef35793c7673p-45, fma(n, -0x1.62e42fefa38p-1, x));
  double p = 1.0 / 6227020800.0;
  constexpr double c[13] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                            1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0};
#pragma unroll
  for (int i = 0; i < 13; ++i) p = fma(p, r, c[i]);
  const int k = static_cast<int>(fmax(n, -1023.0));
  return x < -708.0 ? 0.0 : p * __longlong_as_double(static_cast<int64_t>(k + 1023) << 52);
}

// A row in 64 bits: `parts` warps make the keys of its experts in `key` (E words of shared memory; 0: not to be had), one of
// them chooses.  The scores of an expert: exponential() of its logit, then key() with the softmax's sum.
template <typename TL>
struct ExactRow {
  const RouteArgs& a;
  const TL* row;
  double mx;
  __device__ __forceinline__ ExactRow(const RouteArgs& args, int64_t t)
      : a(args), row(static_cast<const TL*>(args.logits) + t * args.ldl), mx(0.0) {
    if (!a.softmax) return;
    float m = -INFINITY;
    for (int e = threadIdx.x & 31; e < a.E; e += 32) m = fmaxf(m, to_f32(row[e]));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    mx = m == -INFINITY ? 0.0 : static_cast<double>(m);
  }
  __device__ __forceinline__ bool scored() const { return a.bias || a.groups > 1; }
  __device__ __forceinline__ double exponential(int e) const {
    const double l = to_f32(row[e]);
    return exp_series(a.softmax ? l - mx : -fabs(l));
  }
  __device__ __forceinline__ uint64_t key(int e, double x, double inv) const {
    const float l = to_f32(row[e]), b = a.bias ? a.bias[e] : 0.0f;
    const double score = a.softmax ? x * inv : (l < 0.0f ? x : 1.0) * __drcp_rn(1.0 + x);
    return l == -INFINITY || b == -INFINITY ? kRuledOut : order_key(score + static_cast<double>(b));
  }
};

// The groups that stay, by the keys of their experts: lanes (groups rounded up to a power of 2, log_l bits of lanes each) as a
// mask, bit g << log_l of group g among them.
__device__ __forceinline__ uint32_t route_groups(const RouteArgs& a, const uint64_t* key) {
  const int lane = threadIdx.x & 31, per = a.E / a.groups, log_l = 5 - a.log_groups, L = 1 << log_l, group = lane >> log_l;
  uint64_t first = 0, second = 0;
  if (group < a.groups)
    for (int i = lane & (L - 1); i < per; i += L) {
      const uint64_t v = key[group * per + i];
      second = max(second, min(first, v));
      first = max(first, v);
    }
  for (int off = 1; off < L; off <<= 1) {
    const uint64_t o1 = __shfl_xor_sync(0xffffffffu, first, off), o2 = __shfl_xor_sync(0xffffffffu, second, off);
    second = max(max(second, o2), min(first, o1));
    first = max(first, o1);
  }
  const uint64_t mine = second <= kRuledOut ? first : order_key(key_value(first) + key_value(second));
  int better = 0;
  for (int g = 0; g < a.groups; ++g) {
    const uint64_t other = __shfl_sync(0xffffffffu, mine, g << log_l);
    better += other > mine || (other == mine && g < group) ? 1 : 0;
  }
  return __ballot_sync(0xffffffffu, group < a.groups && better < a.kept);
}

// The score of expert e of a row whose softmax has these.
__device__ __forceinline__ float route_score(const RouteArgs& a, float l, float mx, float inv) {
  if (a.softmax) return exp_below(l, mx) * inv;
  const float x = exp_below(-fabsf(l), 0.0f), y = recip_approx(1.0f + x);
  return l < 0.0f ? x * y : y;
}
__device__ __forceinline__ float route_weight(const RouteArgs& a, float l, int e, float mx, float inv) {  // 0: ruled out
  return l == -INFINITY || (a.bias && a.bias[e] == -INFINITY) ? 0.0f : route_score(a, l, mx, inv);
}

// Where the chosen scores add up to less than this, down to what fp32 does not hold at all, weights over their sum are formed
// from common multiples of the scores (route_share): with `top` the largest chosen logit, and for a sigmoid at most 0, the
// largest is 1/2 to 1.  (Formed so always: 57 instead of 56 us, 64 rows 5.6 instead of 5.3.)
constexpr float kRouteSmall = 0x1p-60f;
__device__ __forceinline__ float route_share(const RouteArgs& a, float l, float top) {
  if (l == -INFINITY) return 0.0f;
  if (a.softmax) return exp_below(l, top);
  return exp_below(fminf(l, 0.0f), top) * recip_approx(1.0f + exp_below(-fabsf(l), 0.0f));
}
__device__ __forceinline__ float route_top(const RouteArgs& a, float l, int lanes) {  // lanes: of a row, a power of 2
  for (int off = 1; off < lanes; off <<= 1) l = fmaxf(l, __shfl_xor_sync(0xffffffffu, l, off));
  return a.softmax ? l : fminf(l, 0.0f);
}

// 1 / the sum of a softmax, for the weights.
template <typename TL>
__device__ __forceinline__ float route_inverse(const RouteArgs& a, const TL* row, float mx) {
  float s = 0.0f;
  for (int e = threadIdx.x & 31; e < a.E; e += 32) s += exp_below(to_f32(row[e]), mx);
  s = warp_sum(s);
  return s == 0.0f ? 0.0f : __fdiv_rn(1.0f, s);
}

// The choice of one warp from the keys: lane j < topk gets the j-th expert and its score.  (Without a bias and groups the keys
// are not looked at, nor is inv.)
template <typename TL>
__device__ __noinline__ void route_choose(const RouteArgs& a, int64_t t, uint64_t* key, double mx, double inv, int& pick,
                                          float& weight) {
  const int lane = threadIdx.x & 31, E = a.E, per = E / a.groups, log_l = 5 - a.log_groups;
  const TL* row = static_cast<const TL*>(a.logits) + t * a.ldl;
  const bool scored = a.bias || a.groups > 1;
  const uint32_t open = a.groups > 1 ? route_groups(a, key) : 0xffffffffu;
  uint64_t best = 0;
  int at = kRouteMaxExperts;
  for (int e = lane; e < E; e += 32) {
    uint64_t v = scored ? key[e] : 0;
    if (!a.bias) v = order_key(static_cast<double>(to_f32(row[e])));  // the scores order as the logits do
    v = open >> (e / per << log_l) & 1u ? v : 0;
    key[e] = v;
    if (v > best) best = v, at = e;
  }
  if (a.softmax && !scored) inv = route_inverse(a, row, static_cast<float>(mx));
  pick = 0;
  for (int j = 0; j < a.topk; ++j) {
    const uint32_t hi = static_cast<uint32_t>(best >> 32), top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = hi == top ? static_cast<uint32_t>(best) : 0u, low = __reduce_max_sync(0xffffffffu, lo);
    const uint32_t e = hi == top && lo == low ? static_cast<uint32_t>(at) : kRouteMaxExperts;
    const int one = static_cast<int>(__reduce_min_sync(0xffffffffu, e));
    if (lane == j) pick = min(one, E - 1);
    if (one == at && one < E) {  // its lane looks for its next one
      key[one] = 0;
      best = 0;
      at = kRouteMaxExperts;
      for (int i = lane; i < E; i += 32)
        if (key[i] > best) best = key[i], at = i;
    }
    __syncwarp();
  }
  weight = lane < a.topk ? route_weight(a, to_f32(row[pick]), pick, static_cast<float>(mx), static_cast<float>(inv)) : 0.0f;
  __syncwarp();
}

// The same choice where few experts can be it: their scores in fp32, off by less than 2^-24 (6 + |bias|), tell which groups
// stay (or which are their two largest, for 64 bits to decide) and which experts may be among the topk, and 64 bits are
// computed for those alone.  False: more than 64 of them, or a logit or bias that is NaN or +inf, or fewer than topk lanes
// with an expert that is not ruled out; then nothing is chosen.  (Not for a softmax with a bias: its sum needs every
// exponential.  Without one the order is that of the exponentials themselves.)
template <typename TL>
__device__ __noinline__ bool route_contenders(const ExactRow<TL>& r, uint64_t* key, int& pick) {
  const RouteArgs& a = r.a;
  const int lane = threadIdx.x & 31, E = a.E, per = E / a.groups, log_l = 5 - a.log_groups, L = 1 << log_l, group = lane >> log_l;
  float* value = reinterpret_cast<float*>(key);          // words 2 e: fp32 scores
  int32_t* list = reinterpret_cast<int32_t*>(key) + 1;   // words 2 i + 1: contenders
  auto slack = [](float v) { return 0x1p-22f * (8.0f + fabsf(v)); };  // twice the error of two such scores, and more
  auto approx = [&](int e) {
    const float l = to_f32(r.row[e]), b = a.bias ? a.bias[e] : 0.0f;
    if (l == -INFINITY || b == -INFINITY) return -INFINITY;
    if (a.softmax) return exp_below(l, static_cast<float>(r.mx));
    const float x = exp_below(-fabsf(l), 0.0f), y = recip_approx(1.0f + x);
    return (l < 0.0f ? x * y : y) + b;
  };
  auto gather = [&](auto in) {  // the experts for which in(e); how many
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const bool mine = in(e) && e < E;
      const uint32_t all = __ballot_sync(0xffffffffu, mine);
      if (mine) list[2 * (n + __popc(all & ((1u << lane) - 1u)))] = e;
      n += __popc(all);
    }
    __syncwarp();
    return n;
  };
  uint32_t open = 0xffffffffu;
  if (a.groups > 1) {
    bool odd = false;
    for (int e = lane; e < E; e += 32) {
      const float v = approx(e);
      value[2 * e] = v;
      odd |= !(v < INFINITY);
    }
    if (__any_sync(0xffffffffu, odd)) return false;
    __syncwarp();
    float first = -INFINITY, second = -INFINITY;
    if (group < a.groups)
      for (int i = lane & (L - 1); i < per; i += L) {
        const float v = value[2 * (group * per + i)];
        second = fmaxf(second, fminf(first, v));
        first = fmaxf(first, v);
      }
    for (int off = 1; off < L; off <<= 1) {
      const float o1 = __shfl_xor_sync(0xffffffffu, first, off), o2 = __shfl_xor_sync(0xffffffffu, second, off);
      second = fmaxf(fmaxf(second, o2), fminf(first, o1));
      first = fmaxf(first, o1);
    }
    const float sum = second == -INFINITY ? first : first + second;
    const float off = first == -INFINITY ? 0.0f : slack(first) + (second == -INFINITY ? 0.0f : slack(second));
    int better = 0;
    for (int g = 0; g < a.groups; ++g) {
      const float other = __shfl_sync(0xffffffffu, sum, g << log_l);
      better += other > sum || (other == sum && g < group) ? 1 : 0;
    }
    const bool stays = group < a.groups && better < a.kept;
    open = __ballot_sync(0xffffffffu, stays);
    float least = stays ? sum - off : INFINITY, most = group < a.groups && !stays ? sum + off : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if (a.kept < a.groups && !(least > most)) {  // 64 bits decide
      const float from = second == -INFINITY ? -INFINITY : second - slack(second);
      const int n = gather([&](int e) {
        const float mine = __shfl_sync(0xffffffffu, from, e < E ? e / per << log_l : 0);
        return e < E && value[2 * e] > -INFINITY && value[2 * e] >= mine;
      });
      if (n > 64) return false;
      const int e0 = lane < n ? list[2 * lane] : 0, e1 = lane + 32 < n ? list[2 * (lane + 32)] : 0;
      __syncwarp();
      for (int e = lane; e < E; e += 32) key[e] = value[2 * e] == -INFINITY ? kRuledOut : kRuledOut + 1;
      __syncwarp();
      if (lane < n) key[e0] = r.key(e0, r.exponential(e0), 1.0);
      if (lane + 32 < n) key[e1] = r.key(e1, r.exponential(e1), 1.0);
      __syncwarp();
      open = route_groups(a, key);
      __syncwarp();
    }
  }
  // (without a bias the order is that of the logits, and nothing is off)
  bool odd = false;
  float best = -INFINITY;
  for (int e = lane; e < E; e += 32) {
    const bool in = open >> (e / per << log_l) & 1u;
    const float v = !in ? -INFINITY : a.bias ? approx(e) : to_f32(r.row[e]);
    value[2 * e] = v;
    odd |= !(v < INFINITY);
    best = fmaxf(best, v);
  }
  if (__any_sync(0xffffffffu, odd)) return false;
  // the topk-th largest of the lanes' best is no larger than the topk-th of all
  uint32_t o = best == -INFINITY ? 0u : fp8g::order_key(best), kth = 0u;  // (of floats)
  for (int j = 0; j < a.topk; ++j) {
    kth = __reduce_max_sync(0xffffffffu, o);
    const uint32_t who = __ballot_sync(0xffffffffu, o == kth);
    if (lane == __ffs(who) - 1) o = 0u;
  }
  if (kth == 0u) return false;
  const float ref = fp8g::key_value(kth), from = a.bias ? ref - slack(ref) : ref;
  __syncwarp();
  const int n = gather([&](int e) { return e < E && value[2 * e] > -INFINITY && value[2 * e] >= from; });
  if (n > 64) return false;
  const int e0 = lane < n ? list[2 * lane] : 0, e1 = lane + 32 < n ? list[2 * (lane + 32)] : 0;
  auto exact = [&](int e) {
    return a.bias ? r.key(e, r.exponential(e), 1.0) : order_key(static_cast<double>(to_f32(r.row[e])));
  };
  uint64_t k0 = lane < n ? exact(e0) : 0, k1 = n > 32 && lane + 32 < n ? exact(e1) : 0;
  pick = 0;
  for (int j = 0; j < a.topk; ++j) {
    const uint64_t top = max(k0, k1);
    const uint32_t hi = static_cast<uint32_t>(top >> 32), high = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = hi == high ? static_cast<uint32_t>(top) : 0u, low = __reduce_max_sync(0xffffffffu, lo);
    const uint64_t best_key = static_cast<uint64_t>(high) << 32 | low;
    const uint32_t own = min(k0 == best_key ? static_cast<uint32_t>(e0) : static_cast<uint32_t>(kRouteMaxExperts),
                             k1 == best_key ? static_cast<uint32_t>(e1) : static_cast<uint32_t>(kRouteMaxExperts));
    const int one = static_cast<int>(__reduce_min_sync(0xffffffffu, own));
    if (lane == j) pick = min(one, E - 1);
    if (k0 == best_key && e0 == one) k0 = 0;
    else if (k1 == best_key && e1 == one) k1 = 0;
  }
  __syncwarp();
  return true;
}

// A row by one warp, where few experts can be chosen (see route_contenders); false: it is not such a row.
template <typename TL>
__device__ __noinline__ bool route_few(const RouteArgs& a, int64_t t, uint64_t* key, int& pick, float& weight) {
  const ExactRow<TL> r(a, t);
  const int lane = threadIdx.x & 31;
  if ((a.softmax && a.bias) || a.topk > (r.scored() ? kRouteFewTopk : kRouteFewLogits)) return false;
  const bool done = route_contenders<TL>(r, key, pick);
  __syncwarp();
  if (!done) return false;
  const float mx = static_cast<float>(r.mx), inv = a.softmax ? route_inverse(a, r.row, mx) : 1.0f;
  weight = lane < a.topk ? route_weight(a, to_f32(r.row[pick]), pick, mx, inv) : 0.0f;
  return true;
}

// A row by one warp, whose softmax's sum is formed as `parts` warps form it: a row's bits are the same wherever it is decided.
template <typename TL>
__device__ __noinline__ void route_row(const RouteArgs& a, int64_t t, uint64_t* key, int parts, int& pick, float& weight) {
  const ExactRow<TL> r(a, t);
  const int lane = threadIdx.x & 31;
  double inv = 1.0;
  if (a.softmax && r.scored()) {
    double s = 0.0;
    for (int p = 0; p < parts; ++p) {
      double part = 0.0;
      for (int e = p * 32 + lane; e < a.E; e += parts * 32) part += r.exponential(e);
      s += warp_sum(part);
    }
    inv = s == 0.0 ? 0.0 : 1.0 / s;
  }
  if (r.scored())
    for (int e = lane; e < a.E; e += 32) key[e] = r.key(e, r.exponential(e), inv);
  __syncwarp();
  route_choose<TL>(a, t, key, r.mx, inv, pick, weight);
}

// A row's result, as lane j < topk has its j-th choice and its score.
template <typename TL>
__device__ __forceinline__ void put_row(const RouteArgs& a, int64_t t, int id, float w, int32_t* counts) {
  const int lane = threadIdx.x & 31;
  const bool real = !a.mask || a.mask[t];
  float sum = warp_sum(w);
  if (a.renorm) {
    if (!(sum >= kRouteSmall)) {  // (the same for all lanes; a sum that is no number stays one)
      float l = -INFINITY;
      if (lane < a.topk && !(a.bias && a.bias[id] == -INFINITY)) l = to_f32(static_cast<const TL*>(a.logits)[t * a.ldl + id]);
      const float share = route_share(a, l, route_top(a, l, 32));
      w = w != w ? w : share;
      sum = warp_sum(w);
    }
    w = sum == 0.0f ? 0.0f : __fdiv_rn(w, sum);
  }
  if (lane < a.topk) {
    a.ids[t * a.topk + lane] = id;
    a.weights[t * a.topk + lane] = real ? w * a.scale : 0.0f;
    if (real) atomicAdd(counts + id, 1);  // whole numbers: the order does not matter
  }
}

// The general form: a warp a row.  4096 rows of 1024, 8 picks: 53 us with a bias, 71 in groups too (with all scores in 64 bits,
// as a softmax with a bias and more than 28 picks have them, 340 to 480; 37 without a bias and groups).
template <typename TL>
__global__ void __launch_bounds__(32 * kRouteWarps) moe_route_any_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ __align__(16) uint64_t choice[];
  const int warp = threadIdx.x >> 5;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp; t < a.T; t += gridDim.x * kRouteWarps) {
    int id;
    float w;
    if (!route_few<TL>(a, t, choice + warp * a.E, id, w)) route_row<TL>(a, t, choice + warp * a.E, 1, id, w);
    put_row<TL>(a, t, id, w, a.counts);
  }
}

// The fast form.  A row is held by LPR lanes of a warp, each expert group by L = LPR / (groups rounded up to a power
// of 2) of them, VPL experts a lane.  A choice score becomes a place on a grid of 2^23 steps over the range that the
// scores can have with these biases, t = 2^23 + 32 + (c - lowest bias) K: a key of 32 bits holds its 23 bits and, below
// them, the expert's slot (ties: the lower one), so that a sorting network of unsigned minima and maxima and one
// maximum over the row a pick choose the experts.  (bf16 logits without a bias need no grid: their own 16 bits order
// them exactly.  A softmax's grid is the row's, up to its largest score: most of them are small.)
//
// What the grid cannot tell apart is found and decided in 64 bits, by all of the CTA's warps when their rows are done (a warp
// alone takes 18 us for a row of 256, most of it this GPU's fp64 exponentials): a row goes there if two neighbours in the order
// of its picks, or a group that stays and one that does not, lie within `near` steps.  Two experts with the same logit
// and the same bias are the exception, as their order is that of their indices in any precision (a router with a bias
// of zeros and bf16 logits has them in every tenth row).  How far t can be off, in steps of R 2^-23, R the grid's
// range: s by 4.3 2^-24 (sigmoid: 1/4 (2^-22 of ex2) + 0.28 2^-24 for the exponent's rounding, one
// unit of the reciprocal and half a unit of the sum) or 36 2^-24 (softmax: ex2, the exponents' roundings weighted by the
// scores, at most log E, the sum's 13), 2.2 or 18 steps; the bias' part 1.5, the sum 0.5.  So two are within 2 x 4.2 or
// 2 x 20.5 steps of their true distance, sums of two within twice that.
//
// Rows with a logit that is NaN or +inf, with fewer experts left than are to be chosen, or with a group that has a single
// one left, go there too.  65536 x 256 normal logits: one row in 1000.
//
// Bound by its instructions (some 600 of a warp a row of 256 in groups, 430 of bf16 without them; 67 to 70% and 84% of the
// issue slots are taken) and by what the rows in 64 bits add at the end (8 us).  65536 x 256, 8 picks: bf16 in 8 groups 56 us,
// without groups 48, without a bias either 29; softmax in groups 77; 64 rows 5.5; 4096 rows 18.
constexpr int kRouteFastWarps = 32;
constexpr int kRouteCluster = 8;
constexpr int kRouteListed = 64;  // rows that a CTA leaves for its end; more are decided where they are met
constexpr float kGrid = 8388608.0f;  // 2^23
// Shared memory, every part a multiple of 16 bytes: a row of 64-bit keys a warp, the CTA's counts, then a warp's lists of
// keys, its rows' picks and their scores.
__host__ __device__ constexpr int route_keys(int E) { return (E + 1) / 2 * 2; }
constexpr int kRouteBatch = 8;  // rows whose picks are worked on at once, at most
template <int VPL>
__host__ __device__ constexpr int route_warp_words(int topk) {
  return (VPL == 8 ? 32 * 12 : 0) + (kRouteBatch * (topk + 2) + 3) / 4 * 4;
}

__device__ __forceinline__ int32_t ld_cluster_s32(uint32_t addr) {
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// The lane's keys by rank, as the row's lanes take them: `next` gives the row's largest that is left (0: none).
template <int VPL, int LPR>
struct KeyList;
template <int LPR>
struct KeyList<8, LPR> {
  uint32_t head, second;
  const uint32_t* at;
  __device__ __forceinline__ void init(uint32_t (&key)[8], uint32_t* list) {
    sort8([&](int a, int b) {
      const uint32_t hi = max(key[a], key[b]), lo = min(key[a], key[b]);
      key[a] = hi;
      key[b] = lo;
    });
    head = key[0];
    second = key[1];
    at = list + 1;
    reinterpret_cast<uint4*>(list)[0] = make_uint4(key[0], key[1], key[2], key[3]);
    reinterpret_cast<uint4*>(list)[1] = make_uint4(key[4], key[5], key[6], key[7]);  // (words 8 and 9 are 0)
  }
  __device__ __forceinline__ uint32_t next() {
    const uint32_t top = row_max<LPR>(head);
    if (head == top && top != 0u) {
      head = second;
      second = *++at;
    }
    return top;
  }
};
template <int LPR>
struct KeyList<16, LPR> {  // unsorted: what is below the last pick, anew each time
  uint32_t key[16];
  uint32_t last;
  __device__ __forceinline__ void init(uint32_t (&k)[16], uint32_t*) {
#pragma unroll
    for (int i = 0; i < 16; ++i) key[i] = k[i];
    last = 0xffffffffu;
  }
  __device__ __forceinline__ uint32_t next() {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, key[i] < last ? key[i] : 0u);
    last = row_max<LPR>(m);
    return last;
  }
};

template <typename TL, int VPL, int LPR, bool KEYS16>
__global__ void __launch_bounds__(32 * kRouteFastWarps, 1) moe_route_kernel(const __grid_constant__ RouteArgs a) {
  constexpr int G = 32 / LPR;  // rows a warp at once
  extern __shared__ __align__(16) uint64_t smem64[];
  __shared__ int64_t list_of_rows[kRouteListed];  // for the end, see there
  __shared__ int listed;
  __shared__ double part_sum[kRouteFastWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int sub = lane % LPR, grp = lane / LPR;
  const uint32_t row_lanes = (LPR == 32 ? 0xffffffffu : (1u << (LPR & 31)) - 1u) << (lane & ~(LPR - 1));
  const int E = a.E, topk = a.topk, per = E / a.groups, L = LPR >> a.log_groups, log_l = 31 - __clz(L);
  const int group = sub >> log_l, base = group * per + (sub & (L - 1)) * VPL;
  const int end = group < a.groups ? group * per + per : 0;
  uint64_t* choice = smem64 + warp * route_keys(E);
  uint32_t* words = reinterpret_cast<uint32_t*>(smem64 + warps * route_keys(E));
  int32_t* cnt = reinterpret_cast<int32_t*>(words);
  uint32_t* mine = words + (E + 3) / 4 * 4 + warp * route_warp_words<VPL>(topk);
  uint32_t* list = mine + lane * 12;
  uint32_t* picks = mine + (VPL == 8 ? 32 * 12 : 0);  // [rows][topk]
  float2* info = reinterpret_cast<float2*>(picks + (kRouteBatch * topk + 1) / 2 * 2);  // a softmax's maximum and 1 / sum
  if constexpr (VPL == 8) list[8] = list[9] = 0u;
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  if (threadIdx.x == 0) listed = 0;
  __syncthreads();
  const TL* logits = static_cast<const TL*>(a.logits);
  const bool scored = !KEYS16 || a.groups > 1;  // whether the choice needs the scores

  // the grid, and the biases' places on it (-inf: no expert there)
  float low = INFINITY, high = -INFINITY;
  bool all_exact = false;
  if (a.bias) {
    for (int e = lane; e < E; e += 32) {
      const float b = a.bias[e];
      if (!(b < INFINITY)) all_exact = true;
      else if (b > -INFINITY) low = fminf(low, b), high = fmaxf(high, b);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      low = fminf(low, __shfl_xor_sync(0xffffffffu, low, off));
      high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, off));
    }
    all_exact = __any_sync(0xffffffffu, all_exact);
  }
  if (!(low <= high)) low = high = 0.0f;
  const float range = 1.0f + (high - low);
  // Biases this far above their range round scores off in the 64-bit sums, and the grid, which starts at the lowest, does not.
  all_exact |= !(fmaxf(fabsf(low), fabsf(high)) <= range * 0x1p20f) || !(range < INFINITY);
  const float K = __fdiv_rn(kGrid - 64.0f, range);
  const float near = a.softmax ? 48.0f : 12.0f;  // steps (see above)
  float place[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float b = base + i < end ? (a.bias ? a.bias[base + i] : 0.0f) : -INFINITY;
    place[i] = a.softmax ? b - low : kGrid + 32.0f + (b - low) * K;
  }

  const int64_t stride = static_cast<int64_t>(gridDim.x) * warps * G;
  int64_t t0 = (static_cast<int64_t>(blockIdx.x) * warps + warp) * G;
  Raw8<TL> next[VPL / 8];
  auto fetch = [&](int64_t at) {
    const TL* row = logits + (at + grp < a.T ? at + grp : a.T - 1) * a.ldl;
#pragma unroll
    for (int v = 0; v < VPL / 8; ++v) {
      const int c = base + 8 * v;
      if (a.vec && c + 8 <= end) {
        next[v].load(row + c);
      } else {
        TL f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < end ? row[c + i] : from_f32<TL>(0.0f);
        next[v].set(f);
      }
    }
  };
  // Picks, scores and results take a lane each, `seg` lanes a row: a whole warp's row waits for others to be worked on
  // together (65536 x 256, 8 picks: one at a time took a third more instructions).
  const int log_seg = topk == 1 ? 0 : 32 - __clz(topk - 1), per_pass = 32 >> log_seg;
  const int batch = LPR == 32 ? min(per_pass, kRouteBatch) : G;
  const uint32_t least = KEYS16 ? 1u : 512u;  // keys below stand for no expert
  auto expert = [&](uint32_t k) {
    const int slot = KEYS16 ? 0xFFFF - static_cast<int>(k & 0xFFFFu) : 511 - static_cast<int>(k & 511u);
    const int l = slot / VPL;
    return min((l >> log_l) * per + (l & (L - 1)) * VPL + slot % VPL, E - 1);  // (a void key's slot is no expert's)
  };
  // whether two experts have the same logit and the same bias
  auto alike = [&](const TL* row, uint32_t p, uint32_t q) {
    const int x = expert(p), y = expert(q);
    return to_f32(row[x]) == to_f32(row[y]) && (!a.bias || a.bias[x] == a.bias[y]);
  };
  auto close = [&](uint32_t hi, uint32_t lo) { return lo >= least && (hi >> 9) - (lo >> 9) <= static_cast<uint32_t>(near); };
  int waiting = 0;
  uint32_t exact_rows = 0;  // of those that wait, a bit each
  int64_t tb = t0;          // the first of them
  if (t0 < a.T) fetch(t0);
  for (; t0 < a.T; t0 += stride) {
    const TL* row = logits + (t0 + grp < a.T ? t0 + grp : a.T - 1) * a.ldl;
    uint32_t* pick = picks + (LPR == 32 ? waiting : grp) * topk;
    float f[VPL];
    uint32_t key[VPL];
#pragma unroll
    for (int v = 0; v < VPL / 8; ++v) next[v].get(reinterpret_cast<float2(&)[4]>(f[8 * v]));
    if constexpr (KEYS16) {
#pragma unroll
      for (int v = 0; v < VPL / 8; ++v) {
        const uint32_t* w = &next[v].v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t k = order_key2(w[i]), c = 0xFFFFu - static_cast<uint32_t>(sub * VPL + 8 * v + 2 * i);
          key[8 * v + 2 * i] = __byte_perm(k, c, 0x1054);          // the low key over the slot
          key[8 * v + 2 * i + 1] = __byte_perm(k, c - 1u, 0x3254);  // the high one
        }
      }
      if (base + VPL > end) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) key[i] = base + i < end ? key[i] : 0u;
      }
    }
    if (t0 + stride < a.T) fetch(t0 + stride);
    float2 odds = make_float2(0.0f, 0.0f);  // NaN where a logit is not finite
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i)
      odds = __ffma2_rn(make_float2(f[2 * i], f[2 * i + 1]), make_float2(0.0f, 0.0f), odds);
    const bool some_odd = __any_sync(0xffffffffu, odds.x + odds.y != 0.0f);
    bool exact = all_exact;
    if (some_odd) {
      bool bad = false;
#pragma unroll
      for (int i = 0; i < VPL; ++i) bad |= !(f[i] < INFINITY);
      exact |= (__ballot_sync(0xffffffffu, bad) & row_lanes) != 0u;
    }
    float mx = 0.0f, inv = 1.0f;
    float c[VPL];  // the choice scores' places
    if (a.softmax) {
      if (base + VPL > end) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) f[i] = base + i < end ? f[i] : -INFINITY;
      }
      mx = f[0];
#pragma unroll
      for (int i = 1; i < VPL; ++i) mx = fmaxf(mx, f[i]);
      mx = row_max<LPR>(mx);
      if (mx == -INFINITY) mx = 0.0f;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        c[i] = exp2_approx((f[i] - mx) * 1.4426950408889634f);
        s += c[i];
      }
      s = row_sum<LPR>(s);
      inv = s == 0.0f ? 0.0f : __fdiv_rn(1.0f, s);
      // the row's own grid: its largest score is inv
      const float k_row = (kGrid - 64.0f) * recip_approx(inv + (high - low)), by = k_row * inv;
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = fmaf(c[i], by, fmaf(place[i], k_row, kGrid + 32.0f));
    } else if (scored) {
#pragma unroll
      for (int i = 0; i < VPL; i += 2) {
        float2 v = __fmul2_rn(make_float2(f[i], f[i + 1]), make_float2(-1.4426950408889634f, -1.4426950408889634f));
        v = __fadd2_rn(make_float2(exp2_approx(v.x), exp2_approx(v.y)), make_float2(1.0f, 1.0f));
        v = __ffma2_rn(make_float2(recip_approx(v.x), recip_approx(v.y)), make_float2(K, K),
                       make_float2(place[i], place[i + 1]));
        c[i] = v.x, c[i + 1] = v.y;
      }
    }
    if (some_odd && scored) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) c[i] = f[i] == -INFINITY ? -INFINITY : c[i];
    }
    if (KEYS16 && some_odd) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = f[i] == -INFINITY ? 0u : key[i];
    }
    if constexpr (!KEYS16) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = __float_as_uint(c[i]) * 512u + (511u - static_cast<uint32_t>(sub * VPL + i));
    }
    if (a.groups > 1) {
      float first = c[0], second = -INFINITY;
#pragma unroll
      for (int i = 1; i < VPL; ++i) {
        second = fmaxf(second, fminf(first, c[i]));
        first = fmaxf(first, c[i]);
      }
      for (int off = 1; off < L; off <<= 1) {
        const float o1 = __shfl_xor_sync(0xffffffffu, first, off), o2 = __shfl_xor_sync(0xffffffffu, second, off);
        second = fmaxf(fmaxf(second, o2), fminf(first, o1));
        first = fmaxf(first, o1);
      }
      const float sum = per == 1 ? first - kGrid : (first - kGrid) + (second - kGrid);
      // the best groups one after the other (a group's lanes have the same key); ties and what lies near a tie at the
      // border go to route_row
      uint32_t g = group < a.groups && sum > -INFINITY ? (static_cast<uint32_t>(sum) << 5) + 31u - group : 0u;
      exact |= (__ballot_sync(0xffffffffu, group < a.groups && g == 0u) & row_lanes) != 0u;
      uint32_t worst = 0u;
      bool stays = false;
      for (int i = 0; i < a.kept; ++i) {
        worst = row_max<LPR>(g);
        stays |= g == worst;
        g = g == worst ? 0u : g;
      }
      const uint32_t out = row_max<LPR>(g);
      exact |= out != 0u && (worst >> 5) - (out >> 5) <= 2u * static_cast<uint32_t>(near);
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = stays ? key[i] : 0u;
    }
    KeyList<VPL, LPR> keys;
    keys.init(key, list);
    uint32_t last = 0u;
#pragma unroll 2
    for (int j = 0; j < topk; ++j) {
      last = keys.next();
      if (sub == 0) pick[j] = last;
    }
    exact |= last < least;
    if constexpr (!KEYS16) {  // the last one that is taken and the first that is not
      uint32_t after = keys.next();
      bool open = close(last, after);
      while (__any_sync(0xffffffffu, open)) {  // those that are alike, down to one that lies further off
        const bool same = open && alike(row, last, after);
        exact |= open && !same;
        last = after;
        after = keys.next();
        open = same && close(last, after);
      }
    }
    if (sub == 0) info[LPR == 32 ? waiting : grp] = make_float2(mx, inv);
    if constexpr (LPR == 32) {
      exact_rows |= exact ? 1u << waiting : 0u;
      if (++waiting < batch && t0 + stride < a.T) continue;
    } else {
      const uint32_t e = __ballot_sync(0xffffffffu, exact);
      exact_rows = __ballot_sync(0xffffffffu, lane < G && (e >> (lane * LPR & 31) & 1u));
      waiting = static_cast<int>(min(static_cast<int64_t>(G), a.T - t0));
      tb = t0;
    }
    __syncwarp();
    const int64_t step = LPR == 32 ? stride : 1;
    for (int r0 = 0; r0 < waiting; r0 += per_pass) {
      const int r = r0 + (lane >> log_seg), j = lane & ((1 << log_seg) - 1);
      const bool has = r < waiting && j < topk;
      const int64_t t = tb + (r < waiting ? r : 0) * step;
      int id = 0;
      float w = 0.0f, l = -INFINITY;
      bool unsure = false;
      if (has) {
        const TL* at = logits + t * a.ldl;
        const uint32_t k = picks[r * topk + j];
        id = expert(k);
        l = to_f32(at[id]);
        w = route_score(a, l, info[r].x, info[r].y);
        if (!KEYS16 && j + 1 < topk) {
          const uint32_t q = picks[r * topk + j + 1];
          unsure = close(k, q) && !alike(at, k, q);
        }
      }
      const uint32_t u = __ballot_sync(0xffffffffu, unsure);
      if (u) {
        const uint32_t seg = log_seg == 5 ? 0xffffffffu : (1u << (1 << log_seg)) - 1u;
        exact_rows |= __ballot_sync(0xffffffffu, lane < per_pass && (u >> (lane << log_seg & 31) & seg)) << r0;
      }
      auto seg_sum = [&](float v) {
        for (int off = 1; off < 1 << log_seg; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        return v;
      };
      if (a.renorm) {
        float all = seg_sum(w);
        const bool small = has && !(all >= kRouteSmall);
        if (__any_sync(0xffffffffu, small)) {
          const float share = route_share(a, l, route_top(a, l, 1 << log_seg)), sum = seg_sum(share);
          if (small) w = share, all = sum;
        }
        w *= recip_approx(all);
      }
      if (has && !(exact_rows >> r & 1u)) {
        const bool real = !a.mask || a.mask[t];
        a.ids[t * topk + j] = id;
        a.weights[t * topk + j] = real ? w * a.scale : 0.0f;
        if (real) atomicAdd(cnt + id, 1);  // whole numbers: the order does not matter
      }
    }
    exact_rows &= (1u << waiting) - 1u;  // (waiting <= 8)
    while (exact_rows) {
      const int64_t at = tb + (__ffs(exact_rows) - 1) * step;
      exact_rows &= exact_rows - 1;
      int place = 0;
      if (lane == 0) place = atomicAdd(&listed, 1);
      place = __shfl_sync(0xffffffffu, place, 0);
      if (place < kRouteListed) {
        if (lane == 0) list_of_rows[place] = at;
        continue;
      }
      int id;
      float w;
      route_row<TL>(a, at, choice, RowShares(E, warps, warp).parts, id, w);
      put_row<TL>(a, at, id, w, cnt);
    }
    __syncwarp();
    waiting = 0;
    tb = t0 + stride;
  }
  __syncthreads();
  // the listed rows
  const RowShares share(E, warps, warp);
  for (int r0 = 0, n = min(listed, kRouteListed); r0 < n; r0 += share.at_once) {
    const bool mine_too = share.some() && r0 + share.slot < n;
    const int64_t t = list_of_rows[min(r0 + share.slot, n - 1)];
    uint64_t* key = smem64 + share.slot * route_keys(E);
    const ExactRow<TL> r(a, t);
    double inv = 1.0;
    if (a.softmax && r.scored()) {
      double sum = 0.0;
      if (mine_too)
        for (int e = share.part * 32 + lane; e < E; e += share.parts * 32) sum += r.exponential(e);
      sum = warp_sum(sum);
      if (lane == 0) part_sum[warp] = sum;
      __syncthreads();
      sum = 0.0;
      if (mine_too)
        for (int i = 0; i < share.parts; ++i) sum += part_sum[share.first() + i];
      inv = sum == 0.0 ? 0.0 : 1.0 / sum;
    }
    if (mine_too && r.scored())
      for (int e = share.part * 32 + lane; e < E; e += share.parts * 32) key[e] = r.key(e, r.exponential(e), inv);
    __syncthreads();
    if (mine_too && share.part == 0) {
      int id;
      float w;
      route_choose<TL>(a, t, key, r.mx, inv, id, w);
      put_row<TL>(a, t, id, w, cnt);
    }
    __syncthreads();
  }
  if (a.single) {  // one cluster: each CTA joins a share of the counts
    cluster_sync();
    const int ranks = static_cast<int>(gridDim.x), each = (E + ranks - 1) / ranks, lo = blockIdx.x * each;
    for (int e = lo + static_cast<int>(threadIdx.x); e < min(E, lo + each); e += blockDim.x) {
      int32_t n = 0;
      for (int r = 0; r < ranks; ++r) n += ld_cluster_s32(mapa_shared(smem_u32(cnt + e), r));
      a.counts[e] = n;
    }
    cluster_sync();  // (nobody leaves while its counts may still be read)
    return;
  }
  griddep_wait();  // the counts are zero
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    if (cnt[e]) atomicAdd(a.counts + e, cnt[e]);
}

__global__ void moe_route_zero_kernel(int32_t* counts, int32_t E) {
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < E; e += blockDim.x) counts[e] = 0;
}

// How a row falls into lanes: VPL experts a lane (8 or 16; 0: the general form), LPR lanes a row.
struct RouteForm {
  int vpl, lpr, log_groups;
};
int ceil_log2(int v) {
  int k = 0;
  while (1 << k < v) ++k;
  return k;
}
RouteForm route_form(int E, int groups) {
  const int per = E / groups, g = ceil_log2(groups);
  for (int vpl = 8; vpl <= 16; vpl *= 2) {
    const int lpr = g + ceil_log2((per + vpl - 1) / vpl);
    if (lpr <= 5) return {vpl, vpl == 16 ? 32 : std::max(4, 1 << lpr), g};
  }
  return {0, 32, g};
}

template <typename TL, int VPL, int LPR, bool KEYS16>
int route_launch(const RouteArgs& a, const DeviceInfo* dev, cudaStream_t s) {
  constexpr int G = 32 / LPR;
  const int64_t groups = (a.T + G - 1) / G;
  // Few rows: one cluster, which joins the counts itself.  More: the counts are zeroed by a launch before, under whose
  // end this one starts, and added up.
  const bool single = groups <= kRouteCluster * 16;
  const int64_t ctas = single ? std::min<int64_t>(kRouteCluster, groups) : std::min<int64_t>((groups + 3) / 4, dev->sm_count);
  const int warps = static_cast<int>(std::min<int64_t>(kRouteFastWarps, (groups + ctas - 1) / ctas));
  const size_t smem = static_cast<size_t>(warps) * (8 * route_keys(a.E) + 4 * route_warp_words<VPL>(a.topk)) +
                      static_cast<size_t>((a.E + 3) / 4 * 4) * 4;
  auto kernel = moe_route_kernel<TL, VPL, LPR, KEYS16>;
  const int st = allow_shared_memory(reinterpret_cast<const void*>(kernel), smem + 2048);  // (and what is static)
  if (st != FP8G_OK) return st;
  if (!single) moe_route_zero_kernel<<<1, 256, 0, s>>>(a.counts, a.E);
  RouteArgs args = a;
  args.single = single ? 1 : 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (single) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  return FP8G_OK;
}
template <typename TL, bool KEYS16>
int route_any_lanes(const RouteArgs& a, const RouteForm& f, const DeviceInfo* dev, cudaStream_t s) {
  if (f.vpl == 16) return route_launch<TL, 16, 32, KEYS16>(a, dev, s);
  switch (f.lpr) {
    case 4: return route_launch<TL, 8, 4, KEYS16>(a, dev, s);
    case 8: return route_launch<TL, 8, 8, KEYS16>(a, dev, s);
    case 16: return route_launch<TL, 8, 16, KEYS16>(a, dev, s);
    default: return route_launch<TL, 8, 32, KEYS16>(a, dev, s);
  }
}

// The gradient.  A row's scores in LPR lanes, 8 V logits each (its chosen ones alone for a sigmoid); its choices in `seg` lanes, a
// choice each; then every expert's value is written, and over it those of the chosen ones.  Bound by memory.
// 65536 x 256 fp32: softmax 30 us (68% of the copy rate), sigmoid 20 (55%); 16383 x 160 softmax 8.4 us (a lane's logits one by
// one and read three times: 18).
constexpr int kRouteGradWarps = 8;
template <typename TL, int V, int LPR>
__global__ void __launch_bounds__(32 * kRouteGradWarps) moe_route_backward_kernel(const RouteArgs a) {
  constexpr int G = 32 / LPR, VPL = 8 * V;
  __shared__ float2 s_info[kRouteGradWarps][G];  // a row's maximum and 1 / sum; then q, and whether it is a real token's
  __shared__ float s_value[kRouteGradWarps][32 * G];
  __shared__ int32_t s_id[kRouteGradWarps][32 * G];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, grp = lane / LPR;
  const int E = a.E, topk = a.topk;
  const int log_seg = topk == 1 ? 0 : 32 - __clz(topk - 1), per_pass = 32 >> log_seg;
  float2* info = s_info[warp];
  float* value = s_value[warp];
  int32_t* ids = s_id[warp];
  const TL* logits = static_cast<const TL*>(a.logits);
  TL* dlogits = static_cast<TL*>(a.dlogits);
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteGradWarps + warp) * G; t0 < a.T;
       t0 += static_cast<int64_t>(gridDim.x) * kRouteGradWarps * G) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(G), a.T - t0));
    const int64_t t = t0 + (grp < rows ? grp : 0);
    float2 f[VPL / 2];
    if (a.softmax) {
#pragma unroll
      for (int v = 0; v < V; ++v) {  // eights of a row go to its lanes in turn
        Logits<TL, 8> l;
        l.load(logits + t * a.ldl, 8 * (v * LPR + sub), E, a.vec);
        l.get(reinterpret_cast<float2(&)[4]>(f[4 * v]));
      }
      float mx = f[0].x;
#pragma unroll
      for (int i = 0; i < VPL / 2; ++i) mx = fmaxf(mx, fmaxf(f[i].x, f[i].y));
      mx = row_max<LPR>(mx);
      if (mx == -INFINITY) mx = 0.0f;
      const float sum = row_sum<LPR>(exp_below(f, mx));
      const float inv = sum == 0.0f ? 0.0f : recip_approx(sum);
#pragma unroll
      for (int i = 0; i < VPL / 2; ++i) f[i] = __fmul2_rn(f[i], make_float2(inv, inv));
      if (sub == 0) info[grp] = make_float2(mx, inv);
      __syncwarp();
    }
    for (int r0 = 0; r0 < rows; r0 += per_pass) {
      const int r = r0 + (lane >> log_seg), j = lane & ((1 << log_seg) - 1);
      const bool has = r < rows && j < topk;
      const int64_t at = t0 + (r < rows ? r : 0);
      const bool real = r < rows && (!a.mask || a.mask[at]);
      int id = -1;
      float d = 0.0f, s = 0.0f, l = -INFINITY, slope = 0.0f;
      if (has) {
        id = a.ids[at * topk + j];
        if (id < 0 || id >= E) id = -1;
      }
      if (id >= 0) {
        d = a.dweights[at * topk + j] * a.scale;
        l = to_f32(logits[at * a.ldl + id]);
        if (a.softmax) {
          s = exp_below(l, info[r].x) * info[r].y;
        } else {
          const float x = exp_below(-fabsf(l), 0.0f), y = recip_approx(1.0f + x);
          s = l >= 0.0f ? y : x * y;
          slope = x * y * y;  // s (1 - s)
        }
      }
      auto seg_sum = [&](float v) {
        for (int off = 1; off < 1 << log_seg; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        return v;
      };
      float p = s;
      bool small = false;
      if (a.renorm) {
        float sum = seg_sum(s), inner = seg_sum(d * s);
        small = !(sum >= kRouteSmall);
        if (__any_sync(0xffffffffu, has && small)) {
          const float share = route_share(a, l, route_top(a, l, 1 << log_seg)), all = seg_sum(share), in = seg_sum(d * share);
          if (small) p = share, sum = all, inner = in;
        }
        const float by = sum == 0.0f ? 0.0f : recip_approx(sum);
        d = id < 0 ? 0.0f : d - inner * by;
        // Over a small sum S, d stays S times the scores' gradient, and what it is multiplied by is divided by S.
        if (small) p *= by, slope = p;  // (1 - s is 1)
        else d *= by;
      }
      const float q = a.softmax ? seg_sum(d * p) : 0.0f;
      // the same expert twice gets the sum of both
      const uint32_t same = __match_any_sync(0xffffffffu, id < 0 ? -1 : r * kRouteMaxExperts + id);
      if (__any_sync(0xffffffffu, id >= 0 && __popc(same) > 1)) {
        float all = 0.0f;
        for (int i = 0; i < 32; ++i) {
          const float v = __shfl_sync(0xffffffffu, d, i);
          if (same >> i & 1u) all += v;
        }
        d = all;
      }
      if (has) {
        ids[r * topk + j] = real ? id : -1;
        value[r * topk + j] = !a.softmax ? d * slope : small ? p * d - s * q : s * (d - q);
      }
      __syncwarp();
      if (r < rows && j == 0) info[r] = make_float2(q, real ? 1.0f : 0.0f);
    }
    __syncwarp();
    if (grp < rows) {
      const float2 row = info[grp];
      const bool some = a.softmax && row.y != 0.0f;
      TL* out = dlogits + t * a.ldd;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (v * LPR + sub);
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = some ? -row.x * (i & 1 ? f[4 * v + i / 2].y : f[4 * v + i / 2].x) : 0.0f;
        if (a.vec && c + 8 <= E) {
          store8_stream(out + c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < E) out[c + i] = from_f32<TL>(o[i]);
        }
      }
    }
    __syncwarp();
    for (int i = lane; i < rows * topk; i += 32)
      if (ids[i] >= 0) dlogits[(t0 + i / topk) * a.ldd + ids[i]] = from_f32<TL>(value[i]);
    __syncwarp();
  }
}

// The same for more experts than lanes hold.
// A warp a row; lane j < topk has the row's j-th choice.
template <typename TL>
__global__ void __launch_bounds__(256) moe_route_backward_any_kernel(const RouteArgs a) {
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
    float mx = 0.0f, inv = 1.0f, s = 0.0f, slope = 0.0f;
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
    float p = s;
    bool small = false;
    if (a.renorm) {  // (as above)
      float sum = warp_sum(s), inner = warp_sum(d * s);
      small = !(sum >= kRouteSmall);
      if (small) {
        p = route_share(a, l, route_top(a, l, 32));
        sum = warp_sum(p), inner = warp_sum(d * p);
      }
      const float by = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      d -= inner * by;
      if (small) p *= by, slope = p;
      else d *= by;
    }
    if (id < 0) d = 0.0f;
    const float q = a.softmax ? warp_sum(d * p) : 0.0f;
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
    if (id >= 0 && real) out[id] = from_f32<TL>(!a.softmax ? d * slope : small ? p * d - s * q : s * (d - q));
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
  RouteArgs a{};
  a.logits = logits, a.bias = bias, a.mask = token_mask, a.ids = topk_ids, a.weights = topk_weights, a.counts = counts;
  a.T = T, a.ldl = ldl, a.E = E, a.topk = topk, a.groups = groups, a.kept = topk_groups, a.softmax = score;
  a.renorm = renormalize, a.scale = scale;
  const RouteForm f = route_form(E, groups);
  a.log_groups = f.log_groups;
  a.vec = aligned16(logits) && (T == 1 || ldl % 8 == 0) && E / groups % 8 == 0;
  if (f.vpl && T > 0) {
    if (dtype == FP8G_F32) return route_any_lanes<float, false>(a, f, dev, s);
    return bias ? route_any_lanes<__nv_bfloat16, false>(a, f, dev, s) : route_any_lanes<__nv_bfloat16, true>(a, f, dev, s);
  }
  if (cudaMemsetAsync(counts, 0, static_cast<size_t>(E) * 4, s) != cudaSuccess) {
    cudaGetLastError();
    return FP8G_ERR_CUDA;
  }
  if (T == 0) return FP8G_OK;
  const size_t smem = sizeof(uint64_t) * kRouteWarps * static_cast<size_t>(E);
  auto kernel = dtype == FP8G_F32 ? moe_route_any_kernel<float> : moe_route_any_kernel<__nv_bfloat16>;
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
  if (!logits || !topk_ids || !dweights || !dlogits || (dlogits == logits && T > 1 && ldd != ldl)) return FP8G_ERR_INVALID_ARG;
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
  a.vec = aligned16(logits) && aligned16(dlogits) && (T == 1 || (ldl % 8 == 0 && ldd % 8 == 0));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int lanes = E <= 256 ? 8 : 16;  // a row
  const int64_t rows = E <= 512 ? kRouteGradWarps * 32 / lanes : 8;
  const unsigned ctas = static_cast<unsigned>(std::min<int64_t>((T + rows - 1) / rows, 8 * dev->sm_count));
  using B = __nv_bfloat16;
  auto pick = [&](auto f32, auto bf16) { return dtype == FP8G_F32 ? f32 : bf16; };
  auto kernel = E <= 64    ? pick(moe_route_backward_kernel<float, 1, 8>, moe_route_backward_kernel<B, 1, 8>)
                : E <= 128 ? pick(moe_route_backward_kernel<float, 2, 8>, moe_route_backward_kernel<B, 2, 8>)
                : E <= 256 ? pick(moe_route_backward_kernel<float, 4, 8>, moe_route_backward_kernel<B, 4, 8>)
                : E <= 512 ? pick(moe_route_backward_kernel<float, 4, 16>, moe_route_backward_kernel<B, 4, 16>)
                           : pick(moe_route_backward_any_kernel<float>, moe_route_backward_any_kernel<B>);
  kernel<<<ctas, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? FP8G_OK : FP8G_ERR_CUDA;
}
