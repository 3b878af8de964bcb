// Routing of tokens to experts (hc_expert_route).
//
// A warp takes a token. The experts of a group lie in L lanes, L the largest power of two for which all groups fit a warp, so
// that what is compared stays in registers: a group's best values come together over L lanes, and a choice is one maximum
// over the warp of keys that have the value's upper bits and the index.
//
// Order: which of two values is the larger must not hang on a rounding. Without a bias the order is that of the logits
// themselves, exactly (but beside a logit of plus infinity all others of a softmax have the score 0). Otherwise values are formed in fp32 first; a comparison is trusted if the difference is larger than
// both errors, which `score_error` bounds by the arithmetic below, and values that fp32 cannot tell apart (groups, neighbours
// in the order, the last that is taken and the first that is not) are ordered by themselves in fp64, which runs at 1/64 of
// fp32's rate here: doing all rows that way would cost ten times the rest.
//
// Bound: latency, not bytes. 8191 tokens and 256 experts in eight groups, two of whose values count, take 15.7 us with their bias
// (8.9 MB: 1.3 us): issue slots are active in 41% of the cycles (58% of those in which an SM has warps), the ALU in 54% of the
// latter; a warp's top_k maxima wait for one another, and 2048 CTAs of 64 registers a thread are 1.7 rounds. One token and 128 experts 3.3 us, a launch. (A maximum and then the
// lowest index that has it: 27 us. All of a row again in fp64 where two neighbours are too close: 19.)
#include <cmath>

#include "hc_common.cuh"
#include "hc_experts_internal.h"

namespace hc {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kFull = 0xffffffffu;
using u64 = unsigned long long;

struct RouteArgs {
  const void* logits;
  const float* bias;
  const int32_t* live;
  int32_t* ids;
  float* weights;
  int64_t tokens, stride;
  int experts, top_k, groups, top_groups, best, each, lanes;  // lanes: of one group
  int sigmoid, renormalise, dtype;
  float scale;
};

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t t, int e) {
  const int64_t at = t * a.stride + e;
  float x;
  if (a.dtype == HC_F32)
    x = static_cast<const float*>(a.logits)[at];
  else if (a.dtype == HC_F16)
    x = __half2float(static_cast<const __half*>(a.logits)[at]);
  else
    x = __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]);
  return x != x ? -INFINITY : x;
}

// Integers in the order of the numbers, above 0 (which stands for none).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // (-0 becomes 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long key_of(double v) {
  const unsigned long long u = __double_as_longlong(v + 0.0), top = 1ull << 63;
  return u & top ? ~u : u | top;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kFull, k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long k) {
  const uint32_t hi = __reduce_max_sync(kFull, static_cast<uint32_t>(k >> 32));
  const uint32_t lo = __reduce_max_sync(kFull, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return static_cast<unsigned long long>(hi) << 32 | lo;
}

template <typename F> struct Num;
template <> struct Num<float> {
  using Key = uint32_t;
  static __device__ __forceinline__ float exp(float x) { return expf(x); }
};
template <> struct Num<double> {
  using Key = unsigned long long;
  static __device__ __forceinline__ double exp(double x) { return ::exp(x); }
};

template <typename F> __device__ __forceinline__ F sigmoid_of(F x) { return F(1) / (F(1) + Num<F>::exp(-x)); }

// exp(x - m), 1 at the maximum (an infinite one among them).
template <typename F> __device__ __forceinline__ F exp_below(F x, F m) { return x == m ? F(1) : Num<F>::exp(x - m); }

template <typename F> __device__ __forceinline__ F warp_total(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// How far an fp32 score can be off, of scores up to 1. Sigmoid: ex2.approx is within 4 u (u = 2^-24), which counts with
// e / (1 + e), its argument's rounding adds |x| u e / (1 + e)^2, less than u, the sum 1 u, the reciprocal 2 u. Softmax: 4 u,
// the argument's two roundings less than u, the sum VPL + 5 roundings and its terms' errors, reciprocal and product 3 u.
constexpr float kU = 5.9604645e-08f;
template <int VPL> __device__ __forceinline__ float score_error(bool sigmoid) { return sigmoid ? 8 * kU : (VPL + 24) * kU; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What is left of a row when its experts are chosen: lane i has the i-th.
struct Choice {
  int id;       // of this lane, -1 past top_k
  float m;      // the largest logit (softmax)
  float total;  // of exp(x - m) (softmax whose weights are not divided by their sum)
};

// The lane's logits, minus infinity for NaN and where it has none.
template <int VPL> __device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t t, int first, int count, float* x) {
  const int64_t at = t * a.stride + first;
  if (a.dtype == HC_F32) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = i < count ? static_cast<const float*>(a.logits)[at + i * a.lanes] : -INFINITY;
  } else if (a.dtype == HC_F16) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      x[i] = i < count ? __half2float(static_cast<const __half*>(a.logits)[at + i * a.lanes]) : -INFINITY;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      x[i] = i < count ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at + i * a.lanes]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] = fmaxf(x[i], -INFINITY);
}

// The two largest values of a group, from those of its lanes.
template <typename F> __device__ __forceinline__ void join_best(const RouteArgs& a, F* a1, F* a2) {
  for (int o = 1; o < a.lanes; o <<= 1) {
    const F b1 = __shfl_xor_sync(kFull, *a1, o), b2 = __shfl_xor_sync(kFull, *a2, o);
    *a2 = fmax(fmax(*a2, b2), fmin(*a1, b1));
    *a1 = fmax(*a1, b1);
  }
}

// Whether this lane's group stays, by the two largest of its values in arithmetic F. `sure` becomes false if fp32 values cannot tell
// that are sums of a score, off by `error`, and a bias, rounded at the size of each: two of them that cancel leave a group's value
// with an error that its own size does not show. So a group's bounds are its value and `best` errors more or less, and 4 u of
// |a1| + |a2| (u of each, u of their sum, and u for the bounds).
template <typename F>
__device__ __forceinline__ bool keep_group(const RouteArgs& a, F a1, F a2, int group, float error, bool* sure) {
  using Key = typename Num<F>::Key;
  const bool in = group < a.groups;
  F value = a.best == 2 && a.each > 1 ? a1 + a2 : a1;
  if (value != value) value = -INFINITY;
  Key k = in ? key_of(value) : Key(0);
  bool kept = false;
  for (int i = 0; i < a.top_groups; ++i) {
    const Key last = warp_max(k);
    const int g = __reduce_min_sync(kFull, k == last ? static_cast<unsigned>(group) : 64u);
    if (group == g) {
      kept = in;
      k = 0;
    }
  }
  if constexpr (sizeof(F) == 4) {
    const float size = value == -INFINITY ? 0.0f : a.best == 2 && a.each > 1 ? fabsf(a1) + fabsf(a2) : fabsf(a1);
    const float reach = a.best * error + 4 * kU * size;
    const bool bounded = reach < INFINITY;
    float out = !in || kept ? -INFINITY : bounded ? value + reach : INFINITY;  // the upper bound of those that go
    float stay = !(in && kept) ? -INFINITY : bounded ? reach - value : INFINITY;  // minus the lower one of those that stay
    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(out));
    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(stay));
    *sure = error == 0.0f || out == -INFINITY || -stay > out;
  }
  return kept;
}

// The sum of exp(x - m) over a row in fp64.
__device__ __forceinline__ double exact_total(const RouteArgs& a, int64_t t, float m) {
  double total = 0;
  for (int e = threadIdx.x & 31; e < a.experts; e += 32) total += m == -INFINITY ? 0.0 : exp_below<double>(load_logit(a, t, e), m);
  return warp_total(total);
}
// What stands for a score where logits are compared: the logit, but for the zeros beside an infinite one in a softmax.
__device__ __forceinline__ float order_logit(const RouteArgs& a, float x, float m) {
  return !a.sigmoid && m == INFINITY && x != INFINITY ? 0.0f : x;
}
// What is compared, in fp64 (with the logits in place of scores where that is the same order).
__device__ __forceinline__ double exact_value(const RouteArgs& a, int64_t t, int e, float m, double total, bool logits) {
  const float x = load_logit(a, t, e);
  double v = logits ? order_logit(a, x, m) : x;
  if (!logits) v = a.sigmoid ? sigmoid_of<double>(v) : m == -INFINITY ? 0.0 : exp_below<double>(v, m) / total;
  if (a.bias != nullptr) v += static_cast<double>(a.bias[e]);
  return v != v ? -INFINITY : v;
}

// Whether this lane's group stays, in fp64. `pending` has the lane's elements that can be among its group's two largest.
__device__ __noinline__ bool keep_group_exactly(const RouteArgs& a, int64_t t, float m, int group, int first, u64 pending) {
  const double total = a.sigmoid ? 1.0 : exact_total(a, t, m);
  double a1 = -INFINITY, a2 = -INFINITY;
  while (__any_sync(kFull, pending != 0)) {
    if (pending != 0) {
      const double v = exact_value(a, t, first + (__ffsll(pending) - 1) * a.lanes, m, total, false);
      a2 = fmax(a2, fmin(a1, v));
      a1 = fmax(a1, v);
      pending &= pending - 1;
    }
  }
  join_best(a, &a1, &a2);
  return keep_group<double>(a, a1, a2, group, 0.0f, nullptr);
}

// All experts of the groups that stay, in fp64.
template <int VPL>
__device__ __noinline__ int choose_exactly(const RouteArgs& a, int64_t t, float m, int first, int count, bool logits) {
  const int lane = threadIdx.x & 31;
  const double total = a.sigmoid || logits ? 1.0 : exact_total(a, t, m);
  unsigned long long key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = i < count ? key_of(exact_value(a, t, first + i * a.lanes, m, total, logits)) : 0;
  int id = -1;
  for (int j = 0; j < a.top_k; ++j) {
    unsigned long long top = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > top) {
        top = key[i];
        at = i;
      }
    const unsigned long long best = warp_max(top);
    const int e = static_cast<int>(
        __reduce_min_sync(kFull, top == best ? static_cast<unsigned>(first + at * a.lanes) : 0x7fffffffu));
    if (lane == j) id = e;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < count && first + i * a.lanes == e) key[i] = 0;
  }
  return id;
}

// Candidates of which some cannot be told apart in fp32, one to a lane: their order in fp64. Lane i gets the i-th.
__device__ __noinline__ int order_exactly(const RouteArgs& a, int64_t t, float m, int id, int candidates, bool logits) {
  const int lane = threadIdx.x & 31;
  const double total = a.sigmoid || logits ? 1.0 : exact_total(a, t, m);
  const double v = lane < candidates ? exact_value(a, t, id, m, total, logits) : -INFINITY;
  int rank = 0;
  for (int i = 0; i < candidates; ++i) {
    const double w = __shfl_sync(kFull, v, i);
    const int e = __shfl_sync(kFull, id, i);
    rank += w > v || (w == v && e < id);
  }
  int got = -1;
  for (int i = 0; i < candidates; ++i) {
    const int e = __shfl_sync(kFull, id, i), at = __shfl_sync(kFull, rank, i);
    if (at == lane) got = e;
  }
  return got;
}

// Choose, in fp32 as far as that can tell.
//
// What is compared is a key and an index in 32 bits, the key's low bits (as many as an index has) giving way to the index,
// lower ones first: a maximum over the warp is then a choice, and the next one the largest below it. Two values are told
// apart if the bounds of what their keys stand for are farther apart than errors reach. Beyond the top_k-th, candidates are
// taken until one is below it for certain; if there are any, or if two of those chosen cannot be told apart, all of them are
// ordered in fp64 (with more than 32, all experts).
template <int VPL> __device__ __forceinline__ void choose(const RouteArgs& a, int64_t t, Choice* out) {
  const int lane = threadIdx.x & 31, group = lane / a.lanes, sub = lane % a.lanes, first = group * a.each + sub;
  const int count = group < a.groups && sub < a.each ? (a.each - sub + a.lanes - 1) / a.lanes : 0;
  const bool by_logit = a.bias == nullptr;  // the order of the scores is that of the logits
  const bool by_group = a.groups > a.top_groups, group_scores = by_group && !(by_logit && a.best == 1);
  const bool whole = !a.sigmoid && !a.renormalise;  // weights that need the sum over all
  float v[VPL], s[VPL];
  load_logits<VPL>(a, t, first, count, v);
  float m = -INFINITY;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(m));
  }
  out->m = m;
  constexpr float kLog2e = 1.44269504f;
  if (!by_logit || group_scores || whole) {
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] = reciprocal(1.0f + ex2(v[i] * -kLog2e));
    } else {
      float total = 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        s[i] = v[i] == m ? 1.0f : whole ? expf(v[i] - m) : ex2((v[i] - m) * kLog2e);
        if (m == -INFINITY || i >= count) s[i] = 0.0f;
        total += s[i];
      }
      total = warp_sum(total);
      out->total = total;
      const float r = total > 0.0f ? __frcp_rn(total) : 0.0f;
#pragma unroll
      for (int i = 0; i < VPL; ++i) s[i] *= r;
    }
  }
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = order_logit(a, v[i], m);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = i < count ? fmaxf(s[i] + a.bias[first + i * a.lanes], -INFINITY) : -INFINITY;
  }
  const float error = score_error<VPL>(a.sigmoid);
  bool kept = group < a.groups;
  if (by_group) {
    float a1 = -INFINITY, a2 = -INFINITY;
    const auto value = [&](int i) { return i >= count ? -INFINITY : by_logit && a.best == 2 ? s[i] : v[i]; };
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      a2 = fmaxf(a2, fminf(a1, value(i)));
      a1 = fmaxf(a1, value(i));
    }
    join_best(a, &a1, &a2);
    bool sure;
    kept = keep_group<float>(a, a1, a2, group, group_scores ? error : 0.0f, &sure);
    if (!sure) {
      const float least = a.best == 2 && a.each > 1 ? a2 : a1, reach = 2 * error + 4 * kU * fabsf(least);
      u64 pending = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i < count && !(value(i) < least - reach)) pending |= 1ull << i;
      kept = keep_group_exactly(a, t, m, group, first, pending);
    }
  }
  const uint32_t low = 0xffffffffu >> __clz(max(a.experts - 1, 1));
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    key[i] = kept && i < count ? (key_of(v[i]) & ~low) | (low - static_cast<uint32_t>(first + i * a.lanes)) : 0u;
  const auto apart = [&](uint32_t above, uint32_t below) {
    // (16-bit logits have nothing in those bits, so that equal ones are equal and in order)
    if (by_logit) return a.dtype != HC_F32 || (above | low) != (below | low);
    const float x = value_of(above & ~low), y = value_of(below | low);
    return y == -INFINITY ? x > y : x - y > 2 * error + 2 * kU * (fabsf(x) + fabsf(y));
  };
  uint32_t mine = 0, last = 0xffffffffu, kth = 0;
  int candidates = 0;
#pragma unroll 1
  for (int j = 0;; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = max(top, key[i] < last ? key[i] : 0u);
    last = __reduce_max_sync(kFull, top);
    if (last == 0 || (j >= a.top_k && apart(kth, last))) break;
    if (j == 32) {
      out->id = choose_exactly<VPL>(a, t, m, first, kept ? count : 0, by_logit);
      return;
    }
    if (lane == j) mine = last;
    if (j == a.top_k - 1) kth = last;
    candidates = j + 1;
  }
  int id = lane < candidates ? static_cast<int>(low - (mine & low)) : -1;
  const uint32_t next = __shfl_down_sync(kFull, mine, 1);
  const bool told = lane + 1 >= candidates || apart(mine, next);
  if (candidates > a.top_k || !__all_sync(kFull, told)) id = order_exactly(a, t, m, id, candidates, by_logit);
  out->id = id;
}

// x - m in two parts, so that the weight of a large logit's neighbour keeps its last bits.
__device__ __forceinline__ float exp_apart(float x, float m) {
  if (x == m) return 1.0f;
  const float d = __fsub_rn(x, m), b = __fsub_rn(d, x);
  const float lo = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(m, b));
  const float e = expf(d);
  return lo == lo ? fmaf(e, lo, e) : e;  // (an infinite logit has no second part)
}

template <int VPL> __global__ void __launch_bounds__(32 * kWarps) route_kernel(RouteArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  int32_t* ids = a.ids + t * a.top_k;
  float* weights = a.weights + t * a.top_k;
  if (a.live != nullptr && t >= *a.live) {
    if (lane < a.top_k) {
      ids[lane] = -1;
      weights[lane] = 0.0f;
    }
    return;
  }
  Choice c;
  choose<VPL>(a, t, &c);
  const float m = c.m;
  const bool mine = lane < a.top_k;
  const float x = mine ? load_logit(a, t, c.id) : -INFINITY;
  float w;
  if (a.renormalise) {
    // the chosen scores against the largest of them, so that none is lost however small they all are
    float top = x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (top == -INFINITY)
      w = 0.0f;
    else if (a.sigmoid)
      w = expf(fminf(x, 0.0f) + fmaxf(-top, 0.0f)) / (1.0f + expf(-fabsf(x)));
    else
      w = exp_apart(x, top);
    if (!mine) w = 0.0f;
    const float sum = warp_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  } else if (a.sigmoid) {
    w = sigmoid_of<float>(x);
  } else {
    w = m == -INFINITY ? 0.0f : exp_apart(x, m) / c.total;
  }
  if (mine) {
    ids[lane] = c.id;
    weights[lane] = w * a.scale;
  }
}

template <int VPL> cudaError_t launch(const RouteArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.tokens + kWarps - 1) / kWarps);
  return launch_pdl(route_kernel<VPL>, dim3(grid), dim3(32 * kWarps), 0, s, 1, a);
}

}  // namespace

cudaError_t launch_expert_route(const hc_expert_route_t& p, cudaStream_t s) {
  RouteArgs a = {p.logits, p.bias,      p.live,   p.experts_out, p.weights_out,      p.tokens, p.logits_stride, p.experts,
                 p.top_k,  p.groups,    p.top_groups, p.group_best, p.experts / p.groups, 32, p.sigmoid,
                 p.renormalise, p.dtype, p.scale};
  if (a.top_groups == a.groups) {  // (no group is left out, so the experts need not lie in groups)
    a.groups = a.top_groups = 1;
    a.each = a.experts;
  }
  while (a.lanes * a.groups > 32) a.lanes >>= 1;
  const int vpl = (a.each + a.lanes - 1) / a.lanes;
  if (vpl <= 1) return launch<1>(a, s);
  if (vpl <= 2) return launch<2>(a, s);
  if (vpl <= 4) return launch<4>(a, s);
  if (vpl <= 8) return launch<8>(a, s);
  if (vpl <= 16) return launch<16>(a, s);
  if (vpl <= 32) return launch<32>(a, s);
  return launch<64>(a, s);
}

}  // namespace hc
