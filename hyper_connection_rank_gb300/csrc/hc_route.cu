// Routing of tokens to experts (hc_expert_route).
//
// A warp takes a token. The experts of a group lie in L lanes, L the largest
// power of two for which all groups fit a warp, so that what is compared stays in
// registers: a group's best values come together over L lanes, and each choice is
// a maximum over a lane's registers, one over the warp and the lowest index that
// has it.
//
// Order: which of two values is the larger must not hang on a rounding. Without a
// bias the order is that of the logits themselves, exactly. Otherwise values are
// formed in fp32 first, and where two neighbours in the order (or the last that is
// taken and the first that is not) are closer than their errors allow, the warp
// does the row again in fp64: `score_error` bounds a score's error by the
// arithmetic below, and a comparison is trusted if the difference is larger than
// both errors. A row in some thousands takes the second pass (fp64 runs at 1/64
// of fp32's rate here, so doing all rows that way would cost ten times the rest).
//
// Bound: latency and issue, not bytes. REPLACE_MEASURED
#include <cmath>

#include "hc_common.cuh"
#include "hc_experts_internal.h"

namespace hc {
namespace {

constexpr int kWarps = 4;
constexpr unsigned kFull = 0xffffffffu;

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

// How far an fp32 score can be off. Softmax: expf is within 2 ulp, x - m rounds once (an error of |d| 2^-24 on exp(d),
// which is below 2^-25 whatever d), the sum adds VPL + 5 roundings and its terms' errors, the quotient 2 more.
// Sigmoid: expf's 2 ulp count with e / (1 + e), the sum and the quotient half an ulp each.
template <int VPL> __device__ __forceinline__ float score_error(bool sigmoid, float s) {
  constexpr float u = 5.9604645e-08f;  // 2^-24
  return sigmoid ? s * (8 * u) : s * ((VPL + 32) * u) + 0.5f * u;
}

// What is left of a row when its experts are chosen: lane i has the i-th.
struct Choice {
  int id;       // of this lane, -1 past top_k
  float total;  // of exp(x - m), where the fp32 pass needed it
};

// Choose in arithmetic F. Returns false if fp32 cannot tell the order.
template <typename F, int VPL>
__device__ __forceinline__ bool choose(const RouteArgs& a, int64_t t, float m, Choice* out) {
  using Key = typename Num<F>::Key;
  constexpr bool kFast = sizeof(F) == 4;
  const int lane = threadIdx.x & 31, group = lane / a.lanes, sub = lane % a.lanes;
  const int first = group * a.each + sub;
  const bool in = group < a.groups;
  const bool by_logit = a.bias == nullptr;              // the order of the scores is that of the logits
  const bool group_scores = a.groups > a.top_groups && !(by_logit && a.best == 1);
  const bool scores = !by_logit || group_scores || (kFast && !a.sigmoid && !a.renormalise);
  F v[VPL];
  F s[VPL];
  F total = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool have = in && sub + i * a.lanes < a.each;
    const F x = have ? F(load_logit(a, t, first + i * a.lanes)) : F(-INFINITY);
    v[i] = x;
    s[i] = 0;
    if (scores) {
      if (a.sigmoid) {
        s[i] = sigmoid_of<F>(x);
      } else {
        s[i] = m == -INFINITY || !have ? F(0) : exp_below<F>(x, F(m));
        total += s[i];
      }
    }
  }
  if (scores && !a.sigmoid) {
    total = warp_total(total);
    const F r = total > F(0) ? F(1) / total : F(0);
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] *= r;
  }
  if (kFast) out->total = static_cast<float>(total);
  if (!by_logit) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const bool have = in && sub + i * a.lanes < a.each;
      v[i] = have ? s[i] + F(a.bias[first + i * a.lanes]) : F(-INFINITY);
      if (v[i] != v[i]) v[i] = F(-INFINITY);
    }
  }
  bool kept = in, sure = true;
  if (a.groups > a.top_groups) {
    F a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const F c = by_logit && a.best == 2 ? (in && sub + i * a.lanes < a.each ? s[i] : F(-INFINITY)) : v[i];
      a2 = fmax(a2, fmin(a1, c));
      a1 = fmax(a1, c);
    }
    for (int o = 1; o < a.lanes; o <<= 1) {
      const F b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
      a2 = fmax(fmax(a2, b2), fmin(a1, b1));
      a1 = fmax(a1, b1);
    }
    F value = a.best == 2 && a.each > 1 ? a1 + a2 : a1;
    if (value != value) value = -INFINITY;
    Key k = in ? key_of(value) : Key(0);
    kept = false;
    Key last = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      last = warp_max(k);
      const int g = __reduce_min_sync(kFull, k == last ? static_cast<unsigned>(group) : 64u);
      if (group == g) {
        kept = in;
        k = 0;
      }
    }
    if constexpr (kFast) {
      if (group_scores) {
        const float x = value_of(last), y = value_of(warp_max(k));
        const float tol = 4.0f * score_error<VPL>(a.sigmoid, 1.0f) + 2.4e-07f * (fabsf(x) + fabsf(y));
        sure = y == -INFINITY || x - y > tol;
      }
    }
  }
  Key key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = kept && sub + i * a.lanes < a.each ? key_of(v[i]) : Key(0);
  Key mine = 0, next = 0;
  int id = -1, next_id = -1;
  for (int j = 0; j <= a.top_k; ++j) {
    Key top = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > top) {
        top = key[i];
        at = i;
      }
    const Key best = warp_max(top);
    const int e = static_cast<int>(
        __reduce_min_sync(kFull, top == best ? static_cast<unsigned>(first + at * a.lanes) : 0x7fffffffu));
    if (j == a.top_k) {
      next = best;
      next_id = e;
      break;
    }
    if (lane == j) {
      mine = best;
      id = e;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (first + i * a.lanes == e && in) key[i] = 0;
  }
  out->id = id;
  if constexpr (kFast) {
    if (!by_logit) {
      // each chosen value against the next one in the order
      Key below = __shfl_down_sync(kFull, mine, 1);
      int below_id = __shfl_down_sync(kFull, id, 1);
      if (lane == a.top_k - 1) {
        below = next;
        below_id = next_id;
      }
      if (lane < a.top_k && below != 0) {
        const float x = value_of(mine), y = value_of(below);
        float err[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float l = load_logit(a, t, i ? below_id : id);
          const float sc = a.sigmoid ? sigmoid_of<float>(l) : total > 0.0f ? exp_below<float>(l, m) / total : 0.0f;
          err[i] = score_error<VPL>(a.sigmoid, sc);
        }
        const float tol = err[0] + err[1] + 5.9604645e-08f * (fabsf(x) + fabsf(y));
        if (y != -INFINITY && !(x - y > tol)) sure = false;
      }
    }
    return __all_sync(kFull, sure);
  }
  return true;
}

template <int VPL> __device__ __noinline__ void choose_exactly(const RouteArgs& a, int64_t t, float m, Choice* out) {
  choose<double, VPL>(a, t, m, out);
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
  float m = -INFINITY;
  for (int e = lane; e < a.experts; e += 32) m = fmaxf(m, load_logit(a, t, e));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  Choice c;
  if (!choose<float, VPL>(a, t, m, &c)) choose_exactly<VPL>(a, t, m, &c);
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
