// What the kernels of the experts' layer share: the list of (token, choice)
// pairs sorted by expert, and the form of the experts' results on their way.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "hc_experts_internal.h"
#include "hc_two.cuh"

namespace hc {

// Device buffers of a call, in its workspace. A pair is t * top_k + j; the list holds the pairs of expert 0, then those of
// expert 1 and so on, each expert's in rising order, and bounds[e] is where expert e's begin.
struct ExpertLists {
  int32_t* bounds;  // [num_experts + 1]
  int32_t* order;   // [pairs]
};

// Sixteen floats as 16-bit integers with one exponent, for results on their way to a sum in fp32: each is off by 2^-15 of
// the largest of the sixteen at most, so that the sum's own rounding to fp16 or bf16 is what shows (rounding each to bf16
// instead would add as much error as that does). With the largest below 2^(e - 126) the unit is 2^(e - 141) / (1 - 2^-14),
// which keeps integers within 32766; infinities and NaN have integers of their own. e is at least 16, so values below
// 2^-126 become 0.
struct BlockFloat {
  static constexpr int kMax = 32766, kInf = 32767, kNan = -32768;
  static constexpr float kShrink = 0.99993896484375f;  // 1 - 2^-14

  static __device__ __forceinline__ uint32_t pack(const float* v, uint32_t* q) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    const bool odd = top >= 0x7f800000u;
    if (odd) {
      top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
        if (u < 0x7f800000u) top = max(top, u);
      }
    }
    const uint32_t e = max(top >> 23, 16u);
    const float scale = __uint_as_float((268u - e) << 23) * kShrink;
    // adding 1.5 * 2^23 rounds to an integer and leaves it in the low bits
    int n[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) n[i] = __float_as_int(fmaf(v[i], scale, 12582912.0f));
    if (odd) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
        if (u > 0x7f800000u) n[i] = kNan;
        if (u == 0x7f800000u) n[i] = v[i] > 0.0f ? kInf : -kInf;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __byte_perm(n[2 * i], n[2 * i + 1], 0x5410);
    return e;
  }

  // sum += by * (eight of them). An integer n is the low half of the float 2^23 + 2^15 + n, so that a subtraction makes a
  // float of it (a conversion has a quarter of the rate).
  static __device__ __forceinline__ void add8(const uint4& u, uint32_t e, float by, Two* sum) {
    const float scale = __uint_as_float((e - 14u) << 23) * (1.0f / kShrink);
    const uint32_t q[4] = {u.x, u.y, u.z, u.w};
    uint32_t most = __vmaxs2(__vmaxs2(q[0], q[1]), __vmaxs2(q[2], q[3]));
    uint32_t least = __vmins2(__vmins2(q[0], q[1]), __vmins2(q[2], q[3]));
    if (__vmaxs2(most, 0x7ffe7ffeu) != 0x7ffe7ffeu || __vmins2(least, 0x80028002u) != 0x80028002u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto value = [&](uint32_t bits) {
          const int n = static_cast<int16_t>(bits);
          return n == kNan ? __int_as_float(0x7fc00000) : n == kInf ? INFINITY : n == -kInf ? -INFINITY : static_cast<float>(n) * scale;
        };
        sum[i] = fma2(Two(by), Two(value(q[i] & 0xffffu), value(q[i] >> 16)), sum[i]);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t biased = q[i] ^ 0x80008000u;
      const Two n = Two(__uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7410)), __uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7432))) +
                    Two(-8421376.0f);
      sum[i] = fma2(Two(by), n * Two(scale), sum[i]);
    }
  }
};

// The products on the tensor cores, for fp16 and bf16 (hc_experts_few.cu, hc_experts_many.cu).
struct ExpertUm {
  ExpertLists lists;
  void *h, *o;             // (pairs, inner) of T in the list's order; (pairs, hidden) at the pairs' places
  uint8_t* exps;           // many: exponents of o's elements, 16 to one; few: how many planes of o count, for each 256
  int64_t h_step, o_step, exp_step;  // elements from row to row, multiples of 16
  float* part;             // partial sums of the inner product
  unsigned int* tickets;   // of the inner product's tiles; zero before the call
  int64_t plane;           // elements from plane to plane of o (few)
  int planes;
  int rows;                // pairs to a tile: 32 (few, o is float) or 256 (many, o is 16-bit integers)
};
int64_t experts_um_tiles(const hc_expert_mlp_t& p, int rows, bool inner);
cudaError_t launch_experts_few(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s);
cudaError_t launch_experts_many(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s);

}  // namespace hc
