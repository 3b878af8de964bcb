// What the kernels of the experts' layer share: the list of (token, choice)
// pairs sorted by expert, and the arguments of its products.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "hc_experts_internal.h"

namespace hc {

// Device buffers of a call, in its workspace. A pair is t * top_k + j; the list holds the pairs of expert 0, then those of
// expert 1 and so on, each expert's in rising order, and bounds[e] is where expert e's begin.
struct ExpertLists {
  int32_t* bounds;  // [num_experts + 1]
  int32_t* order;   // [pairs]
};

// silu(g) u = g u / (1 + e^-g) with e = e^(-|g| / 2) and r = 1 / (1 + e^2): g r u above 0, (g e r)(u e) below. In this order no
// product overflows where the result does not (g u does: g = -10 and u = 4e37 make -1.8e34), nor does e^-g (from g = -89 on, where
// u can still be large enough for the result to count). No branch, since lanes must not part between the loads from tensor
// memory that a warp makes as one.
__device__ __forceinline__ float silu_times(float g, float u, float e, float r) {
  const float by = g < 0.0f ? e : 1.0f;
  return g * by * r * (u * by);
}

// Inner values beyond fp16, whose products with down can be within it: h has the largest finite value in their place, and what that
// leaves, in fp32, is kept here, for the sum over a token's experts to multiply with down itself. A pair's values count in blocks
// of 32 features that have their bit set in `over`, which is zero before the call.
struct Excess {
  float* values;   // (pairs, step) at the pairs' places
  uint32_t* over;  // (pairs, words)
  int64_t step;    // a multiple of 32
  int words;
};
constexpr float kMostHalf = 65504.0f;
__device__ __forceinline__ bool past_half(float h) { return fabsf(h) > kMostHalf && fabsf(h) < INFINITY; }
__device__ __forceinline__ float excess_of(float h) { return past_half(h) ? h - copysignf(kMostHalf, h) : 0.0f; }

// The products on the tensor cores, for fp16 and bf16 (hc_experts_few.cu, hc_experts_many.cu).
struct ExpertUm {
  ExpertLists lists;
  void* h;                 // (pairs, inner) of T in the list's order
  float* o;                // (pairs, hidden) at the pairs' places
  uint8_t* counts;         // (few) how many planes of o count, for each 256 elements
  int64_t h_step, o_step, count_step;  // elements from row to row, the first two multiples of 16
  float* part;             // partial sums of the inner product
  unsigned int* tickets;   // of the inner product's tiles; zero before the call
  Excess excess;           // (fp16)
  unsigned int* gave_up;   // becomes 1 if a wait gave up; zero before the call
  int64_t plane;           // elements from plane to plane of o (few)
  int planes;
  int rows;                // pairs to a tile: 32 (few) or 256 (many)
};
int64_t experts_um_tiles(const hc_expert_mlp_t& p, int rows, bool inner);
cudaError_t launch_experts_few(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s);
cudaError_t launch_experts_many(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s);

}  // namespace hc
