// What the kernels of the experts' layer share: the list of (token, choice)
// pairs sorted by expert, and the tiles of its rows.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hc_experts_internal.h"

namespace hc {

// Device buffers of a call, in its workspace. A pair is t * top_k + j; the list holds the pairs of expert 0, then those of
// expert 1 and so on, each expert's in rising order, and bounds[e] is where expert e's begin.
struct ExpertLists {
  int32_t* bounds;  // [num_experts + 1]
  int32_t* order;   // [pairs]
};

// The products on the tensor cores (hc_experts_um.cu), for fp16 and bf16.
struct ExpertUm {
  ExpertLists lists;
  void *h, *o;             // (pairs, inner) of T in the list's order; (pairs, hidden) at the pairs' places, of T or float
  int64_t h_step, o_step;  // elements from row to row, multiples of 8
  float* part;             // partial sums
  unsigned int* tickets;   // of the inner product's tiles, then of the outer one's; zero before the call
  int64_t inner_tickets;
  int rows;                // pairs to a tile: 32 and 64 (few, o is float), 128 (many, o is T)
};
int64_t experts_um_tiles(const hc_expert_mlp_t& p, int rows, bool inner);
cudaError_t launch_experts_um(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s);

// Tiles of up to `rows` rows of one expert's part of the list have numbers ("slots") that follow from the bounds without a
// sum over experts: expert e's tiles are slots bounds[e] / rows + e, ... A slot past an expert's last tile is empty. There
// are pairs / rows + num_experts slots.
struct ExpertTile {
  int expert;
  int first;  // place in the list of its first row
  int rows;   // 0: an empty slot
};

__host__ __device__ constexpr int64_t expert_slots(int64_t pairs, int rows, int experts) { return pairs / rows + experts; }

__device__ __forceinline__ ExpertTile expert_tile(const int32_t* bounds, int experts, int rows, int slot) {
  int lo = 0, hi = experts - 1;  // the last expert whose first slot is not after this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (bounds[mid] / rows + mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int begin = bounds[lo], end = bounds[lo + 1];
  const int first = begin + (slot - (begin / rows + lo)) * rows;
  return ExpertTile{lo, first, max(0, min(rows, end - first))};
}

}  // namespace hc
