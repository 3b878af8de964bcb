// Device helpers shared by the kernels that serve a batch of new tokens over
// a paged cache (include/hc_paged.h): which sequence a row belongs to, and
// where a position lies in the pool.
#pragma once

#include <stdint.h>

namespace hc {

// New tokens of the batch as the kernels see them.
struct BatchView {
  const int32_t *page_table, *kv_lens, *cu_q;  // cu_q NULL: one new token per sequence
  int64_t table_stride, num_pages;
  int32_t seqs, max_pages, page_size;
  int64_t tokens;
};

// First new token of sequence s, as a row of q (within the call's rows,
// whatever cu_q says).
__device__ __forceinline__ int64_t first_row(const BatchView& b, int s) {
  if (!b.cu_q) return s;
  const int64_t t = b.cu_q[s];
  return t < 0 ? 0 : t < b.tokens ? t : b.tokens;
}
// Length of sequence s with its new tokens, cut to what its table row can hold.
__device__ __forceinline__ int64_t kv_len_of(const BatchView& b, int s) {
  const int64_t n = b.kv_lens[s], cap = static_cast<int64_t>(b.max_pages) * b.page_size;
  return n < 0 ? 0 : n < cap ? n : cap;
}
// Pool page of the table's entry `i` of sequence s, or -1 outside the pool.
__device__ __forceinline__ int page_of(const BatchView& b, int s, int64_t i) {
  const int p = b.page_table[s * b.table_stride + i];
  return p >= 0 && p < b.num_pages ? p : -1;
}

// The largest s in [0, n) with f(s) <= v for a non-decreasing f with
// f(0) <= v, by the 32 lanes of a full warp: every step tests 32 candidates at
// once, so a batch of up to 32 (1024) sequences takes one (two) round trips to
// memory where a binary search would take 5 (10).
template <class F>
__device__ __forceinline__ int warp_last_le(int n, int64_t v, F f) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int s = lo + lane * step;
    const bool ok = s < hi && (lane == 0 || f(s) <= v);
    const int c = __popc(__ballot_sync(0xffffffffu, ok));
    lo += (c - 1) * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  return lo;
}

}  // namespace hc
