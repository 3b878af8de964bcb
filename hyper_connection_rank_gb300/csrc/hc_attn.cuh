// What the attention kernels over a paged cache share: the arguments, how the
// rows of a batch are cut into tiles and a tile's keys into splits, and the
// form of partial results.
//
// Rows: with G = heads / kv_heads query heads to a key head, the new tokens of
// a sequence are, for one key head, q_len * G rows that read the same keys: row
// r is token r / G, head r % G of the group. A tile is `rows` consecutive rows.
// Tiles of all sequences are numbered by slots: sequence s owns the slots from
// first_row(s) * G / rows + s on, which leaves each sequence at least as many
// slots as it has tiles (a floor and one more) without a prefix sum over the
// batch; a slot past its sequence's last tile does nothing.
//
// Splits: a tile's keys, from the first that its first row sees (rounded down
// to `align`) to the last that its last row sees, are cut into pieces of
// split_len keys. Where there is more than one, each writes its sums, not
// divided, with its maximum and its sum of weights, and combine_kernel joins
// them; a single one writes the result itself.
#pragma once

#include <type_traits>

#include "hc_common.cuh"
#include "hc_paged_batch.cuh"

namespace hc {

struct AttnGeometry {
  int rows;       // rows of a tile
  int align;      // a tile's first key is a multiple of it (a power of two)
  int split_len;  // keys of a split, a multiple of align
  int splits;     // splits of the grid; the last one takes what is left
};

struct AttnArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  float* part_o;   // [split][token][head][dim], sums of weights times values
  float2* part_ml; // [split][token][head], maximum (of base-2 exponents) and sum of weights
  BatchView b;
  int64_t tokens;
  int64_t q_ts, q_hs, o_ts, o_hs, c_ps, c_ts, c_hs;
  int heads, kv_heads, group, dim, window;
  float scale, softcap;
  AttnGeometry g;
  int64_t min_rows, max_rows;  // only sequences with that many rows (q_len * group)
  bool slot_is_seq;            // slot s is the first tile of sequence s
  bool clears;                 // the last slot's CTAs clear the rows that no sequence has
  // hc_attn_rows.cu, where it splits single-token sequences itself: CTAs that there may be beside one for each tile, and pieces at
  // most (0: the splits above)
  int spare_ctas, units;
  bool clusters;  // there, a cluster to a sequence
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One tile of a sequence.
struct AttnTile {
  int s;
  int64_t token0;   // the sequence's first new token, as a row of q
  int64_t row0;     // the tile's first row in the sequence
  int rows;         // its rows (0: nothing to do)
  int64_t pos0;     // position of the sequence's first new token (negative: before its start)
  int64_t lo, hi;   // keys that any of its rows sees: [lo, hi)
  int64_t base;     // first key of split 0
  int splits;       // splits with keys; at least 1
};

// a / b for a >= 0, in 32 bits where a has no more (a 64-bit division is a hundred instructions).
__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
  return (a >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

__device__ __forceinline__ int64_t row_position(const AttnTile& t, int64_t row, int group) {
  return t.pos0 + quotient(row, group);
}

// Fills in a tile of sequence s, `index` tiles into it.
__device__ __forceinline__ void tile_at(const AttnArgs& a, const AttnGeometry& g, int s, int64_t index, AttnTile* t) {
  const int64_t first = first_row(a.b, s), q_len = first_row(a.b, s + 1) - first;
  const int64_t all = q_len * a.group, n = kv_len_of(a.b, s);
  t->s = s;
  t->token0 = first;
  t->row0 = index * g.rows;
  const int64_t left = all - t->row0;
  t->rows = left <= 0 ? 0 : left < g.rows ? static_cast<int>(left) : g.rows;
  t->pos0 = n - q_len;
  if (t->rows == 0) return;
  const int64_t p_first = row_position(*t, t->row0, a.group), p_last = row_position(*t, t->row0 + t->rows - 1, a.group);
  t->hi = p_last + 1 < 0 ? 0 : p_last + 1;
  t->lo = a.window > 0 && p_first - a.window + 1 > 0 ? p_first - a.window + 1 : 0;
  if (t->lo > t->hi) t->lo = t->hi;
  t->base = t->lo & -static_cast<int64_t>(g.align);
  const int64_t want = quotient(t->hi - t->base + g.split_len - 1, g.split_len);
  t->splits = want < 1 ? 1 : want < g.splits ? static_cast<int>(want) : g.splits;
}

// The tile of a slot, found by a full warp; rows == 0 if the slot is not used.
__device__ __forceinline__ void tile_of_slot(const AttnArgs& a, int64_t slot, AttnTile* t) {
  const auto start = [&](int s) { return quotient(first_row(a.b, s) * a.group, a.g.rows) + s; };
  const int s = a.slot_is_seq ? static_cast<int>(slot) : warp_last_le(a.b.seqs, slot, start);
  const int64_t index = a.slot_is_seq ? 0 : slot - start(s);
  tile_at(a, a.g, s, index < 0 ? 0 : index, t);
  const int64_t all = (first_row(a.b, s + 1) - t->token0) * a.group;
  if (index < 0 || all < a.min_rows || all > a.max_rows) t->rows = 0;  // (before the first bound there is no sequence)
}

// Keys of split z of a tile: [*k0, *k1).
__device__ __forceinline__ void split_range(const AttnGeometry& g, const AttnTile& t, int z, int64_t* k0, int64_t* k1) {
  *k0 = t.base + static_cast<int64_t>(z) * g.split_len;
  *k1 = z == t.splits - 1 ? t.hi : *k0 + g.split_len;
}

// Row r of tile t as (token, head).
__device__ __forceinline__ void row_owner(const AttnArgs& a, const AttnTile& t, int kv_head, int r, int64_t* token,
                                          int* head) {
  const int64_t row = t.row0 + r;
  const int64_t i = quotient(row, a.group);
  *token = t.token0 + i;
  *head = kv_head * a.group + static_cast<int>(row - i * a.group);
}

__device__ __forceinline__ int64_t part_index(const AttnArgs& a, int z, int64_t token, int head) {
  return (static_cast<int64_t>(z) * a.tokens + token) * a.heads + head;
}

// Rows before the first bound and from the last one on are no sequence's and see nothing: zeros, and minus infinity, by CTA `part`
// of `parts`.
template <typename T>
__device__ __forceinline__ void clear_unowned(const AttnArgs& a, int part, int parts) {
  if (!a.b.cu_q) return;
  const int64_t lo = first_row(a.b, 0), end = first_row(a.b, a.b.seqs), hi = end < lo ? lo : end;
  const int n = a.heads * a.dim;
  for (int64_t i = part; i < lo + a.tokens - hi; i += parts) {
    const int64_t token = i < lo ? i : hi + (i - lo);
    for (int e = threadIdx.x; e < n; e += blockDim.x) {
      const int head = e / a.dim;
      stf(static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs + (e - head * a.dim), 0.0f);
    }
    if (a.lse)
      for (int h = threadIdx.x; h < a.heads; h += blockDim.x) a.lse[token * a.heads + h] = neg_inf();
  }
}

// Whether either of two 16-bit numbers is infinite or NaN.
template <typename T>
__device__ __forceinline__ bool not_finite2(uint32_t w) {
  constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  return __vcmpeq2(w & kExp, kExp) != 0;
}

// Score to base-2 exponent: scale * log2(e) * x, and with a cap c on the scaled
// score, c * log2(e) * tanh(y) with y = scale / c * x. The error is a few units
// of the result's own size whatever c is, so that a large cap is as good as
// none: for |y| <= 3/5, tanh(y) = y P(y^2) with P of degree 4, fitted to
// tanh(sqrt(u)) / sqrt(u) for the least relative error (7.3e-8; 1.8e-7 with
// float32's roundings), and beyond (1 - e) / (1 + e) with e = exp(-2 |y|), where
// 1 - e loses nothing (4e-7). (c - 2 c / (exp(2 y) + 1) for every y is a
// difference of two numbers of size c, and off by 1e-7 of c.)
struct ScoreMap {
  float mul, k, cap;  // cap 0: none
};
constexpr float kCapTurn = 0.6f;  // where the polynomial ends
constexpr float kCap0 = 0.99999994f, kCap1 = -0.33332309f, kCap2 = 0.13310173f, kCap3 = -0.052101482f, kCap4 = 0.015475428f;
__host__ __device__ __forceinline__ ScoreMap score_map(float scale, float softcap) {
  // (k stays finite, so that a score of zero stays zero however small the cap)
  return softcap > 0.0f ? ScoreMap{scale * kLog2e, fmaxf(fminf(scale / softcap, 3e38f), -3e38f), softcap * kLog2e}
                        : ScoreMap{scale * kLog2e, 0.0f, 0.0f};
}
__device__ __forceinline__ float cap_beyond(const ScoreMap& m, float y) {  // for |y| > kCapTurn
  const float e = ex2(-2.0f * kLog2e * fabsf(y));
  return copysignf(__fdividef(m.cap * (1.0f - e), 1.0f + e), y);
}
__device__ __forceinline__ bool cap_far(const ScoreMap& m, float x) { return fabsf(x * m.k) > kCapTurn; }
__device__ __forceinline__ float cap_near(const ScoreMap& m, float x) {
  const float y = x * m.k, u = y * y;
  return x * m.mul * fmaf(fmaf(fmaf(fmaf(kCap4, u, kCap3), u, kCap2), u, kCap1), u, kCap0);
}
__device__ __forceinline__ float map_score(const ScoreMap& m, float x) {
  if (m.cap == 0.0f) return x * m.mul;
  const float near = cap_near(m, x), far = cap_beyond(m, x * m.k);
  return cap_far(m, x) ? far : near;
}

}  // namespace hc
