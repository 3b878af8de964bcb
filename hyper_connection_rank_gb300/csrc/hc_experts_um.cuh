// What the tensor-core kernels of the experts' products share (hc_experts_few.cu,
// hc_experts_many.cu): arguments, the ring's barriers, the division of the work
// into pieces, the gathering of rows, and the inner product's activation.
//
// Both products of the layer run through one kernel of either form,
//
//   inner  h = silu(x gate) * (x up), rows of x gathered by the list of pairs
//   outer  o = h down, rows of h in the list's order
//
// h is rounded to T, which the tensor core's operands are: results are off by 2.3e-3 of their size against 64 bits in bf16 and
// 2.9e-4 in fp16, where rounding them alone costs 1.65e-3 and 2.1e-4. (What the rounding takes off as a second operand
// would give that back for twice the outer product's MMAs, which where experts have many pairs set its pace.)
//
// A tile is a number of pairs of one expert by two halves of 128 features: the
// gate's and the up projection's for the inner product, 256 features for the outer
// one. A stage of a CTA's ring holds 64 inputs (a row of 128 bytes, in 128-byte
// swizzle) of pairs and of weights. Weights come by TMA in either layout, with
// their inputs or their outputs contiguous: the MMA's descriptor says which. Rows
// of h come by TMA, too; rows of x by 16-byte copies of gathering warps (TMA's
// gather of four rows took some 40 ns each, so that 128 rows of 128 bytes came at
// a third of the tensor cores' pace).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "hc_async.cuh"
#include "hc_common.cuh"
#include "hc_experts.cuh"
#include "hc_tc.cuh"
#include "hc_vec.cuh"

namespace hc {
namespace um {

constexpr int kHalf = 128;  // features of half a tile
constexpr int kBK = 64;     // inputs of a stage: one 128-byte row
constexpr int kHalfBytes = kHalf * kBK * 2;
constexpr int kMaxExperts = 1024;
constexpr int kMaxStages = 6;

struct Args {
  CUtensorMap tm_rows;         // outer: h, a box of 64 inputs and a CTA's pairs
  CUtensorMap tm_w[2];         // the halves: gate and up, or down twice
  const int32_t *bounds, *order;
  const void* x;               // inner: rows that are gathered, and their step
  int64_t x_step;
  void* out;                   // inner: h in the list's order; outer: o at the pairs' places
  uint8_t* counts;             // (few, outer) the planes of each 256 elements of o
  int64_t out_step, count_step;  // elements from row to row of out, and of counts
  int64_t plane;               // (few, outer) elements from plane to plane of out
  Excess excess;               // (inner, fp16)
  float* part;                 // (few, inner) [2 * CTAs][2 halves][rows][128], for tiles that a cut goes through
  unsigned int* gave_up;       // becomes 1 if a wait gave up
  unsigned int* tickets;       // (few, inner) of each tile: pieces that have been written
  int experts, top_k, inputs, features, kblocks, fblocks, k_major;
  int most_parts;              // (few) that a tile may be cut into
};

// Behind it in shared memory: the bounds, and the tiles of the experts before each (num_experts + 1 both).
struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  uint32_t tmem_base, last;
  int32_t red[32];
};
inline size_t bars_bytes(int experts) { return sizeof(Bars) + 2 * (static_cast<size_t>(experts) + 1) * sizeof(int32_t); }

// Arrive on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Ordinary writes into shared memory (cp.async's among them) that this thread knows of, before the tensor core reads them.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// silu(g) u. The approximate exponential and reciprocal and the products are within (1.5 |g| + 16) 2^-24 of it for g < 0 (the
// argument's rounding counts), within 2^-20 above; from g = -174 on, where it is below 2^-251 u, it is 0.
__device__ __forceinline__ float gated(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(g) * -0.72134752f));  // e^(-|g| / 2)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(e, e, 1.0f)));
  return silu_times(g, u, e, r);
}

// A finite value too large for T becomes its largest one, and an entry of the excess.
template <typename T> __device__ __forceinline__ float saturate(float v) { return v; }
template <> __device__ __forceinline__ float saturate<__half>(float v) { return past_half(v) ? copysignf(kMostHalf, v) : v; }
__device__ __forceinline__ void mark_excess(const Excess& x, int64_t pair, int feature) {
  atomicOr(x.over + pair * x.words + (feature >> 10), 1u << ((feature >> 5) & 31));
}

// The pieces of work of a CTA (or a pair of them), the same for all its warps: whole tiles in turn, or, with kSplit, parts of
// them. If there are no more tiles than CTAs, a tile is cut into as many parts of its blocks of inputs as leave every CTA at
// most one (so that few CTAs wait for others' sums, and none twice; two thirds of the SMs can take what the memory gives);
// otherwise all tiles' blocks, laid end to end, are cut into equal runs, of which the pieces of cut tiles come first, so that
// their sums are joined while whole tiles are still on their way. (Units, blocks of inputs, are below 2^31 in number
// where tiles are split: at most 2^11 tiles of pairs, and 2^19 blocks of features and inputs.)
template <int kRows, bool kSplit> struct Pieces {
  const Args& a;
  const int32_t *bounds, *tiles;
  uint32_t at, end, units, ctas, each, rest, parts;  // parts: of a tile, 0 for runs
  uint32_t head, tail;                               // of a run: blocks of its first tile that are not its own, of its last that are

  __device__ __forceinline__ Pieces(const Args& args, const Bars* bars, uint32_t cta, uint32_t count)
      : a(args), bounds(reinterpret_cast<const int32_t*>(bars + 1)), tiles(bounds + args.experts + 1) {
    const uint32_t total = static_cast<uint32_t>(tiles[a.experts]) * a.fblocks;
    at = end = parts = 0;
    if (!kSplit) {
      ctas = count;
      at = cta;
      end = total;
    } else if (total <= count) {
      parts = total == 0 ? 1u : min(count / total, static_cast<uint32_t>(min(a.kblocks, a.most_parts)));
      at = cta;
      end = cta < total * parts ? cta + 1 : cta;
    } else {
      units = total * a.kblocks;
      ctas = count;
      each = units / ctas;
      rest = units - each * ctas;
      // from here on in tiles: the whole ones are at .. end - 1
      const uint32_t from = first_unit(cta), to = first_unit(cta + 1);
      at = from / a.kblocks;
      end = to / a.kblocks;
      head = from - at * a.kblocks;
      tail = to - end * a.kblocks;
      at += head > 0;
    }
  }
  // first_unit(cta) = cta * units / ctas
  __device__ __forceinline__ uint32_t first_unit(uint32_t cta) const { return cta * each + cta * rest / ctas; }

  int tile, k0, k1;                  // blocks of inputs k0 .. k1 - 1 of this tile
  int expert, first, rows, feature;  // its pairs in the list, its first feature (of either half)

  __device__ __forceinline__ bool next(int features) {
    if (kSplit && parts == 0) {
      if (tail > 0) {
        tile = static_cast<int>(end);
        k0 = 0;
        k1 = static_cast<int>(tail);
        tail = 0;
      } else if (head > 0) {
        tile = static_cast<int>(at - 1);
        k0 = static_cast<int>(head);
        k1 = a.kblocks;
        head = 0;
      } else {
        if (at >= end) return false;
        tile = static_cast<int>(at++);
        k0 = 0;
        k1 = a.kblocks;
      }
    } else if (at >= end) {
      return false;
    } else if (!kSplit) {
      tile = static_cast<int>(at);
      k0 = 0;
      k1 = a.kblocks;
      at += ctas;
    } else {
      tile = static_cast<int>(at / parts);
      const uint32_t part = at - tile * parts;
      k0 = static_cast<int>(part * a.kblocks / parts);
      k1 = static_cast<int>((part + 1) * a.kblocks / parts);
      ++at;
    }
    const int m = tile / a.fblocks;
    feature = (tile - m * a.fblocks) * features;
    int lo = 0, hi = a.experts - 1;  // the last expert whose tiles begin at m or before (empty ones have none)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tiles[mid] <= m) lo = mid;
      else hi = mid - 1;
    }
    expert = lo;
    first = bounds[lo] + (m - tiles[lo]) * kRows;
    rows = min(kRows, bounds[lo + 1] - first);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == a.kblocks; }

  // The number of pieces that this piece's tile is in, and which one this is. (Runs are no shorter than a tile, so that at
  // most one cut goes through it.)
  __device__ __forceinline__ int pieces() const { return parts > 0 ? parts : whole() ? 1 : 2; }
  __device__ __forceinline__ int piece() const { return parts > 0 ? (at - 1) % parts : k0 > 0 ? 1 : 0; }

  // Where partial sums lie: two places to a CTA, the first for a piece that does not begin its tile (or is a part).
  __device__ __forceinline__ int place(uint32_t cta) const {
    return 2 * cta + (parts > 0 || first_unit(cta) > static_cast<uint32_t>(tile) * a.kblocks ? 0 : 1);
  }
  // The CTAs that have pieces of this tile, the first and the last.
  __device__ __forceinline__ void sharers(uint32_t* c0, uint32_t* c1) const {
    if (parts > 0) {
      *c0 = tile * parts;
      *c1 = *c0 + parts - 1;
    } else {
      const unsigned long long unit = static_cast<unsigned long long>(tile) * a.kblocks;
      *c0 = static_cast<uint32_t>(((unit + 1) * ctas - 1) / units);
      *c1 = static_cast<uint32_t>(((unit + a.kblocks) * ctas - 1) / units);
    }
  }
};

// Tiles of each expert, summed up, and the bounds.
template <int kRows, int kThreads> __device__ __forceinline__ void count_tiles(const Args& a, Bars* b) {
  constexpr int kEach = (kMaxExperts + kThreads - 1) / kThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t *bounds = reinterpret_cast<int32_t*>(b + 1), *tiles = bounds + a.experts + 1;
  for (int e = threadIdx.x; e <= a.experts; e += kThreads) bounds[e] = a.bounds[e];
  __syncthreads();
  int n[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = threadIdx.x * kEach + i;
    n[i] = e < a.experts ? (bounds[e + 1] - bounds[e] + kRows - 1) / kRows : 0;
    sum += n[i];
  }
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) b->red[warp] = upto;
  __syncthreads();
  int before = upto - sum;
  for (int w = 0; w < warp; ++w) before += b->red[w];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = threadIdx.x * kEach + i;
    if (e <= a.experts) tiles[e] = before;
    before += n[i];
  }
  __syncthreads();
}

// A weight's half of 128 features from n, 64 inputs from k, into 16 KB.
__device__ __forceinline__ void load_half(uint8_t* to, const CUtensorMap* map, bool k_major, int k, int n, int expert,
                                          uint64_t* bar) {
  if (k_major) {
    tma_load_3d(to, map, k, n, expert, bar);
  } else {
    tma_load_3d(to, map, n, k, expert, bar);
    tma_load_3d(to + kHalfBytes / 2, map, n + 64, k, expert, bar);
  }
}

// The same half into L2 only.
__device__ __forceinline__ void prefetch_half(const CUtensorMap* map, bool k_major, int k, int n, int expert) {
  const auto fetch = [&](int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(expert) : "memory");
  };
  if (k_major) {
    fetch(k, n);
  } else {
    fetch(n, k);
    fetch(n + 64, k);
  }
}

// A gathering warp's part of a tile: 32 rows of x, from place `first` of the list, `rows` of them (past those whatever was
// there: nobody looks at the results). A lane has the same 16 bytes of eight rows.
template <typename T> struct Gather {
  const T* src[8];
  uint32_t there;  // a bit for each
  bool all;        // of the warp's

  __device__ __forceinline__ void begin(const Args& a, int first, int rows, int group) {
    const int lane = threadIdx.x & 31;
    there = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = group * 32 + 4 * i + (lane >> 3);
      there |= r < rows ? 1u << i : 0u;
      const int pair = a.order[first + max(0, min(r, rows - 1))];
      src[i] = static_cast<const T*>(a.x) + static_cast<int64_t>(pair / a.top_k) * a.x_step + (lane & 7) * 8;
    }
    all = __all_sync(0xffffffffu, there == 0xffu);
  }
  // Inputs from k into the stage's rows at `to`, zeros past the last one; arrives on `bar` when they have landed.
  __device__ __forceinline__ void copy(const Args& a, uint32_t to, int k, int group, uint64_t* bar) const {
    const int lane = threadIdx.x & 31, chunk = lane & 7;
    const auto place = [&](int i) {
      const int r = group * 32 + 4 * i + (lane >> 3);
      return to + r * 128 + ((chunk ^ (r & 7)) << 4);
    };
    if (all && k + kBK <= a.inputs) {
#pragma unroll
      for (int i = 0; i < 8; ++i) cp_async16_zfill(place(i), src[i] + k, 16);
    } else {
      const int left = a.inputs - (k + chunk * 8);  // elements of this chunk and after it
      const uint32_t bytes = left <= 0 ? 0u : left >= 8 ? 16u : static_cast<uint32_t>(left * 2);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (there >> i & 1u) cp_async16_zfill(place(i), bytes ? src[i] + k : src[i] - chunk * 8, bytes);
    }
    cp_async_arrive(bar);
  }
};

// Host side: maps of the rows (64 elements and box_rows rows to a box) and of a weight, its contiguous axis first.
bool map_rows(CUtensorMap* m, const void* base, bool bf16, int64_t cols, int64_t rows, int64_t step, int box_rows);
bool map_weight(CUtensorMap* m, const void* base, bool bf16, int experts, int inputs, int outputs, int64_t es, int64_t is,
                int64_t os);
// The arguments of either product but for what the forms add.
bool fill_args(Args* a, const hc_expert_mlp_t& p, const ExpertUm& u, bool inner, int box_rows);

}  // namespace um
}  // namespace hc
