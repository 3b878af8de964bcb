// The experts' products in fp16/bf16 on the tensor cores (tcgen05): both products
// of the layer run through one kernel,
//
//   inner  h = silu(x gate) * (x up), rows of x gathered by the list of pairs
//   outer  o = h down, rows of h in the list's order
//
// A tile is kRows pairs of one expert by two halves of 128 features: the gate's
// and the up projection's for the inner product, 256 features for the outer one.
// A stage of the ring holds 64 inputs of both: the halves' weights by TMA (either
// layout; the MMA's descriptor says which axis is contiguous), the pairs' rows by
// TMA's gather of four rows (inner) or as a box (outer), all in 128-byte swizzle.
//
// Two forms, by the pairs that an expert has on average:
//   few   the weights are the MMA's A operand, two accumulators of 128 features by
//         kRows (32 or 64) pairs: the weights' 128 rows fill the tensor core however
//         few pairs there are. Bound: bytes of the weights. The tiles' blocks of
//         inputs, laid end to end, are cut into equal runs, one for each SM; a tile
//         that a cut goes through is written as partial sums, and the CTA that
//         finishes last adds them up in the order of the runs (so that which one
//         that is does not show in the result).
//   many  the pairs are the A operand (128 rows), the halves together B (256): one
//         accumulator of 128 by 256, two of them in turn, so that a tile is written
//         while the next one is multiplied. Bound: the tensor cores. Whole tiles
//         are dealt out in turn.
//
// One TMA warp, one MMA warp, four warps that write results; stages are handed over
// through mbarriers (all waits bounded, see hc_async.cuh).
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "hc_async.cuh"
#include "hc_common.cuh"
#include "hc_experts.cuh"
#include "hc_tc.cuh"
#include "hc_vec.cuh"

namespace hc {

__device__ unsigned int g_experts_wait_timeouts = 0;

namespace {

constexpr int kHalf = 128;                 // features of half a tile
constexpr int kBK = 64;                    // inputs of a stage: one 128-byte row
constexpr int kWeightBytes = 2 * kHalf * kBK * 2;
constexpr int kGatherWarps = 4;
constexpr int kStageOut = 32 * 64;          // (many) results of a warp on their way out
constexpr int kMaxExperts = 1024;

struct UmArgs {
  CUtensorMap tm_rows;      // inner: x, box {64, 1} (gathered); outer: h, box {64, kRows}
  CUtensorMap tm_w[2];      // the halves: gate and up, or down twice
  const int32_t *bounds, *order;
  void* out;                // inner: h in the list's order; outer: o at the pairs' places
  float* part;              // [2 * CTAs][2 halves][kRows][128], for tiles that a cut goes through
  unsigned int* tickets;    // of each tile: pieces that have been written
  uint8_t* exps;            // (many, outer) an exponent for each 16 elements of o
  int64_t out_step, exp_step;  // elements from row to row of out, and of exps
  const void* x;            // (many, inner) rows that are gathered, and their step
  int64_t x_step;
  int inputs;
  int experts, top_k, kblocks, fblocks, features, k_major;
};

template <int kRows, bool kFew> struct Cfg {
  static constexpr int kRowBytes = kRows * kBK * 2;
  static constexpr int kStage = kWeightBytes + kRowBytes;
  static constexpr int kStages = kRows == 32 ? 6 : kRows == 64 ? 5 : 4;
  static constexpr int kAccCols = kFew ? 2 * kRows : 256;  // columns of tensor memory of an accumulator
};

struct Bars {
  uint64_t full[6], empty[6], acc_full[2], acc_empty[2];
  uint32_t tmem_base, last;
  int32_t bounds[kMaxExperts + 1], tiles[kMaxExperts + 1];  // tiles: of the experts before each
  int32_t red[16];
};

template <int kRows, bool kFew> constexpr size_t smem_bytes() {
  return Cfg<kRows, kFew>::kStages * Cfg<kRows, kFew>::kStage + (kFew ? 0 : 8 * kStageOut) + sizeof(Bars) + 1024;
}

// Four rows of 64 elements (x a multiple of 64) into 512 bytes.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int x, int r0, int r1, int r2, int r3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_addr(bar))
      : "memory");
}

// silu(g) * u. The approximate exponential and quotient are within 2^-21, T's rounding at least 2^-12.
__device__ __forceinline__ float gated(float g, float u) { return __fdividef(g * u, 1.0f + __expf(-g)); }

// A finite value too large for T becomes its largest one: h of fp16 can pass 65504 where its products with down do not.
template <typename T> __device__ __forceinline__ float saturate(float v) { return v; }
template <> __device__ __forceinline__ float saturate<__half>(float v) {
  const float m = fabsf(v);
  return m > 65504.0f && m < INFINITY ? copysignf(65504.0f, v) : v;
}

// Arrive on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// Ordinary writes into shared memory (cp.async's among them) that this thread knows of, before the tensor core reads them.
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A CTA's pieces of work, the same for all its warps.
template <int kRows, bool kFew> struct Pieces {
  const UmArgs& a;
  const Bars& b;
  int64_t at, end, units, ctas;
  int total;

  __device__ __forceinline__ Pieces(const UmArgs& args, const Bars& bars) : a(args), b(bars) {
    total = b.tiles[a.experts] * a.fblocks;
    units = static_cast<int64_t>(total) * a.kblocks;
    ctas = min(static_cast<int64_t>(gridDim.x), units);  // that have work, at least a unit each
    if (kFew) {
      at = end = 0;
      if (blockIdx.x < ctas) {
        at = first_unit(blockIdx.x);
        end = first_unit(blockIdx.x + 1);
      }
    } else {
      at = blockIdx.x;
      end = total;
    }
  }
  __device__ __forceinline__ int64_t first_unit(int64_t cta) const { return cta * units / ctas; }
  __device__ __forceinline__ int cta_of(int64_t unit) const {
    return static_cast<int>(((unit + 1) * ctas - 1) / units);
  }

  int tile, k0, k1;                  // blocks of inputs k0 .. k1 - 1 of this tile
  int expert, first, rows, feature;  // its pairs in the list, its first feature (of either half)
  int mine;                          // which of a CTA's two places for partial sums

  __device__ __forceinline__ bool next(int halves_step) {
    if (at >= end) return false;
    if (kFew) {
      tile = static_cast<int>(at / a.kblocks);
      k0 = static_cast<int>(at - static_cast<int64_t>(tile) * a.kblocks);
      k1 = static_cast<int>(min(static_cast<int64_t>(a.kblocks), k0 + (end - at)));
      at += k1 - k0;
    } else {
      tile = static_cast<int>(at);
      k0 = 0;
      k1 = a.kblocks;
      at += gridDim.x;
    }
    mine = k0 > 0 ? 0 : 1;
    const int m = tile / a.fblocks;
    feature = (tile - m * a.fblocks) * halves_step;
    int lo = 0, hi = a.experts - 1;  // the last expert whose tiles begin at m or before (empty ones have none)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (b.tiles[mid] <= m) lo = mid;
      else hi = mid - 1;
    }
    expert = lo;
    first = b.bounds[lo] + (m - b.tiles[lo]) * kRows;
    rows = min(kRows, b.bounds[lo + 1] - first);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == a.kblocks; }
};

// Tiles of each expert, summed up, and the bounds.
template <int kRows, int kThreads> __device__ __forceinline__ void count_tiles(const UmArgs& a, Bars* b) {
  constexpr int kEach = (kMaxExperts + kThreads - 1) / kThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= a.experts; e += kThreads) b->bounds[e] = a.bounds[e];
  __syncthreads();
  int n[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = threadIdx.x * kEach + i;
    n[i] = e < a.experts ? (b->bounds[e + 1] - b->bounds[e] + kRows - 1) / kRows : 0;
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
    if (e <= a.experts) b->tiles[e] = before;
    before += n[i];
  }
  __syncthreads();
}

template <bool kFew, bool kInner> constexpr bool kGathers = kInner && !kFew;
// Warps that write results: a tile of the outer product has a quarter of the inner one's MMAs to a result, or less.
template <bool kFew, bool kInner> constexpr int kResultWarps = !kFew && !kInner ? 8 : 4;
template <bool kFew, bool kInner>
constexpr int kBlock = 64 + 32 * kResultWarps<kFew, kInner> + (kGathers<kFew, kInner> ? 32 * kGatherWarps : 0);

template <typename T, int kRows, bool kFew, bool kInner>
__global__ void __launch_bounds__(kBlock<kFew, kInner>, 1) product_kernel(const __grid_constant__ UmArgs a) {
  using C = Cfg<kRows, kFew>;
  constexpr bool kGather = kGathers<kFew, kInner>;
  constexpr int kResults = kResultWarps<kFew, kInner>;  // warps 2 .., after them those that gather
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kStep = kInner ? kHalf : 2 * kHalf;  // features from tile to tile
  constexpr int kCols = 2 * C::kAccCols;             // (a power of two from 128 to 512)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Bars* b = reinterpret_cast<Bars*>(smem + C::kStages * C::kStage + (kFew ? 0 : 8 * kStageOut));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&b->full[i], kGather ? 1 + 32 * kGatherWarps : 1);
      mbar_init(&b->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->acc_full[i], 1);
      mbar_init(&b->acc_empty[i], kResults);
    }
    fence_mbar_init();
    tma_prefetch_desc(&a.tm_rows);
    tma_prefetch_desc(&a.tm_w[0]);
    tma_prefetch_desc(&a.tm_w[1]);
  }
  if (warp == 1) {
    tmem_alloc(&b->tmem_base, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b->tmem_base;
  pdl_wait();
  pdl_trigger();
  count_tiles<kRows, kBlock<kFew, kInner>>(a, b);
  Pieces<kRows, kFew> p(a, *b);
  bool ok = true;

  if (warp == 0) {
    int it = 0;
    while (ok && p.next(kStep)) {
      // the rows that this lane gathers (past the tile's last one any row will do: nobody looks at the results)
      int row[4];
      if (kInner && !kGather && lane * 4 < kRows) {
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = a.order[p.first + min(lane * 4 + i, p.rows - 1)] / a.top_k;
      }
      for (int k = p.k0; k < p.k1; ++k, ++it) {
        const int st = it % C::kStages;
        if (lane == 0) ok = mbar_wait(&b->empty[st], ((it / C::kStages) & 1) ^ 1, &g_experts_wait_timeouts);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        uint8_t* w = smem + st * C::kStage;
        uint8_t* r = w + kWeightBytes;
        uint64_t* bar = &b->full[st];
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, kGather ? kWeightBytes : C::kStage);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int n = p.feature + (kInner ? 0 : h * kHalf);
            if (a.k_major) {
              tma_load_3d(w + h * (kWeightBytes / 2), &a.tm_w[h], k * kBK, n, p.expert, bar);
            } else {
              tma_load_3d(w + h * (kWeightBytes / 2), &a.tm_w[h], n, k * kBK, p.expert, bar);
              tma_load_3d(w + h * (kWeightBytes / 2) + kWeightBytes / 4, &a.tm_w[h], n + 64, k * kBK, p.expert, bar);
            }
          }
          if (!kInner) tma_load_2d(r, &a.tm_rows, k * kBK, p.first, bar);
        }
        __syncwarp();
        if (kInner && !kGather && lane * 4 < kRows)
          tma_gather4(r + lane * 4 * 128, &a.tm_rows, k * kBK, row[0], row[1], row[2], row[3], bar);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t w0 = smem_addr(smem), r0 = w0 + kWeightBytes;
      const uint64_t wd = a.k_major ? smem_desc_sw128(w0, 16, 1024) : smem_desc_sw128(w0, kWeightBytes / 4, 1024);
      const uint64_t wk = a.k_major ? 2 : 128;  // 16 inputs on, in 16 bytes
      const uint64_t rd = smem_desc_sw128(r0, 16, 1024);
      const uint32_t id = kFew ? idesc_f16(kBf16, 128, kRows, !a.k_major, false) : idesc_f16(kBf16, 128, 256, false, !a.k_major);
      int it = 0;
      for (int acc = 0; ok && p.next(kStep); ++acc) {
        const int buf = acc & 1;
        ok = mbar_wait(&b->acc_empty[buf], ((acc >> 1) & 1) ^ 1, &g_experts_wait_timeouts);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * C::kAccCols;
        for (int k = p.k0; k < p.k1; ++k, ++it) {
          const int st = it % C::kStages;
          ok = mbar_wait(&b->full[st], (it / C::kStages) & 1, &g_experts_wait_timeouts);
          if (!ok) break;
          if (kGather) fence_proxy_async();
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>((st * C::kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint32_t add = k > p.k0 || kk > 0 ? 1u : 0u;
            const uint64_t w = wd + so + kk * wk, r = rd + so + kk * 2;
            if (kFew) {
              mma_f16(d, w, r, id, add);
              mma_f16(d + kRows, w + (kWeightBytes / 2 >> 4), r, id, add);
            } else {
              mma_f16(d, r, w, id, add);
            }
          }
          mma_commit(&b->empty[st]);
        }
        mma_commit(&b->acc_full[buf]);
      }
    }
  } else if (warp < 2 + kResults) {
    const int quarter = warp & 3;  // of the lanes of tensor memory, which a warp's place decides
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int me = quarter * 32 + lane;
    for (int acc = 0; ok && p.next(kStep); ++acc) {
      const int buf = acc & 1;
      const uint32_t d = tmem + buf * C::kAccCols + lanes;
      // places of the results
      int place[(kRows + 31) / 32];
      if (kFew) {
#pragma unroll
        for (int i = 0; i < (kRows + 31) / 32; ++i) {
          const int at = p.first + min(32 * i + lane, p.rows - 1);
          place[i] = kInner ? at : a.order[at];
        }
      } else {
        const int at = p.first + min(me, p.rows - 1);
        place[0] = kInner ? at : a.order[at];
      }
      ok = mbar_wait(&b->acc_full[buf], (acc >> 1) & 1, &g_experts_wait_timeouts);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if constexpr (kFew) {
        // this thread has feature `me` of both halves, a column for each pair
        const bool whole = p.whole();
        const int f = p.feature + me;
        const auto put = [&](int c, float v0, float v1) {
          const int64_t to = static_cast<int64_t>(__shfl_sync(0xffffffffu, place[c / 32], c % 32)) * a.out_step;
          if (kInner) {
            if (f < a.features) stf(static_cast<T*>(a.out) + to + f, saturate<T>(gated(v0, v1)));
          } else {
            if (f < a.features) static_cast<float*>(a.out)[to + f] = v0;
            if (f + kHalf < a.features) static_cast<float*>(a.out)[to + f + kHalf] = v1;
          }
        };
        float* part = a.part + (2 * static_cast<int64_t>(blockIdx.x) + p.mine) * (2 * kRows * kHalf) + me;
#pragma unroll
        for (int c0 = 0; c0 < kRows; c0 += 16) {
          if (c0 < p.rows) {
            float v[2][16];
            tmem_ld16(d + c0, v[0]);
            tmem_ld16(d + kRows + c0, v[1]);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if (c0 + c < p.rows) {
                if (whole) {
                  put(c0 + c, v[0][c], v[1][c]);
                } else {
                  __stcg(part + (c0 + c) * kHalf, v[0][c]);
                  __stcg(part + (kRows + c0 + c) * kHalf, v[1][c]);
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->acc_empty[buf]);
        if (!whole) {
          const int64_t unit = static_cast<int64_t>(p.tile) * a.kblocks;
          const int c0 = p.cta_of(unit), c1 = p.cta_of(unit + a.kblocks - 1);
          __threadfence();
          named_bar_sync(1, 128);
          if (warp == 2 && lane == 0) b->last = atomicAdd(&a.tickets[p.tile], 1u) == static_cast<unsigned>(c1 - c0);
          named_bar_sync(1, 128);
          const bool last = b->last != 0;
          if (last) {
            __threadfence();
            // (sixteen pairs' sums at a time, so that their loads overlap)
            for (int b0 = 0; b0 < p.rows; b0 += 16) {
              float v0[16] = {}, v1[16] = {};
              for (int q = c0; q <= c1; ++q) {
                const int slot = p.first_unit(q) > unit ? 0 : 1;
                const float* from = a.part + (2 * static_cast<int64_t>(q) + slot) * (2 * kRows * kHalf) + b0 * kHalf + me;
                float w0[16], w1[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  w0[c] = b0 + c < p.rows ? __ldcg(from + c * kHalf) : 0.0f;
                  w1[c] = b0 + c < p.rows ? __ldcg(from + (kRows + c) * kHalf) : 0.0f;
                }
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  v0[c] += w0[c];
                  v1[c] += w1[c];
                }
              }
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (b0 + c < p.rows) put(b0 + c, v0[c], v1[c]);
            }
          }
          named_bar_sync(1, 128);  // (`last` is read before it is written again)
        }
      } else {
        // This thread has pair `me`, a column for each feature. Thirty-two features of the warp's 32 pairs at a time go through
        // shared memory, so that four lanes write 64 bytes of one row (a row for each lane would be 32 requests an instruction).
        constexpr int kCols32 = (kInner ? kHalf : 2 * kHalf) / 32 / (kResults / 4);  // that a warp has, from the first-th on
        const int part = (warp - 2) / 4, first = part * kCols32;
        uint8_t* stage = smem + C::kStages * C::kStage + (warp - 2) * kStageOut;
        uint32_t exps[2] = {};
#pragma unroll
        for (int h = 0; h < kCols32; ++h) {
          const int c0 = (first + h) * 32;
          uint32_t x[2][16], y[2][16];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tmem_ld16_nowait(d + c0 + 16 * i, x[i]);
            if (kInner) tmem_ld16_nowait(d + kHalf + c0 + 16 * i, y[i]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 q[2];
            float v[16];
            tmem_ld_wait_r(x[i]);
            if (kInner) tmem_ld_wait_r(y[i]);
            if (kInner) {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = saturate<T>(gated(__uint_as_float(x[i][j]), __uint_as_float(y[i][j])));
              q[0] = V8<T>::pack(v);
              q[1] = V8<T>::pack(v + 8);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(x[i][j]);
              exps[h >> 1] |= BlockFloat::pack(v, reinterpret_cast<uint32_t*>(q)) << (16 * (h & 1) + 8 * i);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
              *reinterpret_cast<uint4*>(stage + lane * 64 + (((2 * i + j) ^ ((lane >> 1) & 3)) << 4)) = q[j];
          }
          __syncwarp();
          const int chunk = lane & 3, f = p.feature + c0 + chunk * 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2);
            const int64_t to = __shfl_sync(0xffffffffu, place[0], r);
            const uint4 q = *reinterpret_cast<const uint4*>(stage + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4));
            // (rows of out are 16-byte aligned and padded to a multiple of 16 elements)
            if (quarter * 32 + r < p.rows && f < a.features) st16(static_cast<T*>(a.out) + to * a.out_step + f, q);
          }
          __syncwarp();
        }
        if (!kInner && me < p.rows)  // (a row's exponents are padded to whole tiles)
          *reinterpret_cast<uint2*>(a.exps + static_cast<int64_t>(place[0]) * a.exp_step + p.feature / 16 + 8 * part) =
              make_uint2(exps[0], exps[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b->acc_empty[buf]);
      }
    }
  } else if constexpr (kGather) {
    // TMA's gather takes some 40 ns for four rows, so that 128 rows of 128 bytes would come at a third of the tensor cores'
    // pace; four warps with 16-byte copies keep up. A lane has the same 16 bytes of eight rows.
    const int g = warp - 2 - kResults, chunk = lane & 7;
    const uint32_t dst = smem_addr(smem) + kWeightBytes;
    int it = 0;
    while (ok && p.next(kStep)) {
      const T* src[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = g * 32 + 4 * i + (lane >> 3);
        src[i] = static_cast<const T*>(a.x) + static_cast<int64_t>(a.order[p.first + min(r, p.rows - 1)] / a.top_k) * a.x_step +
                 chunk * 8;
      }
      for (int k = p.k0; k < p.k1; ++k, ++it) {
        const int st = it % C::kStages;
        if (lane == 0) ok = mbar_wait(&b->empty[st], ((it / C::kStages) & 1) ^ 1, &g_experts_wait_timeouts);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        const int left = a.inputs - (k * kBK + chunk * 8);  // elements of this chunk and after it
        const uint32_t bytes = left <= 0 ? 0u : left >= 8 ? 16u : static_cast<uint32_t>(left * 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = g * 32 + 4 * i + (lane >> 3);
          cp_async16_zfill(dst + st * C::kStage + r * 128 + ((chunk ^ (r & 7)) << 4), bytes ? src[i] + k * kBK : src[i] - chunk * 8,
                           bytes);
        }
        cp_async_arrive(&b->full[st]);
      }
    }
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// A map over rows of 16-bit elements, 64 to a box.
bool map_2d(CUtensorMap* m, const void* base, bool bf16, int64_t cols, int64_t rows, int64_t step, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(step) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
  const auto fn = tmap_encoder();
  return fn != nullptr &&
         fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A map over experts' weights; the axis with contiguous elements comes first.
bool map_weight(CUtensorMap* m, const void* base, bool bf16, int experts, int inputs, int outputs, int64_t es, int64_t is,
                int64_t os) {
  const bool k_major = is == 1;
  const int64_t cols = k_major ? inputs : outputs, rows = k_major ? outputs : inputs, step = k_major ? os : is;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(experts)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(step) * 2, static_cast<cuuint64_t>(experts > 1 ? es : rows * step) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(k_major ? kHalf : kBK), 1}, one[3] = {1, 1, 1};
  const auto fn = tmap_encoder();
  return fn != nullptr &&
         fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int kRows, bool kFew>
cudaError_t launch_products(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  const int64_t pairs = p.tokens * p.top_k;
  UmArgs a;
  a.bounds = u.lists.bounds;
  a.order = u.lists.order;
  a.part = u.part;
  a.experts = p.num_experts;
  a.top_k = p.top_k;
  // (no more CTAs than there can be units of work)
  const auto grid = [&](int fblocks, int kblocks) {
    const int64_t tiles = std::min(pairs, pairs / kRows + p.num_experts) * fblocks;
    return static_cast<unsigned>(std::min<int64_t>(num_sms, kFew ? tiles * kblocks : tiles));
  };
  a.out = u.h;
  a.out_step = u.h_step;
  a.features = p.inner;
  a.fblocks = (p.inner + kHalf - 1) / kHalf;
  a.kblocks = (p.hidden + kBK - 1) / kBK;
  a.k_major = p.up_in_stride == 1;
  a.tickets = u.tickets;
  a.exps = u.exps;
  a.exp_step = u.exp_step;
  a.x = p.x;
  a.x_step = p.x_stride;
  a.inputs = p.hidden;
  if (!map_2d(&a.tm_rows, p.x, kBf16, p.hidden, p.tokens, p.x_stride, 1) ||
      !map_weight(&a.tm_w[0], p.gate, kBf16, p.num_experts, p.hidden, p.inner, p.up_expert_stride, p.up_in_stride,
                  p.up_out_stride) ||
      !map_weight(&a.tm_w[1], p.up, kBf16, p.num_experts, p.hidden, p.inner, p.up_expert_stride, p.up_in_stride, p.up_out_stride))
    return cudaErrorInvalidValue;
  constexpr size_t smem = smem_bytes<kRows, kFew>();
  cudaError_t e = ensure_smem<product_kernel<T, kRows, kFew, true>>(smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(product_kernel<T, kRows, kFew, true>, dim3(grid(a.fblocks, a.kblocks)), dim3(kBlock<kFew, true>), smem, s, 1, a);
  if (e != cudaSuccess) return e;
  a.tickets += u.inner_tickets;
  a.out = u.o;
  a.out_step = u.o_step;
  a.features = p.hidden;
  a.fblocks = (p.hidden + 2 * kHalf - 1) / (2 * kHalf);
  a.kblocks = (p.inner + kBK - 1) / kBK;
  a.k_major = p.down_in_stride == 1;
  if (!map_2d(&a.tm_rows, u.h, kBf16, p.inner, pairs, u.h_step, kRows) ||
      !map_weight(&a.tm_w[0], p.down, kBf16, p.num_experts, p.inner, p.hidden, p.down_expert_stride, p.down_in_stride,
                  p.down_out_stride))
    return cudaErrorInvalidValue;
  a.tm_w[1] = a.tm_w[0];
  e = ensure_smem<product_kernel<T, kRows, kFew, false>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(product_kernel<T, kRows, kFew, false>, dim3(grid(a.fblocks, a.kblocks)), dim3(kBlock<kFew, false>), smem, s, 1, a);
}

template <typename T> cudaError_t launch_form(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s) {
  if (u.rows == 32) return launch_products<T, 32, true>(p, u, num_sms, s);
  if (u.rows == 64) return launch_products<T, 64, true>(p, u, num_sms, s);
  return launch_products<T, 128, false>(p, u, num_sms, s);
}

}  // namespace

int64_t experts_um_tiles(const hc_expert_mlp_t& p, int rows, bool inner) {
  const int64_t pairs = p.tokens * p.top_k, step = inner ? kHalf : 2 * kHalf, features = inner ? p.inner : p.hidden;
  return std::min(pairs, pairs / rows + p.num_experts) * ((features + step - 1) / step);
}

cudaError_t launch_experts_um(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s) {
  return p.dtype == HC_F16 ? launch_form<__half>(p, u, num_sms, s) : launch_form<__nv_bfloat16>(p, u, num_sms, s);
}

unsigned int read_experts_wait_timeouts(bool reset) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_experts_wait_timeouts, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (reset) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_experts_wait_timeouts, &z, sizeof(z));
  }
  return v;
}

}  // namespace hc
