// The experts' products on the tensor cores where experts have many pairs (prompts):
// the pairs are the MMA's A operand, 256 of them to a pair of CTAs (cta_group::2,
// 128 rows from each one's shared memory into its own tensor memory), and the two
// halves of a tile's features together are B (N = 256), of which each CTA holds one
// half: D (256 x 256) += R (256 x 64) W (64 x 256).
//
// Bound: the tensor cores. A stage of a CTA is 16 KB of rows and 16 KB of weights
// for 512 cycles of MMAs; with one CTA to a tile it would be 48 KB, four stages
// instead of six, and what L2 delivered set the pace (14 to 16 TB/s, 58% of the
// tensor cores' cycles). Accumulators take turns, so that a tile is written while
// the next one is multiplied. Whole tiles are dealt out in turn.
//
// 8191 tokens at eight of 64 experts of 2560 x 640 in bf16: 294 to 307 us (inner, 1.42 PFLOP/s, 75% of measured; tensor cores active
// for 74% of the cycles) and 195 (outer, 1.10; 55%: 671 MB of results leave at 3.4 TB/s beside L2's feed of the stages); a stage takes
// 0.32 us where the MMAs take 0.27, and tiles are 90% full. 1301 tokens at two of 16 experts of 1280 x 2560 in fp16: 60 and
// 39 us, 3.5 and 2.7 TB/s of weights; tiles are half full, 20
// tiles of pairs by 20 and 5 of features are 5.3 and 1.3 rounds of 76 pairs of CTAs, and the first two tiles of each wait for cold
// weights. (Sending those to L2 earlier, by TMA or by the gathering warps, took 10 to 20% longer: both have no time to spare.
// For the same reason the gathering warps copy full tiles without a look at their rows, and nothing for rows that are not
// there: with copies of some row in their place the inner product took 75 us.)
//
// Of the pair, the first CTA issues the MMAs. The second one's stages are made known
// to it by a warp that waits for them and arrives at the first one's barrier, behind
// a fence that releases its CTA's shared memory to the cluster; the MMAs' thread
// waits with acquire at that scope. Releases of stages come by commits that arrive
// in both. All waits are bounded (see
// hc_async.cuh).
#include <algorithm>

#include "hc_experts_um.cuh"

namespace hc {

__device__ unsigned int g_many_wait_timeouts = 0;

namespace {

using namespace um;

constexpr int kRows = 256, kCtaRows = 128;  // pairs of a tile, and of a CTA
constexpr int kStage = kHalfBytes + kCtaRows * kBK * 2;
constexpr int kStages = 6;
constexpr int kAccCols = 2 * kHalf;      // columns of tensor memory of an accumulator
constexpr int kStageOut = 32 * 64;       // bytes of a warp's results on their way out
constexpr int kGatherWarps = 4;
// Warps that write results: a tile of the outer product has a quarter of the inner one's MMAs to a result, or less.
template <bool kInner> constexpr int kResults = kInner ? 4 : 8;
template <bool kInner> constexpr int kThreads = 64 + 32 * kResults<kInner> + (kInner ? 32 * kGatherWarps : 0);
constexpr size_t kSmem = kStages * kStage + 8 * kStageOut + 1024;  // and the bars

// ------------------------------------------------------- pairs of CTAs, as inline PTX

__device__ __forceinline__ void pair_tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive once on `bar` in both CTAs when every MMA issued so far by this thread is done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// Arrive at the first CTA's barrier, in order after tensor-memory loads before a tc_fence_before ...
__device__ __forceinline__ void first_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_addr(bar), 0)) : "memory");
}
// ... or after the writes into this CTA's shared memory that this thread knows of (a releasing arrival would wait for all others, too,
// and take twice as long as a stage).
__device__ __forceinline__ void first_release(uint64_t* bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  first_arrive(bar);
}

template <typename T, bool kInner>
__global__ void __launch_bounds__(kThreads<kInner>, 1) many_kernel(const __grid_constant__ Args a) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kStep = kInner ? kHalf : 2 * kHalf;  // features from tile to tile
  constexpr int kWriters = kResults<kInner>;         // warps 2 .., after them those that gather
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Bars* b = reinterpret_cast<Bars*>(smem + kStages * kStage + 8 * kStageOut);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&b->full[i], 1 + (kInner ? 32 * kGatherWarps : 0) + (rank == 0 ? 1 : 0));
      mbar_init(&b->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->acc_full[i], 1);
      mbar_init(&b->acc_empty[i], 2 * kWriters);
    }
    fence_mbar_init();
    if (!kInner) tma_prefetch_desc(&a.tm_rows);
    tma_prefetch_desc(&a.tm_w[rank]);
  }
  if (warp == 1) pair_tmem_alloc(&b->tmem_base, 2 * kAccCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // (both CTAs' barriers are ready)
  tc_fence_after();
  const uint32_t tmem = b->tmem_base;
  pdl_wait();
  pdl_trigger();
  count_tiles<kRows, kThreads<kInner>>(a, b);
  Pieces<kRows, false> p(a, b, blockIdx.x / 2, gridDim.x / 2);
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      while (ok && p.next(kStep)) {
        for (int k = p.k0; k < p.k1; ++k, ++it) {
          const int st = it % kStages;
          ok = mbar_wait(&b->empty[st], ((it / kStages) & 1) ^ 1, &g_many_wait_timeouts);
          if (!ok) break;
          uint8_t* w = smem + st * kStage;
          mbar_arrive_expect_tx(&b->full[st], kInner ? kHalfBytes : kStage);
          load_half(w, &a.tm_w[rank], a.k_major, k * kBK, p.feature + (kInner ? 0 : rank * kHalf), p.expert, &b->full[st]);
          if (!kInner) tma_load_2d(w + kHalfBytes, &a.tm_rows, k * kBK, p.first + rank * kCtaRows, &b->full[st]);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 1) {
      int it = 0;
      while (ok && p.next(kStep)) {
        for (int k = p.k0; k < p.k1; ++k, ++it) {
          const int st = it % kStages;
          ok = mbar_wait(&b->full[st], (it / kStages) & 1, &g_many_wait_timeouts);
          if (!ok) break;
          if (kInner) fence_proxy_async();
          first_release(&b->full[st]);
        }
      }
    } else if (lane == 0) {
      const uint32_t w0 = smem_addr(smem), r0 = w0 + kHalfBytes;
      const uint64_t wd = a.k_major ? smem_desc_sw128(w0, 16, 1024) : smem_desc_sw128(w0, kHalfBytes / 2, 1024);
      const uint64_t wk = a.k_major ? 2 : 128;  // 16 inputs on, in 16 bytes
      const uint64_t rd = smem_desc_sw128(r0, 16, 1024);
      const uint32_t id = idesc_f16(kBf16, kRows, 2 * kHalf, false, !a.k_major);
      int it = 0;
      for (int acc = 0; ok && p.next(kStep); ++acc) {
        const int buf = acc & 1;
        ok = mbar_wait(&b->acc_empty[buf], ((acc >> 1) & 1) ^ 1, &g_many_wait_timeouts);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * kAccCols;
        for (int k = p.k0; k < p.k1; ++k, ++it) {
          const int st = it % kStages;
          ok = mbar_wait_cluster(&b->full[st], (it / kStages) & 1, &g_many_wait_timeouts);
          if (!ok) break;
          if (kInner) fence_proxy_async();
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>((st * kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            pair_mma(d, rd + so + kk * 2, wd + so + kk * wk, id, k > p.k0 || kk > 0 ? 1u : 0u);
          pair_commit(&b->empty[st]);
        }
        pair_commit(&b->acc_full[buf]);
      }
    }
  } else if (warp < 2 + kWriters) {
    const int quarter = warp & 3;  // of the lanes of tensor memory, which a warp's place decides
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int me = quarter * 32 + lane;
    for (int acc = 0; ok && p.next(kStep); ++acc) {
      const int buf = acc & 1;
      const uint32_t d = tmem + buf * kAccCols + lanes;
      const int rows = p.rows - rank * kCtaRows;  // this CTA's (none or less: it only helps)
      const int at = p.first + max(0, min(rank * kCtaRows + me, p.rows - 1));
      const int place = kInner ? at : a.order[at];  // of the pair's results, in out
      ok = mbar_wait(&b->acc_full[buf], (acc >> 1) & 1, &g_many_wait_timeouts);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // This thread has pair `me`, a column for each feature. 64 bytes (32 features of h, 16 of o) of the warp's 32 pairs at a
      // time go through shared memory, so that four lanes write 64 bytes of one row (a row for each lane would be 32 requests an
      // instruction).
      constexpr int kCols32 = (kInner ? kHalf : 2 * kHalf) / 32 / (kWriters / 4);  // that a warp has, from the first-th on
      const int first = (warp - 2) / 4 * kCols32;
      uint8_t* stage = smem + kStages * kStage + (warp - 2) * kStageOut;
      const int chunk = lane & 3;
      const auto put = [&](const uint4* q, auto* out, int f0) {
        constexpr int kEach = 16 / sizeof(*out);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = q[j];
        __syncwarp();
        const int f = f0 + chunk * kEach;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 2);
          const int64_t to = __shfl_sync(0xffffffffu, place, r);
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4));
          // (rows of out are 16-byte aligned and padded to a multiple of 16 elements)
          if (quarter * 32 + r < rows && f < a.features) *reinterpret_cast<uint4*>(out + to * a.out_step + f) = v;
        }
        __syncwarp();
      };
#pragma unroll
      for (int h = 0; h < kCols32; ++h) {
        const int c0 = (first + h) * 32;
        uint32_t x[2][16], y[2][16];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          tmem_ld16_nowait(d + c0 + 16 * i, x[i]);
          if (kInner) tmem_ld16_nowait(d + kHalf + c0 + 16 * i, y[i]);
        }
        // (all at once: lanes may part below, and the wait is one of the whole warp)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          tmem_ld_wait_r(x[i]);
          if (kInner) tmem_ld_wait_r(y[i]);
        }
        if constexpr (kInner) {
          uint4 q[4];
          float v[32];
          float most = 0.0f;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            v[j] = gated(__uint_as_float(x[j / 16][j % 16]), __uint_as_float(y[j / 16][j % 16]));
            if (!kBf16) most = fmaxf(most, fabsf(v[j]));
          }
          if (!kBf16 && most > kMostHalf && me < rows) {  // (or infinite)
            const int64_t pair = a.order[at];
            float4* to = reinterpret_cast<float4*>(a.excess.values + pair * a.excess.step + p.feature + c0);
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              to[j / 4] = make_float4(excess_of(v[j]), excess_of(v[j + 1]), excess_of(v[j + 2]), excess_of(v[j + 3]));
            mark_excess(a.excess, pair, p.feature + c0);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = saturate<T>(v[j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) q[j] = V8<T>::pack(v + 8 * j);
          put(q, static_cast<T*>(a.out), p.feature + c0);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = make_uint4(x[i][4 * j], x[i][4 * j + 1], x[i][4 * j + 2], x[i][4 * j + 3]);
            put(q, static_cast<float*>(a.out), p.feature + c0 + 16 * i);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) first_arrive(&b->acc_empty[buf]);
    }
  } else if constexpr (kInner) {
    const int group = warp - 2 - kWriters;
    Gather<T> g;
    int it = 0;
    while (ok && p.next(kStep)) {
      g.begin(a, p.first + min(rank * kCtaRows, p.rows - 1), p.rows - rank * kCtaRows, group);
      for (int k = p.k0; k < p.k1; ++k, ++it) {
        const int st = it % kStages;
        if (lane == 0) ok = mbar_wait(&b->empty[st], ((it / kStages) & 1) ^ 1, &g_many_wait_timeouts);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        g.copy(a, smem_addr(smem) + st * kStage + kHalfBytes, k * kBK, group, &b->full[st]);
      }
    }
    cp_async_wait_all();
  }
  if (!ok) *a.gave_up = 1u;
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // (nothing is on its way to the other CTA any more)
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, 2 * kAccCols);
  }
}

template <typename T, bool kInner>
cudaError_t launch_product(const Args& a, const hc_expert_mlp_t& p, int num_sms, cudaStream_t s) {
  const int64_t tiles = experts_um_tiles(p, kRows, kInner);
  const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(num_sms / 2, tiles));
  const size_t smem = kSmem + bars_bytes(a.experts);
  const cudaError_t e = ensure_smem<many_kernel<T, kInner>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(many_kernel<T, kInner>, dim3(grid), dim3(kThreads<kInner>), smem, s, 2, a);
}

template <typename T> cudaError_t launch_both(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  for (const bool inner : {true, false}) {
    Args a;
    if (!fill_args(&a, p, u, inner, kCtaRows)) return cudaErrorInvalidValue;
    e = inner ? launch_product<T, true>(a, p, num_sms, s) : launch_product<T, false>(a, p, num_sms, s);
    if (e != cudaSuccess) break;
  }
  return e;
}

}  // namespace

cudaError_t launch_experts_many(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s) {
  return p.dtype == HC_F16 ? launch_both<__half>(p, u, num_sms, s) : launch_both<__nv_bfloat16>(p, u, num_sms, s);
}

unsigned int read_experts_many_wait_timeouts(bool reset) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_many_wait_timeouts, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (reset) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_many_wait_timeouts, &z, sizeof(z));
  }
  return v;
}

}  // namespace hc
