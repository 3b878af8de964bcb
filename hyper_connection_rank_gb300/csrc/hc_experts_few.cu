// The experts' products on the tensor cores where experts have few pairs (a serving
// batch of single tokens): the weights are the MMA's A operand and the pairs its
// columns, D (128 features x pairs) += W (128 x 64) R (64 x pairs), for both halves
// of a tile. A weight's 128 rows fill the tensor core however few pairs there are.
//
// Bound: the bytes of the weights. All tiles' blocks of inputs, laid end to end, are cut into equal runs, one for each SM (or,
// with fewer tiles than SMs, each tile into equal parts), so that one token with eight experts and a batch that hits all of
// them keep every SM's copies going; see Pieces. A piece of a tile that was cut is written as partial sums: the inner
// product's go to memory of their own, and the CTA that finishes a tile last adds them up in the order of the pieces, so
// that which one that is does not show in the result; the outer product's go to planes of o, which the sum over a token's
// experts adds up. Pieces of cut tiles come first in a run, so that their sums are joined while whole tiles are on their way.
//
// The outer product's CTAs share the SMs with the inner one's and have their first weights when those finish, and the inner
// one's send the weights after those to L2 before their last sums.
//
// 61 tokens at six of 64 experts of 2560 x 640 in bf16 (629 MB of weights): the call takes 108 us, 5.8 TB/s, 86% of measured
// copy bandwidth; the inner product reads at 74% of DRAM's cycles, the outer one, which starts in its shadow, at 65%. One token at
// eight experts (79 MB): 27 us against 11.6 for the bytes; the rest is four kernels' latencies. (Equal parts of few tiles took one
// token from 34 to 27 us; the two products' overlap 61 tokens from 120 to 114, cut tiles first from 117 to 109.)
//
// One warp copies weights, one issues MMAs, four write results, and for the inner product a warp gathers rows; stages are
// handed over through mbarriers (all waits bounded, see hc_async.cuh).
#include <algorithm>

#include "hc_experts_um.cuh"

namespace hc {

__device__ unsigned int g_few_wait_timeouts = 0;

namespace {

using namespace um;

constexpr int kRows = 32;  // pairs of a tile
constexpr int kStage = 2 * kHalfBytes + kRows * kBK * 2;
// As few stages as let two CTAs share an SM (up to some 470 experts), so that the outer product's are there, with their first
// weights, when the inner one's finish.
constexpr int kStages = 3;
constexpr int kCols = 4 * kRows;  // of tensor memory: two accumulators of two halves each
constexpr size_t kSmem = kStages * kStage + 1024;  // and the bars
constexpr int kFetched = 8;  // units of 32 KB
template <bool kInner> constexpr int kThreads = 192 + (kInner ? 32 : 0);

template <typename T, bool kInner>
__global__ void __launch_bounds__(kThreads<kInner>, 2) few_kernel(const __grid_constant__ Args a, const __grid_constant__ Args outer) {
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kStep = kInner ? kHalf : 2 * kHalf;  // features from tile to tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Bars* b = reinterpret_cast<Bars*>(smem + kStages * kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&b->full[i], kInner ? 1 + 32 : 1);
      mbar_init(&b->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->acc_full[i], 1);
      mbar_init(&b->acc_empty[i], 4);
    }
    fence_mbar_init();
    if (!kInner) tma_prefetch_desc(&a.tm_rows);
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
  // The outer product needs the inner one's results for its rows only. What comes before that was there when this kernel
  // began: the inner product's CTAs let it begin after they had waited for the lists, and the weights are older.
  if (kInner) {
    pdl_wait();
    pdl_trigger();
  }
  count_tiles<kRows, kThreads<kInner>>(a, b);
  Pieces<kRows, true> p(a, b, blockIdx.x, gridDim.x);
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      const auto weights = [&](int st, int k, const Pieces<kRows, true>& p) {
        uint8_t* w = smem + st * kStage;
        mbar_arrive_expect_tx(&b->full[st], kInner ? 2 * kHalfBytes : kStage);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          load_half(w + h * kHalfBytes, &a.tm_w[h], a.k_major, k * kBK, p.feature + (kInner ? 0 : h * kHalf), p.expert,
                    &b->full[st]);
      };
      int early = 0;  // stages whose weights are on their way before the wait
      if (!kInner) {
        Pieces<kRows, true> q = p;
        while (early < kStages && q.next(kStep))
          for (int k = q.k0; k < q.k1 && early < kStages; ++k) weights(early++, k, q);
        pdl_wait();
        pdl_trigger();
      }
      int it = 0;
      while (ok && p.next(kStep)) {
        for (int k = p.k0; k < p.k1; ++k, ++it) {
          const int st = it % kStages;
          if (it >= early) {
            ok = mbar_wait(&b->empty[st], ((it / kStages) & 1) ^ 1, &g_few_wait_timeouts);
            if (!ok) break;
            weights(st, k, p);
          }
          if (!kInner) tma_load_2d(smem + st * kStage + 2 * kHalfBytes, &a.tm_rows, k * kBK, p.first, &b->full[st]);
        }
      }
      if (kInner) {
        // While the last sums are formed and joined, the memory would have nothing to do: the outer product's weights of
        // this place, past those that its stages hold, go to L2.
        Pieces<kRows, true> q(outer, b, blockIdx.x, gridDim.x);
        int unit = 0;
        while (unit < kFetched && q.next(2 * kHalf))
          for (int k = q.k0; k < q.k1 && unit < kFetched; ++k, ++unit)
            if (unit >= kStages)
              for (int h = 0; h < 2; ++h)
                prefetch_half(&outer.tm_w[h], outer.k_major, k * kBK, q.feature + h * kHalf, q.expert);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t w0 = smem_addr(smem), r0 = w0 + 2 * kHalfBytes;
      const uint64_t wd = a.k_major ? smem_desc_sw128(w0, 16, 1024) : smem_desc_sw128(w0, kHalfBytes / 2, 1024);
      const uint64_t wk = a.k_major ? 2 : 128;  // 16 inputs on, in 16 bytes
      const uint64_t rd = smem_desc_sw128(r0, 16, 1024);
      const uint32_t id = idesc_f16(kBf16, 128, kRows, !a.k_major, false);
      int it = 0;
      for (int acc = 0; ok && p.next(kStep); ++acc) {
        const int buf = acc & 1;
        ok = mbar_wait(&b->acc_empty[buf], ((acc >> 1) & 1) ^ 1, &g_few_wait_timeouts);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * 2 * kRows;
        for (int k = p.k0; k < p.k1; ++k, ++it) {
          const int st = it % kStages;
          ok = mbar_wait(&b->full[st], (it / kStages) & 1, &g_few_wait_timeouts);
          if (!ok) break;
          if (kInner) fence_proxy_async();
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>((st * kStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint32_t add = k > p.k0 || kk > 0 ? 1u : 0u;
            const uint64_t w = wd + so + kk * wk, r = rd + so + kk * 2;
            mma_f16(d, w, r, id, add);
            mma_f16(d + kRows, w + (kHalfBytes >> 4), r, id, add);
          }
          mma_commit(&b->empty[st]);
        }
        mma_commit(&b->acc_full[buf]);
      }
    }
  } else if (warp < 6) {
    if (!kInner) pdl_wait();  // (where its results go, others may still read until then)
    const int quarter = warp & 3;  // of the lanes of tensor memory, which a warp's place decides
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int me = quarter * 32 + lane;
    const auto meet = [] {  // (of the four warps)
      __syncwarp();
      named_bar_sync(1, 128);
    };
    for (int acc = 0; ok && p.next(kStep); ++acc) {
      const int buf = acc & 1;
      const uint32_t d = tmem + buf * 2 * kRows + lanes;
      const int at = p.first + min(lane, p.rows - 1), place = kInner ? at : a.order[at];  // of the lane's pair, in out
      ok = mbar_wait(&b->acc_full[buf], (acc >> 1) & 1, &g_few_wait_timeouts);
      // The inner product's four warps meet below where a piece of a cut tile is joined, so there they go on as one; whole tiles
      // come behind all of those, and a warp that leaves at one of them leaves nobody waiting.
      ok = kInner && !p.whole() ? named_bar_all(1, 128, ok) : __all_sync(0xffffffffu, ok) != 0;
      if (!ok) break;
      tc_fence_after();
      // this thread has feature `me` of both halves, a column for each pair
      // (a piece of the outer product goes to a plane of its own, which the sum over a token's experts adds to the others)
      const bool whole = !kInner || p.whole();
      const int f = p.feature + me;
      float* o = static_cast<float*>(a.out) + (kInner ? 0 : p.piece() * a.plane);
      const auto put = [&](int c, float v0, float v1) {
        const int64_t to = static_cast<int64_t>(__shfl_sync(0xffffffffu, place, c)) * a.out_step;
        if constexpr (kInner) {
          const float h = gated(v0, v1);
          if (f < a.features) stf(static_cast<T*>(a.out) + to + f, saturate<T>(h));
          if constexpr (!kBf16) {
            if (__any_sync(0xffffffffu, f < a.features && past_half(h))) {  // (32 features from a multiple of 32 on)
              const int64_t pair = a.order[p.first + c];
              if (f < a.features) a.excess.values[pair * a.excess.step + f] = excess_of(h);
              if (lane == 0) mark_excess(a.excess, pair, f);
            }
          }
        } else {
          if (f < a.features) o[to + f] = v0;
          if (f + kHalf < a.features) o[to + f + kHalf] = v1;
        }
      };
      if (!kInner && warp == 2 && lane < p.rows)
        a.counts[place * a.count_step + p.feature / (2 * kHalf)] = static_cast<uint8_t>(p.pieces());
      float* part = a.part + static_cast<int64_t>(p.place(blockIdx.x)) * (2 * kRows * kHalf) + me;
#pragma unroll
      for (int c0 = 0; c0 < kRows; c0 += 16) {
        if (c0 < p.rows) {
          float v[2][16];
          __syncwarp();  // (lanes part where they write, and the loads are the whole warp's)
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
        uint32_t c0, c1;
        p.sharers(&c0, &c1);
        __threadfence();
        meet();
        if (warp == 2 && lane == 0) b->last = atomicAdd(&a.tickets[p.tile], 1u) == c1 - c0;
        meet();
        if (b->last != 0) {
          __threadfence();
          // sums of kAt pairs from kOf CTAs' pieces at a time, so that their loads overlap
          const auto join = [&](auto at_once, auto pieces) {
            constexpr int kAt = decltype(at_once)::value, kOf = decltype(pieces)::value;
            for (int b0 = 0; b0 < p.rows; b0 += kAt) {
              float v[2][kAt] = {};
              for (uint32_t q0 = c0; q0 <= c1; q0 += kOf) {
                float w[kOf][2][kAt];
#pragma unroll
                for (int q = 0; q < kOf; ++q) {
                  const float* from = a.part + static_cast<int64_t>(p.place(min(q0 + q, c1))) * (2 * kRows * kHalf) + b0 * kHalf + me;
#pragma unroll
                  for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < kAt; ++c)
                      w[q][h][c] = q0 + q <= c1 && b0 + c < p.rows ? __ldcg(from + (h * kRows + c) * kHalf) : 0.0f;
                }
#pragma unroll
                for (int q = 0; q < kOf; ++q)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < kAt; ++c) v[h][c] += w[q][h][c];
              }
#pragma unroll
              for (int c = 0; c < kAt; ++c)
                if (b0 + c < p.rows) put(b0 + c, v[0][c], v[1][c]);
            }
          };
          if (p.rows <= 4) join(std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
          else join(std::integral_constant<int, 8>(), std::integral_constant<int, 2>());
        }
        meet();  // (`last` is read before it is written again)
      }
    }
  } else if constexpr (kInner) {
    Gather<T> g;
    int it = 0;
    while (ok && p.next(kStep)) {
      g.begin(a, p.first, p.rows, 0);
      for (int k = p.k0; k < p.k1; ++k, ++it) {
        const int st = it % kStages;
        if (lane == 0) ok = mbar_wait(&b->empty[st], ((it / kStages) & 1) ^ 1, &g_few_wait_timeouts);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        g.copy(a, smem_addr(smem) + st * kStage + 2 * kHalfBytes, k * kBK, 0, &b->full[st]);
      }
    }
    cp_async_wait_all();
  }
  if (!ok) *a.gave_up = 1u;
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <typename T, bool kInner>
cudaError_t launch_product(const Args& a, const Args& outer, int num_sms, cudaStream_t s) {
  const size_t smem = kSmem + bars_bytes(a.experts);
  const cudaError_t e = ensure_smem<few_kernel<T, kInner>>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(few_kernel<T, kInner>, dim3(static_cast<unsigned>(num_sms)), dim3(kThreads<kInner>), smem, s, 1, a, outer);
}

template <typename T> cudaError_t launch_both(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s) {
  Args inner, outer;
  if (!fill_args(&inner, p, u, true, kRows) || !fill_args(&outer, p, u, false, kRows)) return cudaErrorInvalidValue;
  inner.part = u.part;
  inner.tickets = u.tickets;
  inner.most_parts = inner.kblocks;
  outer.plane = u.plane;
  outer.most_parts = u.planes;
  const cudaError_t e = launch_product<T, true>(inner, outer, num_sms, s);
  return e != cudaSuccess ? e : launch_product<T, false>(outer, outer, num_sms, s);
}

}  // namespace

namespace um {

bool map_rows(CUtensorMap* m, const void* base, bool bf16, int64_t cols, int64_t rows, int64_t step, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(step) * 2};
  const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
  const auto fn = tmap_encoder();
  return fn != nullptr &&
         fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_weight(CUtensorMap* m, const void* base, bool bf16, int experts, int inputs, int outputs, int64_t es, int64_t is,
                int64_t os) {
  const bool k_major = is == 1;
  const int64_t cols = k_major ? inputs : outputs, rows = k_major ? outputs : inputs, step = k_major ? os : is;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(experts)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(step) * 2, static_cast<cuuint64_t>(experts > 1 ? es : rows * step) * 2};
  const cuuint32_t box[3] = {kBK, static_cast<cuuint32_t>(k_major ? kHalf : kBK), 1}, one[3] = {1, 1, 1};
  const auto fn = tmap_encoder();
  return fn != nullptr &&
         fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool fill_args(Args* a, const hc_expert_mlp_t& p, const ExpertUm& u, bool inner, int box_rows) {
  const bool bf16 = p.dtype == HC_BF16;
  *a = Args{};
  a->bounds = u.lists.bounds;
  a->order = u.lists.order;
  a->excess = u.excess;
  a->gave_up = u.gave_up;
  a->x = p.x;
  a->x_step = p.x_stride;
  a->out = inner ? u.h : static_cast<void*>(u.o);
  a->out_step = inner ? u.h_step : u.o_step;
  a->counts = u.counts;
  a->count_step = u.count_step;
  a->experts = p.num_experts;
  a->top_k = p.top_k;
  a->inputs = inner ? p.hidden : p.inner;
  a->features = inner ? p.inner : p.hidden;
  a->kblocks = (a->inputs + kBK - 1) / kBK;
  a->fblocks = (a->features + (inner ? kHalf : 2 * kHalf) - 1) / (inner ? kHalf : 2 * kHalf);
  const int64_t es = inner ? p.up_expert_stride : p.down_expert_stride, is = inner ? p.up_in_stride : p.down_in_stride,
                os = inner ? p.up_out_stride : p.down_out_stride;
  a->k_major = is == 1;
  return (inner || map_rows(&a->tm_rows, u.h, bf16, p.inner, p.tokens * p.top_k, u.h_step, box_rows)) &&
         map_weight(&a->tm_w[0], inner ? p.gate : p.down, bf16, p.num_experts, a->inputs, a->features, es, is, os) &&
         map_weight(&a->tm_w[1], inner ? p.up : p.down, bf16, p.num_experts, a->inputs, a->features, es, is, os);
}

}  // namespace um

int64_t experts_um_tiles(const hc_expert_mlp_t& p, int rows, bool inner) {
  const int64_t pairs = p.tokens * p.top_k, step = inner ? um::kHalf : 2 * um::kHalf, features = inner ? p.inner : p.hidden;
  return std::min(pairs, pairs / rows + p.num_experts) * ((features + step - 1) / step);
}

cudaError_t launch_experts_few(const hc_expert_mlp_t& p, const ExpertUm& u, int num_sms, cudaStream_t s) {
  return p.dtype == HC_F16 ? launch_both<__half>(p, u, num_sms, s) : launch_both<__nv_bfloat16>(p, u, num_sms, s);
}

// Four warps wait by themselves, those in `stuck` for an mbarrier that nothing arrives on, and go on as one.
__global__ void __launch_bounds__(128) wait_together_probe(float* out, unsigned int stuck, long long limit) {
  __shared__ uint64_t bars[2];
  if (threadIdx.x == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_arrive(&bars[0]);
  const bool ok = mbar_wait_limit(&bars[stuck >> (threadIdx.x >> 5) & 1u], 0, &g_few_wait_timeouts, limit);
  const bool all = named_bar_all(1, 128, ok);
  if (all) named_bar_sync(1, 128);
  out[threadIdx.x] = all ? 1.0f : __int_as_float(0x7fc00000);
}

cudaError_t launch_wait_together_probe(float* out, unsigned int stuck, long long limit_cycles, cudaStream_t s) {
  wait_together_probe<<<1, 128, 0, s>>>(out, stuck, limit_cycles);
  return cudaGetLastError();
}

unsigned int read_experts_few_wait_timeouts(bool reset) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_few_wait_timeouts, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (reset) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_few_wait_timeouts, &z, sizeof(z));
  }
  return v;
}

}  // namespace hc
