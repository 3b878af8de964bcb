// The experts' products (hc_expert_mlp): lists of the pairs by expert, the general
// kernels for any shape, stride and type, and the sum over a token's experts.
//
//   lists_kernel    a CTA per expert: bounds and the sorted list of pairs
//   general_kernel  h = silu(x gate) * (x up), a row for each pair, in the list's order;
//                   then o = h down, a row for each pair, at the pair's own place
//   combine_kernel  out_t = sum_j weights[t, j] o[t top_k + j], in the order of j
#include <algorithm>
#include <type_traits>

#include "hc_async.cuh"
#include "hc_common.cuh"
#include "hc_experts.cuh"
#include "hc_two.cuh"
#include "hc_vec.cuh"

namespace hc {
namespace {

// ------------------------------------------------------------------ lists --

// CTA e counts the pairs of the experts before e, which is where its own begin, and its own in each warp's run of pairs;
// then every warp writes its own. All CTAs read all experts (tokens * top_k numbers from L2), and none waits for another.
// Together they clear the words that the products count and mark in.
// Bound: latency up to some thousand pairs (5 us by itself, less behind the call before), issue beyond (65528 pairs and 64
// experts: 15 us).
template <int kThreads>
__global__ void __launch_bounds__(kThreads)
lists_kernel(const int32_t* __restrict__ ids, int pairs, int experts, ExpertLists lists, unsigned int* zeros, int64_t num_zeros) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int own[kWarps], less[kWarps];
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t i = e * kThreads + threadIdx.x; i < num_zeros; i += experts * kThreads) zeros[i] = 0;
  // four neighbouring pairs to a lane, 128 to a warp's step
  const bool vec = (reinterpret_cast<uintptr_t>(ids) & 15u) == 0;
  const auto load4 = [&](int i) {
    if (vec && i + 4 <= pairs) return *reinterpret_cast<const int4*>(ids + i);
    return make_int4(i < pairs ? ids[i] : -1, i + 1 < pairs ? ids[i + 1] : -1, i + 2 < pairs ? ids[i + 2] : -1,
                     i + 3 < pairs ? ids[i + 3] : -1);
  };
  const int run = (pairs + kThreads * 4 - 1) / (kThreads * 4) * 128;
  const int lo = min(pairs, warp * run), hi = min(pairs, lo + run);
  int mine = 0, before = 0;
#pragma unroll 4
  for (int i = lo + lane * 4; i < hi; i += 128) {
    const int4 v = load4(i);
    mine += (v.x == e) + (v.y == e) + (v.z == e) + (v.w == e);
    const auto less_than = [&](int id) { return id >= 0 && id < e; };
    before += less_than(v.x) + less_than(v.y) + less_than(v.z) + less_than(v.w);
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) {
    own[warp] = mine;
    less[warp] = before;
  }
  __syncthreads();
  int at = 0, end = 0;
  for (int w = 0; w < kWarps; ++w) {
    at += less[w] + (w < warp ? own[w] : 0);
    end += less[w] + own[w];
  }
  if (threadIdx.x == 0) {
    lists.bounds[e] = at;
    if (e == experts - 1) lists.bounds[experts] = end;
  }
  if (mine == 0) return;
  constexpr int kAhead = 4;
  const unsigned below = (1u << lane) - 1u;
  for (int i0 = lo; i0 < hi; i0 += 128 * kAhead) {
    int4 v[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      v[j] = i0 + 128 * j + lane * 4 < hi ? load4(i0 + 128 * j + lane * 4) : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const bool hit[4] = {v[j].x == e, v[j].y == e, v[j].z == e, v[j].w == e};
      int rank = 0, all = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const unsigned hits = __ballot_sync(0xffffffffu, hit[c]);
        rank += __popc(hits & below);
        all += __popc(hits);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (hit[c]) lists.order[at + rank++] = i0 + 128 * j + lane * 4 + c;
      at += all;
    }
  }
}

// ------------------------------------------------------- general products --
//
// On the CUDA cores in fp32, for float32 and for any type, stride and alignment. A CTA takes units of up to 24 pairs of one
// expert (its pairs are cut evenly) and 32 kPer features of gate and up (64 kPer of down, as two halves). Its four warps
// share the inputs among them, eight at a time; a lane has kPer features of both matrices, and sums of two rows in one packed
// multiply-add. A weight is used by one lane alone, so it goes from global memory to a register, eight inputs ahead (where
// inputs are contiguous, by way of the warp's shared memory, so that eight lanes read neighbouring inputs of a feature: a
// feature to a lane took three times as long). Rows come through a warp's own shared memory, an input of four rows to a
// broadcast load for 4 kPer multiply-adds of two. Sums of the four warps are added at the end, so that a sum of n products is
// four of n / 4 (one of n was off by twice as much).
//
// Bound: the CUDA cores' multiply-adds with rows to spare, the weights' bytes without. 131 tokens at three of 12 experts of
// 1280 x 704 in fp32 take 57 and 33 us for the two products, 25 and 21 TFLOP/s, where the busiest SM has half as much again as
// the average one; 2000 tokens take 529 and 289 us, 41 and 37 TFLOP/s of some 75.
//
// Two features to a lane need fewer loads to a multiply-add, one leaves registers for a third CTA to an SM and gives twice
// as many units: with one and two, 131 tokens took 57 and 62 us (inner) and 33 and 38 (outer; 73 and 90, 41 and 50 with the
// inputs contiguous), 300 tokens 109 and 107, 60 and 63, 600 tokens 200 and 174, 99 and 101, 2000 tokens 625 and 529, 319
// and 289. One is for calls that have fewer units of two than two rounds of CTAs.

constexpr int kGroup = 4, kGroups = 6, kTM = kGroup * kGroups;  // pairs of a tile, in groups that are left out if empty
constexpr int kTK = 8, kGenWarps = 4, kGenThreads = 32 * kGenWarps;
constexpr int kRowStep = kTM + 4;  // rows of an input in shared memory (28 words: eight inputs' rows in different banks)

struct GeneralArgs {
  hc_expert_mlp_t p;
  ExpertLists lists;
  float *h, *o;  // (pairs, inner) in the list's order, (pairs, hidden) at the pairs' places
  int64_t o_step;
};

// Tiles of each expert's pairs (as few as hold them, cut evenly), summed up: upto[e] before expert e. All threads.
__device__ __forceinline__ void count_even_tiles(const int32_t* bounds, int experts, int* upto) {
  __shared__ int red[kGenWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, each = (experts + kGenThreads - 1) / kGenThreads;
  const int lo = min(experts, static_cast<int>(threadIdx.x) * each), hi = min(experts, lo + each);
  int mine = 0;
  for (int e = lo; e < hi; ++e) mine += (bounds[e + 1] - bounds[e] + kTM - 1) / kTM;
  int before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) red[warp] = before;
  __syncthreads();
  before -= mine;
  for (int w = 0; w < warp; ++w) before += red[w];
  for (int e = lo; e < hi; ++e) {
    upto[e] = before;
    before += (bounds[e + 1] - bounds[e] + kTM - 1) / kTM;
  }
  if (hi == experts) upto[experts] = before;  // (the same from every thread that has the last one or none)
  __syncthreads();
}

template <typename T, bool kInner, bool kByInput, int kPer>
__global__ void __launch_bounds__(kGenThreads, kPer == 1 ? 3 : 2) general_kernel(GeneralArgs g) {
  constexpr int kTN = 32 * kPer;
  constexpr int kAcc = kTM * 2 * kPer;  // sums of a lane
  using In = typename std::conditional<kInner, T, float>::type;
  extern __shared__ __align__(16) float smem[];
  const hc_expert_mlp_t& p = g.p;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inputs = kInner ? p.hidden : p.inner, features = kInner ? p.inner : p.hidden;
  const int64_t is = kInner ? p.up_in_stride : p.down_in_stride, os = kInner ? p.up_out_stride : p.down_out_stride;
  constexpr int kStep = kTN * (kInner ? 1 : 2);  // features of a unit
  int* upto = reinterpret_cast<int*>(smem + kGenWarps * kAcc * 32);
  count_even_tiles(g.lists.bounds, p.num_experts, upto);
  const int blocks = (features + kStep - 1) / kStep, units = upto[p.num_experts] * blocks;
  float* rows = smem + warp * (2 * kTK * kRowStep);
  float* turned = smem + kGenWarps * (2 * kTK * kRowStep) + warp * (2 * kPer * 32 * kTK);  // weights on their way to their lanes
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int tile = unit / blocks, n0 = (unit - tile * blocks) * kStep;
    int expert = 0;  // the last one whose tiles begin here or before (empty ones have none)
    for (int hi = p.num_experts - 1; expert < hi;) {
      const int mid = (expert + hi + 1) >> 1;
      if (upto[mid] <= tile) expert = mid;
      else hi = mid - 1;
    }
    const int begin = g.lists.bounds[expert], pairs = g.lists.bounds[expert + 1] - begin;
    const int each = (pairs + upto[expert + 1] - upto[expert] - 1) / (upto[expert + 1] - upto[expert]);
    const int first = begin + (tile - upto[expert]) * each, count = min(each, begin + pairs - first);
    if (count <= 0) continue;  // (even shares can leave the last tile nothing)
    // [matrix or half][of the lane's two features]; with kByInput the lane reads input lane % 8 of features lane / 8, + 4, ...
    const T* w[2][kPer];
    bool have[2][kPer];
    const int mine = kByInput ? lane / 8 : lane;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int f = n0 + mine + 32 * j + (kInner ? 0 : kTN * m);
        have[m][j] = f < features;
        w[m][j] = static_cast<const T*>(kInner ? (m ? p.up : p.gate) : p.down) +
                  expert * (kInner ? p.up_expert_stride : p.down_expert_stride) + (have[m][j] ? f : 0) * os + (kByInput ? lane % 8 : 0);
      }
    // the lane's six elements of a block of rows: input lane % 8 of rows lane / 8, + 4, ...
    const In* x[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) {
      const int at = first + min(lane / 8 + 4 * i, count - 1);
      x[i] = (kInner ? static_cast<const In*>(p.x) + static_cast<int64_t>(g.lists.order[at] / p.top_k) * p.x_stride
                     : reinterpret_cast<const In*>(g.h) + static_cast<int64_t>(at) * p.inner) + lane % 8;
    }
    const int groups = (count + kGroup - 1) / kGroup;
    Two acc[kTM / 2][2][kPer];  // of two rows each
#pragma unroll
    for (int r = 0; r < kTM / 2; ++r)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < kPer; ++j) acc[r][m][j] = Two(0.0f);
    float wn[kTK][2][kPer], xn[6];
    const auto load = [&](int k0) {
#pragma unroll
      for (int i = 0; i < 6; ++i) xn[i] = k0 + lane % 8 < inputs ? ldf(x[i] + k0) : 0.0f;
#pragma unroll
      for (int k = 0; k < kTK; ++k)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            if (kByInput) {
              const bool in = k0 + lane % 8 < inputs && n0 + mine + 4 * k + 32 * j + (kInner ? 0 : kTN * m) < features;
              wn[k][m][j] = in ? ldf(w[m][j] + k0 + 4 * k * os) : 0.0f;
            } else {
              wn[k][m][j] = have[m][j] && k0 + k < inputs ? ldf(w[m][j] + (k0 + k) * is) : 0.0f;
            }
          }
    };
    __syncthreads();  // (the last unit's sums are read)
    if (warp * kTK < inputs) load(warp * kTK);
    int turn = 0;
    for (int k0 = warp * kTK; k0 < inputs; k0 += kGenWarps * kTK, turn ^= 1) {
      float* buf = rows + turn * (kTK * kRowStep);
#pragma unroll
      for (int i = 0; i < 6; ++i) buf[lane % 8 * kRowStep + lane / 8 + 4 * i] = xn[i];
      float wc[kTK][2][kPer];
      if (kByInput) {
        // feature f's inputs in 32 bytes, their halves exchanged for every other four features (no bank is hit twice)
#pragma unroll
        for (int k = 0; k < kTK; ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < kPer; ++j)
              turned[((m * kPer + j) * 32 + 4 * k + lane / 8) * 8 + ((lane % 8) ^ (4 * (k & 1)))] = wn[k][m][j];
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < kPer; ++j)
#pragma unroll
            for (int k4 = 0; k4 < kTK; k4 += 4) {
              const float4 v = *reinterpret_cast<const float4*>(turned + ((m * kPer + j) * 32 + lane) * 8 + (k4 ^ (lane & 4)));
              wc[k4][m][j] = v.x, wc[k4 + 1][m][j] = v.y, wc[k4 + 2][m][j] = v.z, wc[k4 + 3][m][j] = v.w;
            }
      } else {
#pragma unroll
        for (int k = 0; k < kTK; ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int j = 0; j < kPer; ++j) wc[k][m][j] = wn[k][m][j];
      }
      __syncwarp();
      if (k0 + kGenWarps * kTK < inputs) load(k0 + kGenWarps * kTK);
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        if (q < groups) {
#pragma unroll
          for (int k = 0; k < kTK; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(buf + k * kRowStep + q * kGroup);
            const Two xs[2] = {Two(v.x, v.y), Two(v.z, v.w)};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int j = 0; j < kPer; ++j) acc[2 * q + i][m][j] = fma2(xs[i], Two(wc[k][m][j]), acc[2 * q + i][m][j]);
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kTM / 2; ++r)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (2 * r < groups * kGroup) {
            const float2 v = acc[r][m][j].get();
            smem[(warp * kAcc + (2 * r * 2 + m) * kPer + j) * 32 + lane] = v.x;
            smem[(warp * kAcc + ((2 * r + 1) * 2 + m) * kPer + j) * 32 + lane] = v.y;
          }
    __syncthreads();
    const auto sum = [&](int r, int m, int f) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kGenWarps; ++i) v += smem[(i * kAcc + (r * 2 + m) * kPer + (f >> 5)) * 32 + (f & 31)];
      return v;
    };
    for (int i = threadIdx.x; i < count * kTN; i += kGenThreads) {
      const int r = i / kTN, f = i % kTN;
      const int64_t at = first + r;
      const float v0 = sum(r, 0, f), v1 = sum(r, 1, f);
      if (kInner) {
        const float e = expf(-0.5f * fabsf(v0));
        if (n0 + f < features) g.h[at * p.inner + n0 + f] = silu_times(v0, v1, e, 1.0f / fmaf(e, e, 1.0f));
      } else {
        float* to = g.o + g.lists.order[at] * g.o_step + n0 + f;
        if (n0 + f < features) to[0] = v0;
        if (n0 + f + kTN < features) to[kTN] = v1;
      }
    }
  }
}

template <typename T, bool kInner> cudaError_t launch_general(const GeneralArgs& g, int num_sms, cudaStream_t s) {
  const auto launch = [&](auto by_input, auto per) {
    constexpr bool kByInput = decltype(by_input)::value;
    constexpr int kPer = decltype(per)::value;
    // (the sums, which take more than the rows and weights before them, and the tiles)
    const size_t smem = sizeof(float) * kGenWarps * kTM * 2 * kPer * 32 + sizeof(int) * (g.p.num_experts + 1);
    const cudaError_t e = ensure_smem<general_kernel<T, kInner, kByInput, kPer>>(smem);
    const dim3 grid((kPer == 1 ? 3 : 2) * num_sms);
    return e != cudaSuccess ? e : launch_pdl(general_kernel<T, kInner, kByInput, kPer>, grid, dim3(kGenThreads), smem, s, 1, g);
  };
  const int64_t pairs = g.p.tokens * g.p.top_k, step = kInner ? 64 : 128, features = kInner ? g.p.inner : g.p.hidden;
  const int64_t units = (pairs / kTM + std::min<int64_t>(pairs, g.p.num_experts) / 2 + 1) * ((features + step - 1) / step);
  const auto one = [&](auto by_input) {
    return units < 4 * num_sms ? launch(by_input, std::integral_constant<int, 1>()) : launch(by_input, std::integral_constant<int, 2>());
  };
  return (kInner ? g.p.up_out_stride : g.p.down_out_stride) == 1 ? one(std::false_type()) : one(std::true_type());
}

// ---------------------------------------------------------------- combine --

// A warp has 256 features of a token, eight to a lane, and loads four or eight experts' rows at a time (rows of o are padded to a
// multiple of sixteen). With kPlanes an expert's result is the sum of some planes of o, counts[] of them.
// Bound: bytes, top_k rows of floats and one of T a token: eight experts' rows of 8191 tokens and 2560 features (713 MB) take 105 us,
// 6.8 TB/s. (16-bit integers with an exponent for sixteen features took 72 and the product before it 164 instead of 195, but cost
// the neighbours of a large feature their digits: with one of 1000 times their size 1.4% of theirs.)
constexpr int kCombineWarps = 4;

// sums += weight * (the products with down of a pair's inner values beyond fp16), eight features from c on to a lane. Bound: latency, one
// row of down after the other: of 8191 tokens at eight of 64 experts of 2560 x 640 (0.75 ms) eight whose values are beyond fp16 by half
// take 1.3 ms more, all 38. (Eight rows at once took 1.1 and 34, and registers from the sum that every call makes.)
__device__ __noinline__ void add_excess(const hc_expert_mlp_t& p, const Excess& x, int64_t pair, int expert, float weight, int c,
                                        float* sums) {
  const __half* down = static_cast<const __half*>(p.down) + expert * p.down_expert_stride + c * p.down_out_stride;
  float v[8] = {};
  for (int word = 0; word < x.words; ++word) {
    for (uint32_t blocks = x.over[pair * x.words + word]; blocks != 0; blocks &= blocks - 1) {
      const int first = (word * 32 + __ffs(blocks) - 1) * 32, i = first + (threadIdx.x & 31);
      const float mine = i < p.inner ? x.values[pair * x.step + i] : 0.0f;
      for (uint32_t left = __ballot_sync(0xffffffffu, mine != 0.0f); left != 0; left &= left - 1) {
        const int l = __ffs(left) - 1;
        const float h = __shfl_sync(0xffffffffu, mine, l);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < p.hidden) v[j] = fmaf(h, __half2float(down[(first + l) * p.down_in_stride + j * p.down_out_stride]), v[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[j] = fmaf(weight, v[j], sums[j]);
}

// excess: of fp16 on the tensor cores, without values otherwise. gave_up: of the tensor cores' products, whether a wait has given
// up (then all results become NaN), NULL otherwise.
template <typename T, bool kPlanes>
__global__ void __launch_bounds__(32 * kCombineWarps, 5)
combine_kernel(const __grid_constant__ hc_expert_mlp_t p, const float* __restrict__ o, int64_t o_step,
               const uint8_t* __restrict__ counts, int64_t count_step, const __grid_constant__ Excess excess,
               const unsigned int* gave_up, bool vec) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, blocks = (p.hidden + 255) / 256;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kCombineWarps + (threadIdx.x >> 5), t = unit / blocks;
  if (t >= p.tokens) return;
  const int c = static_cast<int>(unit - t * blocks) * 256 + lane * 8;
  // lane j has the j-th expert's number, weight and planes; those that take part are in `valid`
  const int64_t first = t * p.top_k;
  const int id = lane < p.top_k ? p.experts[first + lane] : -1;
  const float weight = lane < p.top_k ? p.weights[first + lane] : 0.0f;
  const int planes = kPlanes && lane < p.top_k ? counts[(first + lane) * count_step + (c - lane * 8) / 256] : 1;
  const unsigned valid = __ballot_sync(0xffffffffu, id >= 0 && id < p.num_experts);
  const int count = __popc(valid);
  T* out = static_cast<T*>(p.out) + t * p.out_stride;
  Two sums[4] = {Two(0.0f), Two(0.0f), Two(0.0f), Two(0.0f)};
  const bool have = c < p.hidden, lost = gave_up != nullptr && *gave_up != 0;
  constexpr int kAhead = kPlanes ? 4 : 8;
  const int64_t plane = p.tokens * p.top_k * o_step;
  unsigned left = valid;
  for (int j0 = 0; j0 < count; j0 += kAhead) {
    float4 q[kAhead][2], other[kPlanes ? kAhead : 1][2];  // other: the second plane, zeros without one
    int parts[kAhead], from[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      from[j] = max(__ffs(left) - 1, 0);
      left &= left - 1;
      const bool take = j0 + j < count && have;
      const float4* row = reinterpret_cast<const float4*>(o + (first + from[j]) * o_step + c);
      parts[j] = kPlanes ? __shfl_sync(0xffffffffu, planes, from[j]) : 1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q[j][i] = take ? row[i] : make_float4(0, 0, 0, 0);
        if constexpr (kPlanes) other[j][i] = take && parts[j] > 1 ? row[plane / 4 + i] : make_float4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (j0 + j < count) {
        const Two by(__shfl_sync(0xffffffffu, weight, from[j]));
        float4 f[2] = {q[j][0], q[j][1]};
        if constexpr (kPlanes) {
          const auto add = [&](const float4* g) {
#pragma unroll
            for (int i = 0; i < 2; ++i) f[i].x += g[i].x, f[i].y += g[i].y, f[i].z += g[i].z, f[i].w += g[i].w;
          };
          add(other[j]);
          for (int n = 2; n < parts[j] && have; ++n)  // (of a few tiles only)
            add(reinterpret_cast<const float4*>(o + n * plane + (first + from[j]) * o_step + c));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sums[2 * i] = fma2(by, Two(f[i].x, f[i].y), sums[2 * i]);
          sums[2 * i + 1] = fma2(by, Two(f[i].z, f[i].w), sums[2 * i + 1]);
        }
      }
    }
  }
  float sum[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = lost ? make_float2(NAN, NAN) : sums[i].get();
    sum[2 * i] = v.x, sum[2 * i + 1] = v.y;
  }
  if constexpr (std::is_same<T, __half>::value) {
    if (excess.values != nullptr) {
      uint32_t over = 0;
      for (int i = 0; i < excess.words && (valid >> lane & 1u); ++i) over |= excess.over[(first + lane) * excess.words + i];
      for (unsigned pairs = __ballot_sync(0xffffffffu, over != 0); pairs != 0; pairs &= pairs - 1) {
        const int j = __ffs(pairs) - 1;
        add_excess(p, excess, first + j, __shfl_sync(0xffffffffu, id, j), __shfl_sync(0xffffffffu, weight, j), c, sum);
      }
    }
  }
  if (have) {
    if (vec) {  // (out's rows are 16-byte aligned and hold whole vectors)
      if constexpr (sizeof(T) == 2) {
        st16(out + c, V8<T>::pack(sum));
      } else {
        reinterpret_cast<float4*>(out + c)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        reinterpret_cast<float4*>(out + c)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < p.hidden) stf(out + c + i, sum[i]);
    }
  }
}

// counts: NULL where o is one plane.
template <typename T>
cudaError_t launch_combine(const hc_expert_mlp_t& a, const float* o, int64_t o_step, const uint8_t* counts, int64_t count_step,
                           const Excess& excess, const unsigned int* gave_up, cudaStream_t s) {
  const bool vec = a.hidden % 8 == 0 && a.out_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
  const int64_t units = a.tokens * ((a.hidden + 255) / 256);
  const dim3 grid(static_cast<unsigned>((units + kCombineWarps - 1) / kCombineWarps)), block(32 * kCombineWarps);
  return counts != nullptr ? launch_pdl(combine_kernel<T, true>, grid, block, 0, s, 1, a, o, o_step, counts, count_step, excess, gave_up,
                                        vec)
                           : launch_pdl(combine_kernel<T, false>, grid, block, 0, s, 1, a, o, o_step, counts, count_step, excess, gave_up,
                                        vec);
}

// ---------------------------------------------------------------- layout --

struct Plan {
  int rows;  // pairs to a tile of the tensor cores' products, 32 or 256; 0: the general ones
  int64_t tickets;
  int planes;  // of o
  int64_t h_step, o_step, count_step;
  int64_t excess_step, excess_words;  // (fp16 on the tensor cores) of the excess of inner values, elements and words of bits to a pair
  size_t bounds, order, zeros, part, h, o, counts, excess, total;  // zeros: whether a wait gave up, tickets, and the words of bits
};

// Which products run, and where their buffers lie in the workspace. Tiles of 32 pairs with the weights as the first operand
// or of 256 with the pairs as the first, by the pairs that an expert has on average: with 8, 16, 24, 28, 32 and 40 of them, 64
// experts of 2560 x 640 (six to a token) took 111, 121, 131, 137, 164 and 194 us with 32 and 128, 133, 135, 136, 139 and 143 with
// 256; 128 of 1024 x 512 (eight to a token) 81, 84, 93, 99, 110 and 135, and 90, 92, 95, 96, 98 and 100; 16 of 1280 x 2560 (two)
// 63, 75, 70, 75, 84 and 87, and 65, 66, 66, 86, 86 and 86; 8 of 512 x 1024 (two) 20, 24, 25, 22, 22 and 22, and 23 throughout.
Plan make_plan(const hc_expert_mlp_t& a, bool aligned, int num_sms) {
  const size_t pairs = static_cast<size_t>(a.tokens) * a.top_k;
  Plan l = {};
  // (TMA steps from row to row and from expert to expert, so strides of 0 are not for it)
  const bool steps = (a.num_experts == 1 || (a.up_expert_stride > 0 && a.down_expert_stride > 0)) && a.up_in_stride > 0 &&
                     a.up_out_stride > 0 && a.down_in_stride > 0 && a.down_out_stride > 0 && (a.tokens == 1 || a.x_stride >= a.hidden);
  if (a.dtype != HC_F32 && aligned && steps && !(a.flags & HC_FLAG_FORCE_GENERAL)) {
    const size_t mean = pairs / a.num_experts;
    l.rows = mean <= 24 ? 32 : 256;
  }
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes, 256);
    return here;
  };
  l.bounds = take((a.num_experts + 1) * sizeof(int32_t));
  l.order = take(pairs * sizeof(int32_t));
  l.h_step = l.rows ? static_cast<int64_t>(align_up(a.inner, 16)) : a.inner;
  l.o_step = static_cast<int64_t>(align_up(a.hidden, 16));
  const bool few = l.rows == 32;
  if (few) l.tickets = experts_um_tiles(a, l.rows, true);
  if (l.rows && a.dtype == HC_F16) {
    l.excess_step = static_cast<int64_t>(align_up(a.inner, 128));
    l.excess_words = (a.inner + 1023) / 1024;
  }
  l.zeros = take((1 + l.tickets + pairs * l.excess_words) * sizeof(uint32_t));
  if (few) {
    l.part = take(static_cast<size_t>(num_sms) * 2 * 2 * l.rows * 128 * sizeof(float));
  }
  l.h = take(pairs * l.h_step * (l.rows ? 2 : 4));
  // A plane of o for each piece that a tile of the outer product can be cut into: two where runs are cut, and four where so
  // few tiles are possible that each can be on three SMs or more.
  l.planes = few ? ((pairs + l.rows - 1) / l.rows * ((a.hidden + 255) / 256) * 3 <= static_cast<size_t>(num_sms) ? 4 : 2) : 1;
  l.o = take(pairs * l.o_step * 4 * l.planes);
  if (few) {
    l.count_step = (a.hidden + 255) / 256;
    l.counts = take(pairs * l.count_step);
  }
  l.excess = take(pairs * l.excess_step * sizeof(float));
  l.total = at;
  return l;
}

template <typename T> cudaError_t launch(const hc_expert_mlp_t& a, bool aligned, int num_sms, cudaStream_t s) {
  const Plan l = make_plan(a, aligned, num_sms);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  const ExpertLists lists = {reinterpret_cast<int32_t*>(ws + l.bounds), reinterpret_cast<int32_t*>(ws + l.order)};
  unsigned int *zeros = reinterpret_cast<unsigned int*>(ws + l.zeros), *tickets = zeros + 1;
  float* o = reinterpret_cast<float*>(ws + l.o);
  const int pairs = static_cast<int>(a.tokens * a.top_k);
  const int64_t count = 1 + l.tickets + pairs * l.excess_words;
  cudaError_t e = pairs > 4096 ? launch_pdl(lists_kernel<1024>, dim3(a.num_experts), dim3(1024), 0, s, 1, a.experts, pairs,
                                            a.num_experts, lists, zeros, count)
                               : launch_pdl(lists_kernel<128>, dim3(a.num_experts), dim3(128), 0, s, 1, a.experts, pairs,
                                            a.num_experts, lists, zeros, count);
  if (e != cudaSuccess) return e;
  if constexpr (sizeof(T) == 2) {
    if (l.rows) {
      uint8_t* counts = l.rows == 32 ? ws + l.counts : nullptr;
      const Excess excess = {l.excess_words ? reinterpret_cast<float*>(ws + l.excess) : nullptr, tickets + l.tickets, l.excess_step,
                             static_cast<int>(l.excess_words)};
      const ExpertUm u = {lists, ws + l.h, o, counts, l.h_step, l.o_step, l.count_step, reinterpret_cast<float*>(ws + l.part), tickets,
                          excess, zeros, static_cast<int64_t>(pairs) * l.o_step, l.planes, l.rows};
      e = l.rows == 256 ? launch_experts_many(a, u, num_sms, s) : launch_experts_few(a, u, num_sms, s);
      return e != cudaSuccess ? e : launch_combine<T>(a, o, l.o_step, counts, l.count_step, excess, zeros, s);
    }
  }
  const GeneralArgs g = {a, lists, reinterpret_cast<float*>(ws + l.h), o, l.o_step};
  e = launch_general<T, true>(g, num_sms, s);
  if (e != cudaSuccess) return e;
  e = launch_general<T, false>(g, num_sms, s);
  return e != cudaSuccess ? e : launch_combine<T>(a, o, l.o_step, nullptr, 0, Excess{}, nullptr, s);
}

}  // namespace

size_t expert_mlp_workspace(const hc_expert_mlp_t& a, bool aligned, int num_sms) {
  return make_plan(a, aligned, num_sms).total;
}

cudaError_t launch_expert_mlp(const hc_expert_mlp_t& a, bool aligned, int num_sms, cudaStream_t s) {
  if (a.dtype == HC_F32) return launch<float>(a, aligned, num_sms, s);
  if (a.dtype == HC_F16) return launch<__half>(a, aligned, num_sms, s);
  return launch<__nv_bfloat16>(a, aligned, num_sms, s);
}

}  // namespace hc
