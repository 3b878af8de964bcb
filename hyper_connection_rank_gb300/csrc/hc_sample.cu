// The choice of the next tokens (hc_token_sample).
//
// Three kernels. Two are for what most calls ask, and leave what they cannot decide to the third, which decides every row:
//
//   pick_kernel    rows that filter, where a few hundred tokens at most stay
//   stream_kernel  calls that filter nothing, from 2^21 logits on
//   sample_kernel  any row: all of a small call that filters nothing, otherwise what the others have left undecided
//
// In the third a cluster of CTAs takes a row and reads it once: each CTA keeps its slice of the row in shared memory, where
// every later pass finds it. The steps are
//
//   1. the largest logit m and its first index;
//   2. with top_k, the k-th token in the order (logit falling, index rising);
//   3. with top_p, the last token of that order that stays;
//   4. the sum of the weights that stay, per warp, CTA and row;
//   5. the token: the CTA, the warp, the lane and at last the element in which the cumulated weight passes uniform * sum.
//
// Steps 2 and 3 find the first element of the order at which a cumulated value (1 each, or the weights) reaches a target: a
// histogram over 2048 equal steps of the exponent, merged over the cluster, then histograms over the logits' bits within the
// step that the target falls into, until one value is left; among elements of that value the index decides. But if no more
// than 2048 elements reach that step, they are listed and sorted by one CTA, which then finishes the row by itself; and if no
// more than that are in the step, they are, and it tells the others where the target falls.
//
// Weights are integers, 2^43 for the largest logit: integer sums have one result in any order, whatever threads, warps and
// CTAs make of it, and a row of 409600 weights stays below 2^62. A weight is 2^-y with y = (m - x) log2(e) / t formed in two
// fp32 parts; y = (64 n + i + f) / 64, and 2^-y = 2^-n T[i] (1 + q), where T is a table and q = 2^(-f/64) - 1 a polynomial in
// fp32 whose leading term is kept apart, so that the whole is good to 2^-38 of itself (fp32's 2^-24 would choose another
// token than the definition once in some thousand rows of 10^5 tokens; fp64 runs at 1/64 of the rate here).
//
// Bound: the third kernel's passes over its slices (four with a border, 50 instructions to a logit in those that weigh), the
// histogram's atomics and its CTAs' steps together. With pick_kernel's attempt before it, one row of 131072 fp32 logits takes
// 35 us with a top_k of 20000 and 37 with a top_p that leaves thousands (56 where all logits are within few steps), 64 rows
// take 102 and 128 (166). With 512 threads to a CTA they took a tenth to a fifth longer.
#include <algorithm>
#include <atomic>

#include "hc_async.cuh"
#include "hc_common.cuh"
#include "hc_experts_internal.h"
#include "hc_two.cuh"

namespace hc {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;
// CTAs to a row at most, and to one of no more rows than the device can have clusters of so many together (one to six of
// 131072 fp32 logits with a top_p that leaves thousands take 44 to 45 us with 8 and 36 to 38 with 16, with one that leaves few
// 18 to 19 with either, a top_k of 20000 of 262144 53 to 55 and 42 to 45).
constexpr int kCluster = 8, kMaxCluster = 16;
constexpr int kMaxSlice = kSampleMaxVocab / kCluster;  // elements that a CTA keeps
constexpr int kOneBits = 43;
constexpr u64 kOne = 1ull << kOneBits;
constexpr float kRange = 44.0f;  // weights below 2^-44 count as 0

// 2^(43 - i / 64), rounded.
__device__ const u64 kExp2[64] = {
    8796093022208ull, 8701341624228ull, 8607610887057ull, 8514889816151ull, 8423167535396ull, 8332433285840ull,
    8242676424423ull, 8153886422733ull, 8066052865769ull, 7979165450722ull, 7893213985764ull, 7808188388852ull,
    7724078686549ull, 7640875012848ull, 7558567608024ull, 7477146817477ull, 7396603090613ull, 7316926979711ull,
    7238109138825ull, 7160140322681ull, 7083011385596ull, 7006713280404ull, 6931237057393ull, 6856573863262ull,
    6782714940072ull, 6709651624229ull, 6637375345460ull, 6565877625812ull, 6495150078656ull, 6425184407706ull,
    6355972406040ull, 6287505955143ull, 6219777023951ull, 6152777667913ull, 6086500028053ull, 6020936330056ull,
    5956078883349ull, 5891920080202ull, 5828452394836ull, 5765668382539ull, 5703560678795ull, 5642121998415ull,
    5581345134690ull, 5521222958540ull, 5461748417677ull, 5402914535784ull, 5344714411690ull, 5287141218566ull,
    5230188203118ull, 5173848684801ull, 5118116055032ull, 5062983776415ull, 5008445381977ull, 4954494474403ull,
    4901124725294ull, 4848329874419ull, 4796103728980ull, 4744440162891ull, 4693333116055ull, 4642776593652ull,
    4592764665442ull, 4543291465063ull, 4494351189345ull, 4445938097632ull,
};

struct SampleArgs {
  const void* logits;
  const float* uniform;
  const float *temperatures, *top_ps, *min_ps;
  const int32_t* top_ks;
  int32_t* tokens;
  float* logprobs;
  int64_t stride;
  int64_t rows;
  int vocab, slice, top_k, dtype;
  float temperature, top_p, min_p;
  bool undecided;  // only rows whose token is kUndecided
};
constexpr int kUndecided = -2;  // stands in tokens until a row's second kernel has run

// What a row's parameters come to.
struct Params {
  u64 least;        // units of the least weight that min_p leaves
  float t, p, u;
  float ch, cl;     // log2(e) / t in two parts
  int k, step;      // step: of the histogram, past which min_p leaves nothing
};

struct Shared {
  u64 table[64];
  Params params;
  u64 exchange[2][kMaxCluster];
  u64 red[kWarps];
  u64 border[4];  // where a target falls: bin, value before it, value in it
  union {
    struct {
      uint32_t lo[kBins], hi[kBins];
    };
    u64 list[kBins];  // of candidates, (key falling, index rising) as rising integers
  };
  uint32_t listed;
};
constexpr int kCandidates = kBins;
// The candidates of all CTAs come to lie where the first one's slice was.
constexpr int kMinSlice = kCandidates * sizeof(u64) / sizeof(float);

__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // (-0 becomes 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ void st_cluster(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// A barrier of a row's CTAs. Its instructions are the whole warp's, whose lanes part before it where they store for themselves.
__device__ __forceinline__ void row_sync() {
  __syncwarp();
  cluster_sync_all();
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Sum over the lanes up to and with this one.
__device__ __forceinline__ u64 warp_scan_u64(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// floor(f * v) for f in 0 .. 1, exactly.
__device__ __forceinline__ u64 part_of(float f, u64 v) {
  if (!(f > 0.0f)) return 0;
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;  // f = m 2^(max(e, 1) - 150)
  const int down = 150 - static_cast<int>(e ? e : 1);                  // at least 23
  const u64 lo = m * v, hi = __umul64hi(m, v);
  if (down < 64) return hi << (64 - down) | lo >> down;
  return down < 128 ? hi >> (down - 64) : 0;
}
// The least integer that is not below f * v, at least 1.
__device__ __forceinline__ u64 reach(float f, u64 v) {
  const u64 n = part_of(f, v);
  if (n == 0) return 1;
  // (whether the product is an integer: compare n / f the other way round, in whole numbers)
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
  const int down = 150 - static_cast<int>(e ? e : 1);
  const u64 lo = m * v, hi = __umul64hi(m, v);
  const bool whole = down < 64 ? (lo & ((1ull << down) - 1)) == 0 : lo == 0 && (hi & ((1ull << (down - 64)) - 1)) == 0;
  return n + (whole ? 0 : 1);
}

// log(w / total) by what the others have, so that a token with nearly all of the sum keeps its digits; or, of a weight of
// few units (below kPlainLog), from the logarithm of it (log2_w).
constexpr u64 kPlainLog = 1ull << 26;
__device__ __forceinline__ float log_share(u64 w, double log2_w, u64 total) {
  if (w >= total / 2) return -log1pf(static_cast<float>(total - w) / static_cast<float>(w));
  if (w >= kPlainLog) return logf(static_cast<float>(w) / static_cast<float>(total));
  const int e = 63 - __clzll(total);
  const float rest = log2f(static_cast<float>(total) * __uint_as_float((127u - e) << 23));  // total = 2^(e + rest)
  return 0.69314718f * (static_cast<float>(log2_w - e) - rest);
}

// The weights of a row.
struct Scale {
  const u64* table;  // in shared memory
  float m, ch, cl;   // largest logit; log2(e) / temperature in two parts

  // The step of the first histogram, never falling as x falls.
  __device__ __forceinline__ int step(float x) const {
    return x == m ? 0 : min(kBins - 1, static_cast<int>((m - x) * ch * (kBins / kRange)));
  }

  __device__ __forceinline__ u64 weight(float x) const {
    if (x == m) return kOne;
    const float d = __fsub_rn(m, x), b = __fsub_rn(d, m);
    const float dl = __fsub_rn(__fsub_rn(m, __fsub_rn(d, b)), __fadd_rn(x, b));
    const float y = __fmul_rn(d, ch);
    if (!(y < kRange)) return 0;
    const float yl = fmaf(d, ch, -y) + fmaf(d, cl, dl * ch);
    const int j = __float2int_rn(y * 64.0f);
    const float f = fmaf(static_cast<float>(j), -0.015625f, y);  // exact, at most 1/128
    const float kLn2 = 0.69314718f, kLn2Tail = -1.9046542e-09f;
    const float h = __fmul_rn(f, kLn2);
    const float l = fmaf(f, kLn2, -h) + fmaf(f, kLn2Tail, yl * kLn2);
    // e^-(h + l) - 1 = -h + (h^2 / 2 - h^3 / 6 + h^4 / 24 - l (1 - h))
    const float c = fmaf(__fmul_rn(h, h), fmaf(h, fmaf(h, 0.041666668f, -0.16666667f), 0.5f), fmaf(h, l, -l));
    const int q = __float2int_rn(h * -274877906944.0f) + __float2int_rn(c * 274877906944.0f);  // in units of 2^-38
    const u64 t = table[j & 63];
    const long long w =
        static_cast<long long>(t) + ((static_cast<long long>(static_cast<int>(t >> 13)) * q) >> 25);
    return static_cast<u64>(w) >> (j >> 6);
  }

  // The logarithm of the weight of a token of row r.
  __device__ __forceinline__ double log2_units(const SampleArgs& a, int64_t r, int token) const {
    const int64_t at = r * a.stride + token;
    const float x = a.dtype == HC_F32   ? static_cast<const float*>(a.logits)[at]
                    : a.dtype == HC_F16 ? __half2float(static_cast<const __half*>(a.logits)[at])
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]);
    if (x == m) return kOneBits;
    return kOneBits + (static_cast<double>(x) - static_cast<double>(m)) * (static_cast<double>(ch) + static_cast<double>(cl));
  }
};

// Sort `n` (a power of two) integers in shared memory.
__device__ __forceinline__ void sort(u64* v, int n) {
  for (int size = 2; size <= n; size *= 2) {
    for (int apart = size / 2; apart > 0; apart /= 2) {
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int i = 2 * t - (t & (apart - 1)), j = i + apart;
        const bool up = (i & size) == 0;
        const u64 x = v[i], y = v[j];
        if ((x > y) == up) {
          v[i] = y;
          v[j] = x;
        }
      }
      __syncthreads();
    }
  }
}

// The sum of the values of all threads before this one, and (in *all) of all of them.
__device__ __forceinline__ u64 block_scan_u64(Shared& sh, u64 v, u64* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 upto = warp_scan_u64(v);
  __syncthreads();
  if (lane == 31) sh.red[warp] = upto;
  __syncthreads();
  u64 before = upto - v, sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.red[w];
    sum += sh.red[w];
  }
  *all = sum;
  return before;
}

// One row, as a thread of the exact kernel sees it.
struct Row : Scale {
  Shared& sh;
  const float* xs;       // this CTA's slice
  int n, base;           // its elements, and the first one's index in the row
  int rank, ctas, turn;  // turn: of the exchanges
  uint32_t cut_key, cut_index;  // what stays: keys above, and equal ones up to this index

  __device__ __forceinline__ Row(Shared& shared, const float* slice, int count, int first, int cta, int of, int at)
      : Scale{shared.table, 0.0f, 0.0f, 0.0f}, sh(shared), xs(slice), n(count), base(first), rank(cta), ctas(of), turn(at),
        cut_key(0u), cut_index(0xffffffffu) {}

  // Every CTA's value, in the order of the ranks, in exchange[turn].
  __device__ __forceinline__ const u64* gather(u64 v) {
    turn ^= 1;
    if (threadIdx.x < ctas) st_cluster(mapa_shared(smem_addr(&sh.exchange[turn][rank]), threadIdx.x), v);
    row_sync();
    return sh.exchange[turn];
  }
  // The same value for all threads of the CTA: the largest one.
  __device__ __forceinline__ u64 block_max_u64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t = max(t, sh.red[w]);
    return t;
  }
  __device__ __forceinline__ u64 cluster_max(u64 v) {
    const u64* all = gather(block_max_u64(v));
    u64 t = 0;
    for (int r = 0; r < ctas; ++r) t = max(t, all[r]);
    return t;
  }

  __device__ __forceinline__ bool stays(float x, int index) const {
    const uint32_t k = key_of(x);
    return k > cut_key || (k == cut_key && static_cast<uint32_t>(index) <= cut_index);
  }

  // Values (not zeros) into the histogram, all lower halves before any upper one.
  static constexpr int kAtOnce = 4;
  __device__ __forceinline__ void add(const int* bin, const u64* v) {
    uint32_t old[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) old[j] = v[j] != 0 ? atomicAdd(&sh.lo[bin[j]], static_cast<uint32_t>(v[j])) : 0u;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const uint32_t lo = static_cast<uint32_t>(v[j]), up = static_cast<uint32_t>(v[j] >> 32) + (old[j] + lo < old[j] ? 1u : 0u);
      if (up != 0) atomicAdd(&sh.hi[bin[j]], up);
    }
  }

  // The histograms of all CTAs together: into which bin the target falls (border[0]), what lies before it (border[1]) and
  // in it (border[2]). target(total) gives the target. The histogram is empty again afterwards.
  template <class F> __device__ __forceinline__ void find(F target) {
    row_sync();
    const int mine = kBins / ctas, per = max(1, mine / kThreads), at = threadIdx.x * per;
    u64 v[kBins / kThreads], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      v[i] = 0;
      if (i < per && at + i < mine) {
        const int bin = rank * mine + at + i;
        uint32_t lo[kMaxCluster], hi[kMaxCluster];  // (all loads before any use)
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          lo[r] = r < ctas ? ld_cluster(mapa_shared(smem_addr(&sh.lo[bin]), r)) : 0u;
          hi[r] = r < ctas ? ld_cluster(mapa_shared(smem_addr(&sh.hi[bin]), r)) : 0u;
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) v[i] += lo[r] + (static_cast<u64>(hi[r]) << 32);
      }
      sum += v[i];
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const u64 upto = warp_scan_u64(sum);
    __syncthreads();
    if (lane == 31) sh.red[warp] = upto;
    __syncthreads();
    u64 before = upto - sum, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.red[w];
      all += sh.red[w];
    }
    const u64* totals = gather(all);
    u64 total = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r < rank) before += totals[r];
      total += totals[r];
    }
    const u64 want = target(total);
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      if (before < want && want <= before + v[i]) {
        for (int r = 0; r < ctas; ++r) {
          const uint32_t to = mapa_shared(smem_addr(sh.border), r);
          st_cluster(to, rank * mine + at + i);
          st_cluster(to + 8, before);
          st_cluster(to + 16, v[i]);
        }
      }
      before += v[i];
    }
    row_sync();
  }

  // Lists the elements of steps 0 .. bin where the first CTA's slice was, or (`only`) those of step bin that stay in place of
  // its histogram, and returns their number; or -1 if they are too many (then the histogram is empty again).
  __device__ __forceinline__ int list(int bin, bool only) {
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float x = xs[i];
      const int at_step = step(x);
      if (at_step > bin || (only && (at_step < bin || !stays(x, base + i)))) continue;
      const uint32_t at = atomicAdd(&sh.listed, 1u);
      if (at < kCandidates) sh.list[at] = static_cast<u64>(~key_of(x)) << 32 | static_cast<uint32_t>(base + i);
    }
    __syncthreads();
    const uint32_t have = sh.listed;
    const u64* counts = gather(have);
    u64 before = 0, all = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r < rank) before += counts[r];
      all += counts[r];
    }
    if (all > kCandidates) {
      for (int i = threadIdx.x; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
      return -1;
    }
    // (the first CTA's own are the first)
    const uint32_t to = mapa_shared(only ? smem_addr(sh.list) : smem_addr(xs), 0) + static_cast<uint32_t>(before) * 8;
    if (!only || rank > 0)
      for (uint32_t i = threadIdx.x; i < have; i += kThreads) st_cluster(to + 8 * i, sh.list[i]);
    row_sync();
    return static_cast<int>(all);
  }

  // The last one that stays is the first of the listed ones of a step at which their cumulated values reach `want`.
  __device__ __forceinline__ void cut_listed(int count, bool mass, u64 want) {
    constexpr int kEach = kCandidates / kThreads;
    if (rank == 0 && count <= kThreads) {  // each with all others
      u64* values = sh.list + kThreads;
      const bool have = threadIdx.x < count;
      const u64 me = have ? sh.list[threadIdx.x] : 0, v = !have ? 0 : mass ? weight(value_of(~static_cast<uint32_t>(me >> 32))) : 1;
      if (have) values[threadIdx.x] = v;
      __syncthreads();
      u64 before = 0;
      if (have) {
#pragma unroll 4
        for (int j = 0; j < count; ++j)
          if (sh.list[j] < me) before += values[j];
        if (before < want && want <= before + v)
          for (int r = 0; r < ctas; ++r) st_cluster(mapa_shared(smem_addr(&sh.border[3]), r), me);
      }
    } else if (rank == 0) {
      int size = 2;
      while (size < count) size *= 2;
      for (int i = count + threadIdx.x; i < size; i += kThreads) sh.list[i] = ~0ull;
      __syncthreads();
      sort(sh.list, size);
      u64 v[kEach], sum = 0, all;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = threadIdx.x * kEach + j;
        v[j] = i >= count ? 0 : mass ? weight(value_of(~static_cast<uint32_t>(sh.list[i] >> 32))) : 1;
        sum += v[j];
      }
      u64 before = block_scan_u64(sh, sum, &all);
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (before < want && want <= before + v[j])
          for (int r = 0; r < ctas; ++r) st_cluster(mapa_shared(smem_addr(&sh.border[3]), r), sh.list[threadIdx.x * kEach + j]);
        before += v[j];
      }
    }
    row_sync();
    cut_key = ~static_cast<uint32_t>(sh.border[3] >> 32);
    cut_index = static_cast<uint32_t>(sh.border[3]);
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
    __syncthreads();
  }

  // The first element, in the order of falling logits and rising indexes, at which the values cumulated over what stays
  // reach a target becomes the last one that stays. With `mass` the values are the weights and the target is p times
  // their sum, otherwise they are 1 and the target is k. If the elements down to the target's step are few, they are listed
  // instead (see list()) and their number is returned; *total is the sum of the values. Otherwise -1.
  __device__ __forceinline__ int cut(bool mass, float p, u64 k, u64* total) {
    u64 want = 0;
    for (int i0 = threadIdx.x; i0 < n; i0 += kAtOnce * kThreads) {
      u64 v[kAtOnce];
      int bin[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * kThreads;
        const float x = i < n ? xs[i] : -INFINITY;
        v[j] = i < n && stays(x, base + i) ? (mass ? weight(x) : 1) : 0;
        bin[j] = step(x);
      }
      add(bin, v);
    }
    find([&](u64 all) {
      *total = all;
      want = min(mass ? reach(p, all) : k, all);
      return want;
    });
    const int bin = static_cast<int>(sh.border[0]);
    if (cut_key == 0 && !mass && sh.border[1] + sh.border[2] <= kCandidates) {
      const int listed = list(bin, false);
      if (listed >= 0) return listed;
      __syncthreads();
    }
    want -= sh.border[1];
    if (mass || sh.border[2] <= kCandidates) {
      const int listed = list(bin, true);
      if (listed >= 0) {
        cut_listed(listed, mass, want);
        return -1;
      }
      __syncthreads();
    }
    // the keys of that step
    uint32_t low = 0xffffffffu, high = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float x = xs[i];
      if (step(x) != bin || !stays(x, base + i)) continue;
      const uint32_t key = key_of(x);
      low = min(low, key);
      high = max(high, key);
    }
    high = static_cast<uint32_t>(cluster_max(high));
    low = 0xffffffffu - static_cast<uint32_t>(cluster_max(0xffffffffu - low));
    u64 in = sh.border[2];
    for (int level = 0; level < 3 && low < high; ++level) {  // (32 bits, then 21, then 10)
      const int shift = max(0, 21 - __clz(high - low));
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float x = xs[i];
        const uint32_t key = key_of(x);
        if (key < low || key > high || !stays(x, base + i)) continue;
        u64 v[kAtOnce] = {mass ? weight(x) : 1};
        const int bin[kAtOnce] = {static_cast<int>((high - key) >> shift)};
        add(bin, v);
      }
      find([&](u64) { return want; });
      const uint32_t j = static_cast<uint32_t>(sh.border[0]);
      want -= sh.border[1];
      in = sh.border[2];
      const uint32_t top = high - (j << shift);
      low = max(low, top - ((1u << shift) - 1));
      high = top;
    }
    const u64 each = mass ? weight(value_of(high)) : 1;
    const u64 take = (want + each - 1) / each, have = in / each;
    uint32_t last = cut_key == high ? cut_index : 0xffffffffu;
    if (take < have) last = nth(high, take);
    cut_key = high;
    cut_index = last;
    return -1;
  }

  // The index of the take-th element with this key.
  __device__ __forceinline__ uint32_t nth(uint32_t key, u64 take) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunk = (n + kWarps - 1) / kWarps, lo = min(n, warp * chunk), hi = min(n, lo + chunk);
    u64 mine = 0;
    for (int i = lo + lane; i < hi; i += 32) mine += key_of(xs[i]) == key;
    mine = warp_sum_u64(mine);
    __syncthreads();
    if (lane == 0) sh.red[warp] = mine;
    __syncthreads();
    u64 before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.red[w];
      all += sh.red[w];
    }
    const u64* totals = gather(all);
    for (int r = 0; r < rank; ++r) before += totals[r];
    u64 found = 0;
    if (before < take && take <= before + mine) {
      for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t hit = __ballot_sync(0xffffffffu, i < hi && key_of(xs[min(i, hi - 1)]) == key);
        const int c = __popc(hit);
        if (before < take && take <= before + c) found = base + i0 + __fns(hit, 0, static_cast<int>(take - before));
        before += c;
      }
    }
    return static_cast<uint32_t>(cluster_max(found));
  }
};

template <typename T> __device__ __forceinline__ float logit(T v) {
  const float x = Ty<T>::to_f(v);
  return x != x ? -INFINITY : x;
}

// A slice of a row into shared memory, and the largest key with the first index that has it.
template <typename T>
__device__ __forceinline__ u64 load_slice(const T* row, int base, int n, float* xs) {
  constexpr int kVec = 16 / sizeof(T);
  u64 best = 0;
  const auto put = [&](int i, T v) {
    const float x = logit(v);
    xs[i] = x;
    best = max(best, static_cast<u64>(key_of(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(base + i)));
  };
  const T* p = row + base;
  const int skip = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / sizeof(T)));
  const int vecs = (n - skip) / kVec;
  if (threadIdx.x < skip) put(threadIdx.x, p[threadIdx.x]);
  const uint4* q = reinterpret_cast<const uint4*>(p + skip);
#pragma unroll 4
  for (int i = threadIdx.x; i < vecs; i += kThreads) {
    const uint4 u = __ldg(q + i);
    const T* v = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < kVec; ++j) put(skip + i * kVec + j, v[j]);
  }
  const int tail = skip + vecs * kVec;
  if (threadIdx.x < n - tail) put(tail + threadIdx.x, p[tail + threadIdx.x]);
  return best;
}

// The rest of a row whose candidates the first CTA has listed, `count` of them: sorted, the first k stay (k > 0), of those
// the ones before which less than p of the sum lies (p < 1; the sum is `total` without a k), of those the ones not below
// `least`; sorted by index, the token.
__device__ __forceinline__ void finish_list(const SampleArgs& a, const Row& row, u64* list, int count, u64 k, float p, u64 total,
                                            u64 least, float u, int64_t r) {
  constexpr int kEach = kCandidates / kThreads;
  Shared& sh = row.sh;
  int size = 2;
  while (size < count) size *= 2;
  for (int i = count + threadIdx.x; i < size; i += kThreads) list[i] = ~0ull;
  __syncthreads();
  sort(list, size);
  u64 w[kEach], sum = 0, all;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = threadIdx.x * kEach + j;
    w[j] = i < count && (k == 0 || i < k) ? row.weight(value_of(~static_cast<uint32_t>(list[i] >> 32))) : 0;
    sum += w[j];
  }
  u64 before = block_scan_u64(sh, sum, &all);
  const u64 goal = p < 1.0f ? reach(p, k > 0 ? all : total) : ~0ull;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = threadIdx.x * kEach + j;
    const bool stays = before < goal && w[j] >= least;
    before += w[j];
    if (i < size) {
      // the index, and where the weight is
      if (!stays) w[j] = 0;
      sh.list[i] = w[j];
      list[i] = stays ? list[i] << 32 | static_cast<uint32_t>(i) : ~0ull;
    }
  }
  __syncthreads();
  sort(list, size);
  sum = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int i = threadIdx.x * kEach + j;
    w[j] = i < size && list[i] != ~0ull ? sh.list[static_cast<uint32_t>(list[i])] : 0;
    sum += w[j];
  }
  before = block_scan_u64(sh, sum, &all);
  const u64 want = min(all, part_of(u, all) + 1);
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (before < want && want <= before + w[j]) {
      a.tokens[r] = static_cast<int>(list[threadIdx.x * kEach + j] >> 32);
      if (a.logprobs)
        a.logprobs[r] = log_share(w[j], w[j] < kPlainLog ? row.log2_units(a, r, static_cast<int>(list[threadIdx.x * kEach + j] >> 32)) : 0.0, all);
    }
    before += w[j];
  }
}

__device__ __forceinline__ void row_params(const SampleArgs& a, int64_t r, Params* to) {
  Params v;
  v.t = a.temperatures ? a.temperatures[r] : a.temperature;
  v.p = a.top_ps ? a.top_ps[r] : a.top_p;
  v.k = a.top_ks ? a.top_ks[r] : a.top_k;
  const float u = a.uniform[r], min_p = a.min_ps ? a.min_ps[r] : a.min_p;
  v.u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;
  const float kLog2e = 1.44269502f, kLog2eTail = 1.9259630e-08f;
  v.ch = __fdiv_rn(kLog2e, v.t);
  v.cl = __fdiv_rn(fmaf(-v.ch, v.t, kLog2e) + kLog2eTail, v.t);  // (the remainder of the quotient is exact)
  if (!(fabsf(v.ch) < 1e30f) || !(fabsf(v.cl) < 1e30f)) v.cl = 0.0f;
  v.least = 1;
  v.step = kBins;
  if (min_p > 0.0f) {
    v.least = max(__float2ull_ru(fminf(min_p, 1.0f) * static_cast<float>(kOne)), 1ull);  // (the product is exact)
    v.step = min(kBins, static_cast<int>((0.01f - log2f(fminf(min_p, 1.0f))) * (kBins / kRange)) + 1);
  }
  *to = v;
}

__device__ __forceinline__ void sample_row(const SampleArgs& a, Shared& sh, float* xs, int64_t r, int rank, int ctas, int* turn) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int base = rank * a.slice, n = max(0, min(a.slice, a.vocab - base));
  if (tid == kThreads - 1) row_params(a, r, &sh.params);
  u64 best;
  if (a.dtype == HC_F32)
    best = load_slice(static_cast<const float*>(a.logits) + r * a.stride, base, n, xs);
  else if (a.dtype == HC_F16)
    best = load_slice(static_cast<const __half*>(a.logits) + r * a.stride, base, n, xs);
  else
    best = load_slice(static_cast<const __nv_bfloat16*>(a.logits) + r * a.stride, base, n, xs);
  // (every CTA of the cluster has begun, its histogram is empty and its parameters are there, before anything is stored into
  // its shared memory)
  row_sync();
  const float t = sh.params.t, p = sh.params.p, u = sh.params.u;
  const int k = sh.params.k;
  const u64 least = sh.params.least;
  Row row(sh, xs, n, base, rank, ctas, *turn);
  best = row.cluster_max(best);
  *turn = row.turn;
  row.m = value_of(static_cast<uint32_t>(best >> 32));
  const int first = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
  const bool none = row.m == -INFINITY;
  if (none || !(t > 0.0f) || k == 1 || p <= 0.0f) {
    if (rank == 0 && tid == 0) {
      a.tokens[r] = none ? -1 : first;
      if (a.logprobs) a.logprobs[r] = none ? -INFINITY : 0.0f;
    }
    return;  // (nothing is on its way to another CTA's memory)
  }
  row.ch = sh.params.ch;
  row.cl = sh.params.cl;
  const bool cut_k = k > 0 && k < a.vocab;
  u64 total = 0;
  int listed = -1;
  if (cut_k) listed = row.cut(false, 0.0f, static_cast<u64>(k), &total);
  if (listed < 0 && p < 1.0f) listed = row.cut(true, p, 0, &total);
  *turn = row.turn;
  if (listed >= 0) {
    if (rank == 0) finish_list(a, row, reinterpret_cast<u64*>(xs), listed, cut_k ? k : 0, p, total, least, u, r);
    __syncthreads();
    // the histogram for the next row
    for (int i = tid; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
    return;
  }
  const auto kept = [&](int i) -> u64 {
    const float x = xs[i];
    if (!row.stays(x, base + i)) return 0;
    const u64 w = row.weight(x);
    return w >= least ? w : 0;
  };

  // a warp's sum over a run of elements, which its lanes take in turn
  const int chunk = (n + kWarps - 1) / kWarps, lo = min(n, warp * chunk), hi = min(n, lo + chunk);
  u64 mine = 0;
#pragma unroll 4
  for (int i = lo + lane; i < hi; i += 32) mine += kept(i);
  mine = warp_sum_u64(mine);
  __syncthreads();
  if (lane == 0) sh.red[warp] = mine;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.red[w];
    all += sh.red[w];
  }
  const u64* totals = row.gather(all);
  *turn = row.turn;
  total = 0;
  for (int i = 0; i < ctas; ++i) {
    if (i < rank) before += totals[i];
    total += totals[i];
  }
  // the first element whose cumulated weight passes uniform * total, so is at least the next integer
  const u64 want = min(total, part_of(u, total) + 1);
  if (!(before < want && want <= before + mine)) return;
  // in one warp: 128 elements at a time, until they pass it, then the 32 of those that do
  for (int i0 = lo; i0 < hi; i0 += 32 * 4) {
    u64 w[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 32 * j + lane;
      w[j] = i < hi ? kept(i) : 0;
      sum += w[j];
    }
    // (sums below 2^45 a lane)
    sum = (static_cast<u64>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(sum >> 23))) << 23) +
          __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(sum) & 0x7fffffu);
    if (before + sum < want) {
      before += sum;
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u64 upto = before + warp_scan_u64(w[j]);
      const uint32_t hit = __ballot_sync(0xffffffffu, upto >= want);
      if (hit != 0) {
        const int i = i0 + 32 * j + lane;
        if (lane == __ffs(hit) - 1) {
          a.tokens[r] = base + i;
          if (a.logprobs) a.logprobs[r] = log_share(w[j], w[j] < kPlainLog ? row.log2_units(a, r, base + i) : 0.0, total);
        }
        return;
      }
      before = __shfl_sync(0xffffffffu, upto, 31);
    }
  }
}

__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a, int ctas) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  float* xs = reinterpret_cast<float*>(smem + sizeof(Shared));
  const int rank = static_cast<int>(blockIdx.x % ctas), clusters = gridDim.x / ctas;
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
  if (threadIdx.x < 64) sh.table[threadIdx.x] = kExp2[threadIdx.x];
  pdl_wait();
  pdl_trigger();
  int turn = 0;
  for (int64_t r = blockIdx.x / ctas; r < a.rows; r += clusters) {
    if (a.undecided && a.tokens[r] != kUndecided) continue;  // (read by all before the first exchange, written after the last)
    sample_row(a, sh, xs, r, rank, ctas, &turn);
    __syncthreads();
  }
}

// ----------------------------------------------------------- the whole distribution --
//
// Where nothing is filtered, a row need not be kept, nor its largest logit known before its weights: warps read chunks of
// 512 logits and leave each chunk's sum in units of the power of two that its own largest weight lies above. With
// x c = n + i / 16 + f (c in two fp32 parts, n whole), 2^(x c) = 2^n T[i] (1 + q), T and the result in 31 bits, each weight to
// within 2^-30 of itself (equal logits have equal weights). Chunks' sums are then shifted to the row's largest n and added,
// and the chunk in which they pass uniform * sum is read again by one warp.
//
// Bound: latency of some 29 instructions to a logit, where two logits share the packed ones. 256 rows of 200003 fp32 logits (205 MB) take
// 76 us here and 84 with what follows, 2.4 TB/s; their bytes alone would take 30. Issue slots are active in 51% of the cycles (58% of
// those in which an SM has warps); a warp waits longest for the pipe of the packed instructions, which hold it twice as long, and
// for its own last result, and 20 of the 28 warps that fit an SM are there on average. (With no loads ahead of the chunk that is
// weighed it was 93. fp32 sums of the exponential unit's weights are quicker, but in every call some rows are then too close to
// decide, and those rows' exact pass takes longer than all others.)
//
// Rows with anything that this does not hold for (an infinite largest logit, one above 512 log2 units in size, where c's
// parts no longer reach, no logit at all, a temperature of 0) keep kUndecided and are the other kernel's.

constexpr int kStreamThreads = 128, kStreamWarps = kStreamThreads / 32, kStreamCtas = 7;  // CTAs to an SM
constexpr int kChunk = 512, kPerLane = kChunk / 32;
constexpr int kMaxChunks = kSampleMaxVocab / kChunk + 1;
// Logits of a call, below which one kernel is less than two: with 8, 16, 32, 64 and 128 rows of 131072 the two took 15, 17, 31,
// 24 and 38 us and sample_kernel alone 16, 26, 25, 48 and 86, with 64, 128 and 256 rows of 32000 22, 32 and 34, and 17, 26 and 49,
// with 256 and 512 rows of 4096 16 and 18, and 15 and 29.
constexpr int64_t kStreamLeast = 1 << 21;
constexpr int kUnitBits = 13;              // a chunk's largest weight is 2^43 to 2^44 units, 409600 of them below 2^63

// 2^(30 + i / 16), rounded.
__device__ const int kExp2Few[16] = {
    1073741824, 1121280436, 1170923762, 1222764986, 1276901417, 1333434672, 1392470869, 1454120821,
    1518500250, 1585730000, 1655936265, 1729250827, 1805811301, 1885761398, 1969251188, 2056437387};

struct Weigh {
  const int* table;  // in shared memory
  float ch, cl;

  static constexpr float kMagic = 786432.0f;  // 1.5 2^19: a sum with it ends at multiples of 1/16, which its low bits count
  static constexpr float kLn2 = 0.69314718f, kLn2Tail = -1.9046542e-09f, k32 = 4294967296.0f;
  static constexpr float kMagicWhole = 12582912.0f;  // 1.5 2^23: the same at whole numbers

  // n of a logit, plus a constant.
  __device__ __forceinline__ int exponent(float x) const {
    return __float_as_int(__fadd_rn(__fmul_rn(x, ch), kMagic)) >> 4;
  }
  // sum += units of two logits' weights, the chunk's n being `top`, that of a number or of minus infinity. (Of minus infinity and of
  // logits far below, kf is so far from kMagic that nothing is left by the shift to the right, of NaN nothing by the one to the
  // left; in a chunk of nothing else the sum says nothing, and its n lets nothing of it count.)
  __device__ __forceinline__ void add_units(float x0, float x1, int top, u64* sum) const {
    const Two x(x0, x1), c(ch);
    // all of n, k and f with the other sign: n = -x c, f = -(x c - k / 16), exact and at most 1/32
    const Two n = x * Two(-ch);
    const Two pl = fma2(x, Two(cl), fma2(x, c, n));
    const Two kf = fma2(n, Two(-1.0f), Two(kMagic));
    const Two f = n + (kf + Two(-kMagic));
    const Two h = f * Two(-kLn2);
    // 2^(x c - k / 16) - 1 = h + (-f ln2 - h) + pl ln2 (1 + h) + f^2 (...), pl what x c has below n
    Two e = fma2(f, Two(-kLn2), f * Two(kLn2));
    e = fma2(f, Two(-kLn2Tail), e);
    e = fma2(fma2(pl, h, pl), Two(kLn2), e);
    Two g = fma2(f, Two(-1.3333558e-03f), Two(9.6181291e-03f));
    g = fma2(f, g, Two(-5.5504109e-02f));
    g = fma2(f, g, Two(2.4022651e-01f));
    e = fma2(f * f, g, e);
    const float2 hi = (h * Two(k32)).get(), lo = fma2(e, Two(k32), Two(kMagicWhole)).get(), kk = kf.get();
    one(hi.x, lo.x, kk.x, top, sum);
    one(hi.y, lo.y, kk.y, top, sum);
  }
  __device__ __forceinline__ u64 units(float x, int top) const {
    u64 sum = 0;
    add_units(x, -INFINITY, top, &sum);
    return sum;
  }

  __device__ __forceinline__ void one(float hi, float lo, float kf, int top, u64* sum) const {
    const int q = __float2int_rn(hi) + (__float_as_int(lo) - 0x4b400000);  // 2^f - 1 in units of 2^-32
    const int bits = __float_as_int(kf), t = table[bits & 15];
    const uint32_t m = static_cast<uint32_t>(t + __mulhi(t, q));
    const int past = top - (bits >> 4) - kUnitBits;
    uint32_t rest, by;
    asm("shr.u32 %0, %1, %2;" : "=r"(rest) : "r"(m), "r"(max(past, 0)));  // (0 from 32 on)
    asm("shl.b32 %0, %1, %2;" : "=r"(by) : "r"(1), "r"(max(-past, 0)));
    *sum += static_cast<u64>(rest) * by;
  }
};

// kCount elements of a row of n from `at` on, minus infinity outside. Aligned: `at` is at a 16-byte boundary.
template <typename T, int kCount> __device__ __forceinline__ void load_inside(const T* row, int at, float* x) {
  constexpr int kVec = 16 / sizeof(T);
#pragma unroll
  for (int v = 0; v < kCount / kVec; ++v) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + at + v * kVec));
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[v * kVec + j] = Ty<T>::to_f(e[j]);
  }
}
template <typename T, int kCount> __device__ __forceinline__ void load_edge(const T* row, int at, int n, float* x) {
#pragma unroll
  for (int j = 0; j < kCount; ++j) x[j] = at + j >= 0 && at + j < n ? Ty<T>::to_f(row[at + j]) : -INFINITY;
}

template <typename T> __global__ void __launch_bounds__(kStreamThreads, kStreamCtas) stream_kernel(SampleArgs a, int ctas) {
  __shared__ u64 sums[kMaxChunks];
  __shared__ int tops[kMaxChunks];
  __shared__ int table[16];
  __shared__ u64 red[kStreamWarps], exchange[2][kMaxCluster];
  __shared__ u64 chosen_before;
  __shared__ int chosen;
  constexpr int kVec = 16 / sizeof(T);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ double scale;
  __shared__ float2 parts;  // of scale
  if (tid < 16) table[tid] = kExp2Few[tid];
  if (tid == 0) chosen = -1;
  pdl_wait();
  pdl_trigger();
  const int64_t r = blockIdx.x / ctas;
  const int rank = static_cast<int>(blockIdx.x % ctas);
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  // chunks begin at 16-byte boundaries, the first one up to a vector before the row
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int chunks = (a.vocab + shift + kChunk - 1) / kChunk, each = (chunks + ctas - 1) / ctas;
  const int c0 = min(chunks, rank * each), c1 = min(chunks, c0 + each);
  const float t = a.temperatures ? a.temperatures[r] : a.temperature;
  if (tid == 0) {  // (fp64 is slow enough here that all threads' would show)
    if (rank == 0) a.tokens[r] = kUndecided;
    scale = 1.4426950408889634 / static_cast<double>(t);
    parts = make_float2(static_cast<float>(scale), static_cast<float>(scale - static_cast<double>(static_cast<float>(scale))));
  }
  __syncthreads();
  const Weigh weigh = {table, parts.x, parts.y};
  if (!(t > 0.0f) || !(weigh.ch < 1e30f) || !(weigh.ch > 1e-30f)) return;  // (all CTAs of the row)
  const auto chunk_top = [&](const float* x) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kPerLane; ++i) top = fmaxf(top, x[i]);
    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(top));
    return fmaxf(top, -INFINITY);  // (of nothing but NaN, too)
  };
  float most = -INFINITY;  // of the chunks that this warp has seen
  const auto inside = [&](int k) { return k * kChunk >= shift && (k + 1) * kChunk - shift <= a.vocab; };
  uint4 next[kPerLane / kVec];  // of the chunk after this one
  const auto fetch = [&](int k) {
#pragma unroll
    for (int v = 0; v < kPerLane / kVec; ++v)
      next[v] = __ldg(reinterpret_cast<const uint4*>(row + k * kChunk - shift + lane * kVec + v * 32 * kVec));
  };
  if (c0 + warp < c1 && inside(c0 + warp)) fetch(c0 + warp);
  for (int k = c0 + warp; k < c1; k += kStreamWarps) {
    float x[kPerLane];
    if (inside(k)) {
#pragma unroll
      for (int v = 0; v < kPerLane / kVec; ++v)
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[v * kVec + j] = Ty<T>::to_f(reinterpret_cast<const T*>(&next[v])[j]);
    } else {
#pragma unroll
      for (int v = 0; v < kPerLane / kVec; ++v)
        load_edge<T, kVec>(row, k * kChunk - shift + lane * kVec + v * 32 * kVec, a.vocab, x + v * kVec);
    }
    if (k + kStreamWarps < c1 && inside(k + kStreamWarps)) fetch(k + kStreamWarps);
    const float top = chunk_top(x);
    most = fmaxf(most, top);
    const int n = weigh.exponent(top);
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; i += 2) weigh.add_units(x[i], x[i + 1], n, &sum);
    // (below 2^49 a lane)
    const uint32_t high = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(sum >> 27));
    sum = (static_cast<u64>(high) << 27) + __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(sum) & 0x7ffffffu);
    if (lane == 0) {
      sums[k - c0] = sum;
      tops[k - c0] = n;
    }
  }
  int turn = 0;
  // every CTA has begun before anything is stored into its shared memory
  row_sync();
  const auto gather = [&](u64 v) -> const u64* {
    turn ^= 1;
    if (tid < ctas) st_cluster(mapa_shared(smem_addr(&exchange[turn][rank]), tid), v);
    row_sync();
    return exchange[turn];
  };
  if (lane == 0) red[warp] = key_of(most);
  __syncthreads();
  u64 highest = 0;
  for (int w = 0; w < kStreamWarps; ++w) highest = max(highest, red[w]);
  __syncthreads();
  const u64* all = gather(highest);
  for (int i = 0; i < ctas; ++i) highest = max(highest, all[i]);
  most = value_of(static_cast<uint32_t>(highest));
  if (!(fabsf(most) * weigh.ch <= 512.0f)) return;
  const int top = weigh.exponent(most);
  // (n is at most top, and far below it in a chunk without any logit above minus infinity)
  const auto down = [&](u64 v, int n) -> u64 { return static_cast<unsigned>(top - n) < 64 ? v >> (top - n) : 0; };
  constexpr int kEach = (kMaxChunks + kStreamThreads - 1) / kStreamThreads;
  u64 v[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int k = tid * kEach + i;
    v[i] = k < c1 - c0 ? down(sums[k], tops[k]) : 0;
    sum += v[i];
  }
  const u64 upto = warp_scan_u64(sum);
  if (lane == 31) red[warp] = upto;
  __syncthreads();
  u64 before = upto - sum, mine = 0;
  for (int w = 0; w < kStreamWarps; ++w) {
    if (w < warp) before += red[w];
    mine += red[w];
  }
  const u64* totals = gather(mine);
  u64 total = 0;
  for (int i = 0; i < ctas; ++i) {
    if (i < rank) before += totals[i];
    total += totals[i];
  }
  float u = a.uniform[r];
  u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;
  const u64 want = min(total, part_of(u, total) + 1);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (before < want && want <= before + v[i]) {
      chosen = tid * kEach + i;
      chosen_before = before;
    }
    before += v[i];
  }
  __syncthreads();
  if (chosen < 0 || warp != 0) return;
  // the chunk again, a run of 32 to a lane
  const int at = (c0 + chosen) * kChunk - shift + lane * kPerLane, n = tops[chosen];
  float x[kPerLane];
  if (at >= 0 && at + kPerLane <= a.vocab) load_inside<T, kPerLane>(row, at, x);
  else load_edge<T, kPerLane>(row, at, a.vocab, x);
  u64 part = 0;
#pragma unroll
  for (int i = 0; i < kPerLane; i += 2) weigh.add_units(x[i], x[i + 1], n, &part);
  u64 run = warp_scan_u64(part) - part;
  // (its sums are shifted like the chunk's, so that the last one is the chunk's)
  u64 from = chosen_before + down(run, n);
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const u64 w = weigh.units(x[i], n);
    run += w;
    const u64 to = chosen_before + down(run, n);
    if (from < want && want <= to) {
      a.tokens[r] = at + i;
      if (a.logprobs) a.logprobs[r] = log_share(down(w, n), static_cast<double>(x[i]) * scale + (43 - (top - weigh.exponent(0.0f))), total);
    }
    from = to;
  }
}

// ------------------------------------------------------------------ few candidates --
//
// Most rows that filter come down to a few tokens, and for those neither a copy of the row nor a histogram of it is needed.
// Each of a CTA's 1024 threads keeps the largest of its logits. The k-th largest logit is not below the k-th largest of the
// threads' (which a histogram of those finds, to within a step), and min_p says how far down it goes; threads whose largest
// reaches that far have theirs looked through again, and what reaches as far is listed. For top_p without top_k the 128-th
// takes the place of the k-th, and it has to turn out that the listed weights come to p of all. One CTA finishes the row:
// with no more than 512 candidates, each is compared with all others. Rows with more keep kUndecided.
//
// Bound: latency, of the logits' bytes (1 to 2 us of them) and of four or five steps of a row's CTAs together. 64 rows of
// 131072 fp32 logits with top_k, top_p and min_p take 15 us (33.6 MB: 4.9 us): 2.8 until all are read, 1.3 for the largest, 2 for the
// border, 2 for the list, 3 to finish, and 2 for the next kernel to see that nothing is left. One row of 131072 bf16 logits with
// top_p takes 19 us, 3 of them for the weights of all. (Dealing out the vectors that are looked through again to all threads
// took 64 rows from 22 to 15 us; a histogram for each CTA rather than the first one's for all, one row from 23 to 20 with 8 CTAs.)
//
// CTAs to a row, as long as rows leave SMs idle: as many as leave 4096 logits to each (one row of 50001 with min_p takes 7.8 us with
// eight and 8.7 with the four that 8192 would make it; from 131072 on 8192 or less make no difference).

constexpr int kPickThreads = 1024, kPickWarps = kPickThreads / 32;
constexpr int kPicked = 512;   // candidates at most
constexpr int kMostK = 400;    // a larger top_k is not tried
constexpr int kTryP = 128;

struct PickShared {
  u64 table[64];
  Params params;
  u64 tops[kMaxCluster], sums[kMaxCluster];
  u64 red[kPickWarps];
  alignas(8) uint32_t hist[kBins];
  int border;
  uint32_t mass;  // of the largest logits of the threads down to the border, in units of the largest (a float's bits)
  uint32_t listed, looking;
  u64 list[kPicked], weights[kPicked];
  uint16_t who[kPickThreads];  // threads whose logits are looked through again
};

__device__ __forceinline__ uint32_t add_cluster(uint32_t addr, uint32_t v) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void st_cluster32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// The halves of row_sync.
__device__ __forceinline__ void row_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void row_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint2 ld_cluster2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ u64 pick_sum(PickShared& sh, u64 v) {
  v = warp_sum_u64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum_u64(sh.red[threadIdx.x & 31]);
}

template <typename T> __global__ void __launch_bounds__(kPickThreads, 1) pick_kernel(SampleArgs a, int ctas) {
  __shared__ PickShared sh;
  constexpr int kVec = 16 / sizeof(T), kAhead = 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster_arrive_relaxed();
  const int64_t r = blockIdx.x / ctas;
  const int rank = static_cast<int>(blockIdx.x % ctas);
  for (int i = tid; i < kBins; i += kPickThreads) sh.hist[i] = 0;
  if (tid < 64) sh.table[tid] = kExp2[tid];
  if (tid == 64) sh.listed = 0;
  if (tid == 65) sh.border = -1;
  if (tid == 67) sh.mass = 0x7f800000u;
  if (tid == 66) sh.looking = 0;
  pdl_wait();
  pdl_trigger();
  if (tid == kPickThreads - 1) row_params(a, r, &sh.params);
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  // vectors begin at 16-byte boundaries, the first one up to 16 bytes before the row
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const int vectors = (a.vocab + shift + kVec - 1) / kVec, each = (vectors + ctas - 1) / ctas;
  const int v0 = min(vectors, rank * each), v1 = min(vectors, v0 + each);
  // f(index, logit) for all of this thread's elements, indexes rising
  const auto one_vector = [&](int v, auto f) {
    const int at = v * kVec - shift;
    float x[kVec];
    if (at >= 0 && at + kVec <= a.vocab) load_inside<T, kVec>(row, at, x);
    else load_edge<T, kVec>(row, at, a.vocab, x);
#pragma unroll
    for (int j = 0; j < kVec; ++j) f(at + j, x[j]);
  };
  const auto visit = [&](auto f) {
#pragma unroll 1
    for (int v = v0 + tid; v < v1; v += kPickThreads) one_vector(v, f);
  };
  float top = -INFINITY;
  int arg = -1;
  const auto look = [&](int i, float x) {
    if (x > top) {  // (not for NaN)
      top = x;
      arg = i;
    }
  };
  for (int v = v0 + tid; v < v1; v += kAhead * kPickThreads) {
    const int at = v * kVec - shift;
    if (at >= 0 && v + (kAhead - 1) * kPickThreads < v1 && at + ((kAhead - 1) * kPickThreads + 1) * kVec <= a.vocab) {
      float x[kAhead][kVec];  // (all loads before any use)
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load_inside<T, kVec>(row, at + i * kPickThreads * kVec, x[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) look(at + i * kPickThreads * kVec + j, x[i][j]);
    } else {
#pragma unroll 1
      for (int i = 0; i < kAhead && v + i * kPickThreads < v1; ++i) one_vector(v + i * kPickThreads, look);
    }
  }
  u64 best = arg < 0 ? 0 : static_cast<u64>(key_of(top)) << 32 | (0xffffffffu - static_cast<uint32_t>(arg));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) sh.red[warp] = best;
  __syncthreads();
  best = sh.red[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  cluster_wait();  // (every CTA has begun)
  if (tid < ctas) st_cluster(mapa_shared(smem_addr(&sh.tops[rank]), tid), best);
  row_sync();
  for (int i = 0; i < ctas; ++i) best = max(best, sh.tops[i]);
  const Params& p = sh.params;
  const bool none = best == 0;
  const bool cut_k = p.k > 0 && p.k < a.vocab, cut_p = p.p < 1.0f, cut_m = p.step < kBins && !cut_p;
  const bool one = none || !(p.t > 0.0f) || p.k == 1 || p.p <= 0.0f;
  if (one || !(cut_k || cut_p || cut_m) || (cut_k && p.k > kMostK && !cut_m)) {
    if (rank == 0 && tid == 0) {
      a.tokens[r] = none ? -1 : one ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : kUndecided;
      if (a.logprobs && one) a.logprobs[r] = none ? -INFINITY : 0.0f;
    }
    return;
  }
  const Scale scale = {sh.table, value_of(static_cast<uint32_t>(best >> 32)), p.ch, p.cl};
  const int mine = arg < 0 ? kBins : scale.step(top);
  int bin = cut_m ? p.step : kBins;
  const uint32_t some = cut_k ? p.k : kTryP;
  if ((cut_k || cut_p) && some <= kMostK) {
    if (arg >= 0) atomicAdd(&sh.hist[mine], 1u);
    row_arrive();
    if (cut_p && !cut_k) {  // (while the others come)
      u64 sum = 0;
      visit([&](int, float x) { sum += scale.weight(x); });
      sum = pick_sum(sh, sum);
      if (tid < ctas) st_cluster(mapa_shared(smem_addr(&sh.sums[rank]), tid), sum);
    }
    row_wait();
    __syncthreads();  // (that sum is read by all)
    if (rank == 0) {
      uint32_t n0 = 0, n1 = 0;
      for (int i = 0; i < ctas; ++i) {
        const uint2 n = ld_cluster2(mapa_shared(smem_addr(&sh.hist[2 * tid]), i));
        n0 += n.x;
        n1 += n.y;
      }
      // counts, and below them the weights of those logits by their steps, in units of 2^-20 (together at most 2^34 of them)
      const auto entry = [&](uint32_t n, int step) {
        return static_cast<u64>(n) << 36 | static_cast<u64>(n * exp2f(20.0f - step * (kRange / kBins)));
      };
      const u64 e0 = entry(n0, 2 * tid), e1 = entry(n1, 2 * tid + 1), upto = warp_scan_u64(e0 + e1);
      if (lane == 31) sh.red[warp] = upto;
      __syncthreads();
      u64 prior = upto - (e0 + e1);
      for (int w = 0; w < warp; ++w) prior += sh.red[w];
      const uint32_t before = static_cast<uint32_t>(prior >> 36);
      const int at = before < some && some <= before + n0 ? 2 * tid : before + n0 < some && some <= before + n0 + n1 ? 2 * tid + 1 : -1;
      if (at >= 0) {
        const u64 upto_it = prior + e0 + (at & 1 ? e1 : 0);
        const float mass = static_cast<float>(upto_it & ((1ull << 36) - 1)) * 0x1p-20f;
        for (int i = 0; i < ctas; ++i) {
          st_cluster32(mapa_shared(smem_addr(&sh.border), i), static_cast<uint32_t>(at));
          st_cluster32(mapa_shared(smem_addr(&sh.mass), i), __float_as_uint(mass));
        }
      }
    }
    row_sync();
    // (fewer threads than that have a logit: all steps, unless min_p has a say)
    bin = min(bin, sh.border < 0 ? kBins : sh.border);
  }
  u64 total = 0;
  if (cut_p && !cut_k) {
    for (int i = 0; i < ctas; ++i) total += sh.sums[i];
    // (most of what would be listed is among those, so there is no hope if p of all is far above them)
    if (p.p * static_cast<float>(total) > 1.3f * __uint_as_float(sh.mass) * static_cast<float>(kOne)) {
      if (rank == 0 && tid == 0) a.tokens[r] = kUndecided;
      return;
    }
  }
  // (their vectors are dealt out to all threads, so that all are on their way at once)
  const uint32_t ballot = __ballot_sync(0xffffffffu, mine <= bin);
  uint32_t place0 = lane == 0 && ballot != 0 ? atomicAdd(&sh.looking, __popc(ballot)) : 0u;
  place0 = __shfl_sync(0xffffffffu, place0, 0);
  if (mine <= bin) sh.who[place0 + __popc(ballot & ((1u << lane) - 1u))] = static_cast<uint16_t>(tid);
  __syncthreads();
  {
    const uint32_t at_most = mapa_shared(smem_addr(&sh.listed), 0), list = mapa_shared(smem_addr(sh.list), 0);
    const int turns = (v1 - v0 + kPickThreads - 1) / kPickThreads, items = static_cast<int>(sh.looking) * turns;
#pragma unroll 1
    for (int item = tid; item < items; item += kPickThreads) {
      const int which = item / turns, v = v0 + sh.who[which] + (item - which * turns) * kPickThreads;
      if (v < v1)
        one_vector(v, [&](int i, float x) {
          if (x > -INFINITY && scale.step(x) <= bin) {
            const uint32_t at = add_cluster(at_most, 1u);
            if (at < kPicked) st_cluster(list + 8 * at, static_cast<u64>(~key_of(x)) << 32 | static_cast<uint32_t>(i));
          }
        });
    }
  }
  row_sync();
  if (rank != 0) return;
  const int count = static_cast<int>(sh.listed);
  if (count > kPicked) {
    if (tid == 0) a.tokens[r] = kUndecided;
    return;
  }
  // In order, the first k stay, of those the ones before which less than p of the sum lies, of those the ones not below least.
  // `share` neighbouring threads have a candidate, each looks at every share-th other one, and the first has the result.
  int share = 2;
  while (share < 32 && 2 * share * count <= kPickThreads) share *= 2;
  const int mate = tid & (share - 1), own = tid / share;
  const bool have = own < count && mate == 0;
  const u64 me = own < count ? sh.list[own] : 0;
  u64 w = have ? scale.weight(value_of(~static_cast<uint32_t>(me >> 32))) : 0;
  if (have) sh.weights[own] = w;
  const u64 listed = pick_sum(sh, w);
  u64 before = 0;
  uint32_t place = 0;
  if (own < count) {
#pragma unroll 4
    for (int j = mate; j < count; j += share)
      if (sh.list[j] < me) {
        before += sh.weights[j];
        ++place;
      }
  }
  for (int o = 1; o < share; o <<= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    place += __shfl_xor_sync(0xffffffffu, place, o);
  }
  u64 goal = ~0ull;
  if (cut_k && place >= p.k) w = 0;
  if (cut_p) {
    if (cut_k) total = pick_sum(sh, w);
    goal = reach(p.p, total);
    if (!cut_k && listed < goal) {  // (the last one that stays is not among them)
      if (tid == 0) a.tokens[r] = kUndecided;
      return;
    }
  }
  if (before >= goal || w < p.least) w = 0;
  const u64 all = pick_sum(sh, w);  // (with barriers, behind which all have read the weights)
  if (have) sh.weights[own] = w;
  __syncthreads();
  // in the order of the index, the token
  const u64 want = min(all, part_of(p.u, all) + 1);
  before = 0;
  if (own < count) {
#pragma unroll 4
    for (int j = mate; j < count; j += share)
      if (static_cast<uint32_t>(sh.list[j]) < static_cast<uint32_t>(me)) before += sh.weights[j];
  }
  for (int o = 1; o < share; o <<= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (w != 0 && before < want && want <= before + w) {
    const int token = static_cast<int>(static_cast<uint32_t>(me));
    a.tokens[r] = token;
    if (a.logprobs) a.logprobs[r] = log_share(w, w < kPlainLog ? scale.log2_units(a, r, token) : 0.0, all);
  }
}

// How many clusters of kMaxCluster CTAs of a kernel the current device can have at once, 0 if none. Asked once for a device.
template <auto Kernel> int wide_clusters(int threads, size_t smem) {
  static std::atomic<int> known[64];  // the number + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCluster);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kMaxCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if ((smem > 0 && ensure_smem<Kernel>(smem) != cudaSuccess) ||
        cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&clusters, Kernel, &cfg) != cudaSuccess) {
      clusters = 0;
      cudaGetLastError();  // (a launch with fewer CTAs has no part in that)
    }
    n = clusters + 1;
    known[dev].store(n, std::memory_order_release);
  }
  return n - 1;
}

}  // namespace

cudaError_t launch_token_sample(const hc_token_sample_t& p, int num_sms, cudaStream_t s) {
  // As few CTAs to a row as its slices allow, and more while rows alone leave SMs idle.
  int ctas = 1;
  while (static_cast<int64_t>(ctas) * kMaxSlice < p.vocab) ctas *= 2;
  const auto more = [&](int c, int most, int least) { return p.rows * c * 2 <= num_sms && c < most && p.vocab / (2 * c) >= least; };
  const auto wide = [&](int clusters) { return p.rows <= clusters ? kMaxCluster : kCluster; };
  const int most = wide(wide_clusters<sample_kernel>(kThreads, sizeof(Shared) + kMaxSlice * sizeof(float)));
  while (more(ctas, most, 2048)) ctas *= 2;
  const int slice = ((p.vocab + ctas - 1) / ctas + 31) / 32 * 32;
  SampleArgs a = {p.logits, p.uniform, p.temperatures, p.top_ps, p.min_ps, p.top_ks, p.tokens_out, p.logprobs_out,
                  p.logits_stride, p.rows, p.vocab, slice, p.top_k, p.dtype, p.temperature, p.top_p, p.min_p, false};
  int64_t clusters = p.rows;
  const bool whole = p.top_ks == nullptr && (p.top_k <= 0 || p.top_k >= p.vocab) && p.top_ps == nullptr && !(p.top_p < 1.0f) &&
                     p.min_ps == nullptr && !(p.min_p > 0.0f);
  if (whole && p.rows * p.vocab >= kStreamLeast) {
    int split = 1;
    // (all at once, since the CTAs of a row wait for one another)
    while (split < kCluster && p.rows * split * 2 <= kStreamCtas * num_sms && p.vocab / (2 * split) >= 4 * kStreamWarps * kChunk)
      split *= 2;
    const dim3 grid(static_cast<unsigned>(p.rows * split)), block(kStreamThreads);
    cudaError_t e;
    if (p.dtype == HC_F32) e = launch_pdl(stream_kernel<float>, grid, block, 0, s, split, a, split);
    else if (p.dtype == HC_F16) e = launch_pdl(stream_kernel<__half>, grid, block, 0, s, split, a, split);
    else e = launch_pdl(stream_kernel<__nv_bfloat16>, grid, block, 0, s, split, a, split);
    if (e != cudaSuccess) return e;
  } else if (!whole) {
    const auto launch = [&](auto type) {
      using T = decltype(type);
      const int most_here = wide(wide_clusters<pick_kernel<T>>(kPickThreads, 0));
      int split = 1;
      while (more(split, most_here, kPickThreads * 4)) split *= 2;
      return launch_pdl(pick_kernel<T>, dim3(static_cast<unsigned>(p.rows * split)), dim3(kPickThreads), 0, s, split, a, split);
    };
    const cudaError_t e = p.dtype == HC_F32   ? launch(float())
                          : p.dtype == HC_F16 ? launch(__half())
                                              : launch(__nv_bfloat16());
    if (e != cudaSuccess) return e;
  }
  if (!whole || p.rows * p.vocab >= kStreamLeast) {  // what those have left
    a.undecided = true;
    clusters = std::min<int64_t>(p.rows, std::max(1, num_sms / ctas));
  }
  const size_t smem = sizeof(Shared) + static_cast<size_t>(std::max(slice, kMinSlice)) * sizeof(float);
  const cudaError_t e = ensure_smem<sample_kernel>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(sample_kernel, dim3(static_cast<unsigned>(clusters * ctas)), dim3(kThreads), smem, s, ctas, a, ctas);
}

}  // namespace hc
