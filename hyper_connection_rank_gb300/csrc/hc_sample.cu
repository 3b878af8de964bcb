// The choice of the next tokens (hc_token_sample).
//
// A cluster of CTAs takes a row and reads it once: each CTA keeps its slice of the
// row in shared memory, where every later pass finds it. The steps are
//
//   1. the largest logit m and its first index;
//   2. with top_k, the k-th token in the order (logit falling, index rising);
//   3. with top_p, the last token of that order that stays;
//   4. the sum of the weights that stay, per warp, CTA and row;
//   5. the token: the CTA, the warp, the lane and at last the element in which the
//      cumulated weight passes uniform * sum.
//
// Steps 2 and 3 find the first element of the order at which a cumulated value
// (1 each, or the weights) reaches a target: a histogram over 2048 equal steps of
// the exponent, merged over the cluster, then histograms over the logits' bits
// within the step that the target falls into, until one value is left; among
// elements of that value the index decides.
//
// Weights are integers, 2^43 for the largest logit: integer sums have one result
// in any order, whatever threads, warps and CTAs make of it, and a row of 409600
// weights stays below 2^62. A weight is 2^-y with y = (m - x) log2(e) / t formed
// in two fp32 parts; y = (64 n + i + f) / 64, and 2^-y = 2^-n T[i] (1 + q), where T
// is a table and q = 2^(-f/64) - 1 a polynomial in fp32 whose leading term is
// kept apart, so that the whole is good to 2^-38 of itself (fp32's 2^-24 would
// choose another token than the definition once in some thousand rows of 10^5
// tokens; fp64 runs at 1/64 of the rate here).
//
// REPLACE_MEASURED
#include "hc_async.cuh"
#include "hc_common.cuh"
#include "hc_experts_internal.h"

namespace hc {
namespace {

using u64 = unsigned long long;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = kSampleMaxVocab / kMaxCluster;  // elements that a CTA keeps
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
  int vocab, slice, top_k, dtype;
  float temperature, top_p, min_p;
};

struct Shared {
  u64 table[64];
  u64 exchange[2][kMaxCluster];
  u64 red[kWarps];
  u64 border[4];  // where a target falls: bin, value before it, value in it
  uint32_t lo[kBins], hi[kBins];
};

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

// One row, as a thread sees it.
struct Row {
  Shared& sh;
  const float* xs;       // this CTA's slice
  int n, base;           // its elements, and the first one's index in the row
  int rank, ctas, turn;  // turn: of the exchanges
  float m, ch, cl;       // largest logit; log2(e) / temperature in two parts
  uint32_t cut_key, cut_index;  // what stays: keys above, and equal ones up to this index

  // Every CTA's value, in the order of the ranks, in exchange[turn].
  __device__ __forceinline__ const u64* gather(u64 v) {
    turn ^= 1;
    if (threadIdx.x < ctas) st_cluster(mapa_shared(smem_addr(&sh.exchange[turn][rank]), threadIdx.x), v);
    cluster_sync_all();
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
    const u64 t = sh.table[j & 63];
    const long long w =
        static_cast<long long>(t) + ((static_cast<long long>(static_cast<int>(t >> 13)) * q) >> 25);
    return static_cast<u64>(w) >> (j >> 6);
  }

  __device__ __forceinline__ void add(int bin, u64 v) {
    const uint32_t lo = static_cast<uint32_t>(v);
    const uint32_t old = atomicAdd(&sh.lo[bin], lo);
    const uint32_t up = static_cast<uint32_t>(v >> 32) + (old + lo < old ? 1u : 0u);
    if (up != 0) atomicAdd(&sh.hi[bin], up);
  }

  // The histograms of all CTAs together: into which bin the target falls (border[0]), what lies before it (border[1]) and
  // in it (border[2]). target(total) gives the target. The histogram is empty again afterwards.
  template <class F> __device__ __forceinline__ void find(F target) {
    cluster_sync_all();
    const int mine = kBins / ctas, per = max(1, mine / kThreads), at = threadIdx.x * per;
    u64 v[kBins / kThreads], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins / kThreads; ++i) {
      v[i] = 0;
      if (i < per && at + i < mine) {
        const int bin = rank * mine + at + i;
        for (int r = 0; r < ctas; ++r)
          v[i] += ld_cluster(mapa_shared(smem_addr(&sh.lo[bin]), r)) +
                  (static_cast<u64>(ld_cluster(mapa_shared(smem_addr(&sh.hi[bin]), r))) << 32);
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
    cluster_sync_all();
  }

  // The first element, in the order of falling logits and rising indexes, at which the values cumulated over what stays
  // reach a target becomes the last one that stays. With `mass` the values are the weights and the target is p times
  // their sum, otherwise they are 1 and the target is k.
  __device__ __forceinline__ void cut(bool mass, double p, u64 k) {
    u64 want = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float x = xs[i];
      if (!stays(x, base + i)) continue;
      const u64 v = mass ? weight(x) : 1;
      if (v != 0) add(step(x), v);
    }
    find([&](u64 total) {
      want = k;
      if (mass) {
        const double t = ceil(p * static_cast<double>(total));
        want = t < 1.0 ? 1 : static_cast<u64>(t);
      }
      want = min(want, total);
      return want;
    });
    const int bin = static_cast<int>(sh.border[0]);
    want -= sh.border[1];
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
        const u64 v = mass ? weight(x) : 1;
        if (v != 0) add((high - key) >> shift, v);
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

__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs a, int ctas) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  float* xs = reinterpret_cast<float*>(smem + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t r = blockIdx.x / ctas;
  const int rank = static_cast<int>(blockIdx.x % ctas);
  const int base = rank * a.slice, n = max(0, min(a.slice, a.vocab - base));
  for (int i = tid; i < kBins; i += kThreads) sh.lo[i] = sh.hi[i] = 0;
  if (tid < 64) sh.table[tid] = kExp2[tid];
  pdl_wait();
  pdl_trigger();
  u64 best;
  if (a.dtype == HC_F32)
    best = load_slice(static_cast<const float*>(a.logits) + r * a.stride, base, n, xs);
  else if (a.dtype == HC_F16)
    best = load_slice(static_cast<const __half*>(a.logits) + r * a.stride, base, n, xs);
  else
    best = load_slice(static_cast<const __nv_bfloat16*>(a.logits) + r * a.stride, base, n, xs);
  const float t = a.temperatures ? a.temperatures[r] : a.temperature;
  const float p = a.top_ps ? a.top_ps[r] : a.top_p;
  const float least = a.min_ps ? a.min_ps[r] : a.min_p;
  const int k = a.top_ks ? a.top_ks[r] : a.top_k;
  float u = a.uniform[r];
  u = u > 0.0f ? fminf(u, 1.0f) : 0.0f;

  // (every CTA of the cluster has begun before anything is stored into its shared memory)
  cluster_sync_all();
  Row row = {sh, xs, n, base, rank, ctas, 0, 0.0f, 0.0f, 0.0f, 0u, 0xffffffffu};
  best = row.cluster_max(best);
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
  const double c = 1.4426950408889634 / static_cast<double>(t);
  row.ch = static_cast<float>(c);
  row.cl = isinf(row.ch) ? 0.0f : static_cast<float>(c - static_cast<double>(row.ch));
  if (k > 0 && k < a.vocab) row.cut(false, 0.0, static_cast<u64>(k));
  if (p < 1.0f) row.cut(true, static_cast<double>(p), 0);
  const u64 floor_w = least > 0.0f ? static_cast<u64>(ceil(static_cast<double>(fminf(least, 1.0f)) * static_cast<double>(kOne))) : 1;
  const auto kept = [&](int i) -> u64 {
    const float x = xs[i];
    if (!row.stays(x, base + i)) return 0;
    const u64 w = row.weight(x);
    return w >= floor_w ? w : 0;
  };

  // a warp's sum over a run of elements, which its lanes take in turn
  const int chunk = (n + kWarps - 1) / kWarps, lo = min(n, warp * chunk), hi = min(n, lo + chunk);
  u64 mine = 0;
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
  u64 total = 0;
  for (int i = 0; i < ctas; ++i) {
    if (i < rank) before += totals[i];
    total += totals[i];
  }
  // the first element whose cumulated weight passes uniform * total, so is at least the next integer
  const u64 want = min(total, static_cast<u64>(static_cast<double>(u) * static_cast<double>(total)) + 1);
  if (!(before < want && want <= before + mine)) return;
  // in one warp: its lanes sum a run each (begun at another place each, for the sake of the memory banks)
  const int run = (hi - lo + 31) / 32, l0 = min(hi, lo + lane * run), ln = min(hi, l0 + run) - l0;
  u64 part = 0;
  for (int i = 0; i < ln; ++i) {
    int j = i + lane;
    j %= ln;
    part += kept(l0 + j);
  }
  u64 upto = before + warp_scan_u64(part);
  const uint32_t passed = __ballot_sync(0xffffffffu, upto >= want);
  const int owner = __ffs(passed) - 1;
  before = __shfl_sync(0xffffffffu, upto - part, owner);
  const int r0 = __shfl_sync(0xffffffffu, l0, owner), rn = __shfl_sync(0xffffffffu, ln, owner);
  for (int i0 = 0; i0 < rn; i0 += 32) {
    const int i = i0 + lane;
    const u64 w = i < rn ? kept(r0 + i) : 0;
    upto = before + warp_scan_u64(w);
    const uint32_t hit = __ballot_sync(0xffffffffu, upto >= want);
    if (hit != 0) {
      if (lane == __ffs(hit) - 1) {
        a.tokens[r] = base + r0 + i;
        // -log(sum / w) by what the others have, so that a token with nearly all of the weight keeps its digits
        if (a.logprobs) a.logprobs[r] = -log1pf(static_cast<float>(total - w) / static_cast<float>(w));
      }
      return;
    }
    before = __shfl_sync(0xffffffffu, upto, 31);
  }
}

}  // namespace

cudaError_t launch_token_sample(const hc_token_sample_t& p, int num_sms, cudaStream_t s) {
  // As few CTAs to a row as its slices allow, and more while rows alone leave SMs idle.
  int ctas = 1;
  while (static_cast<int64_t>(ctas) * kMaxSlice < p.vocab) ctas *= 2;
  while (ctas < kMaxCluster && p.rows * ctas * 2 <= num_sms && p.vocab / (2 * ctas) >= 2048) ctas *= 2;
  const int slice = ((p.vocab + ctas - 1) / ctas + 31) / 32 * 32;
  const SampleArgs a = {p.logits, p.uniform, p.temperatures, p.top_ps, p.min_ps, p.top_ks, p.tokens_out, p.logprobs_out,
                        p.logits_stride, p.vocab, slice, p.top_k, p.dtype, p.temperature, p.top_p, p.min_p};
  const size_t smem = sizeof(Shared) + static_cast<size_t>(slice) * sizeof(float);
  const cudaError_t e = ensure_smem<sample_kernel>(smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(sample_kernel, dim3(static_cast<unsigned>(p.rows * ctas)), dim3(kThreads), smem, s, ctas, a, ctas);
}

}  // namespace hc
