// Upkeep of a paged pool (include/hc_paged.h): copies of pages, and the
// kernels that rewrite tables and reference counts when sequences fork, grow,
// end, or when the pool is compacted.
//
// Two kernels to a call at most. The first works on the tables and counts: a
// cluster of up to 8 CTAs, whose phases are separated by cluster barriers
// (counts need every table entry before a page is known to be free, and free
// pages need counts). The second moves the pages. All sums are of integers, so
// the order of atomics does not show in the results.
//
// Bound: the tables and counts are small and their phases depend on one
// another, so that part is latency; the copies are bound by bytes, each page
// read and written once. More CTAs than fit at once copy faster than a
// persistent grid does (8 of 256 threads to an SM 56 and 163 us, 64 of 512
// threads 51 and 141 us for the two below), but not one for each piece (159
// us): a grid-stride loop keeps the tail short, new CTAs keep loads coming.
//
// Measured: 100 pages of 16 KB in 96 planes copied in 49.5 us, 6.4 TB/s, 95% of the
// measured copy bandwidth; a pool of 1501 pages of 32 KB in 48 planes compacted
// (285 pages moved) in 139.5 us, 6.4 TB/s, 96%.
#include <algorithm>

#include "hc_async.cuh"
#include "hc_common.cuh"
#include "hc_paged_internal.h"

namespace hc {
namespace {

constexpr int kMeta = 1024;       // threads of a CTA of the table kernels
constexpr int kMaxCluster = 8;    // their CTAs (the portable cluster size)
constexpr int kSmallPages = 8192;  // pool that one CTA's shared memory holds the counts of
constexpr int kPer = kSmallPages / kMeta;  // pages of a thread in one step over them
constexpr int kCopyThreads = 512;
constexpr int kCopyVecs = 4;      // 16-byte vectors in flight per thread
constexpr int kCopyCtas = 64;     // CTAs to an SM, of which four run at once

// ------------------------------------------------------------------ copies --

// Moves list[i]: page src[i] -> dst[i] of every plane, for i < *count (or
// count_max where count is NULL). Units are pieces of kCopyThreads * kCopyVecs
// vectors of one page of one plane; a CTA takes every gridDim.x-th. The lists and
// the count may be the work of the kernel before, which still runs when this one
// starts: they are read after the wait, and not as data that never changes.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(V* cache, int64_t planes, int64_t num_pages,
                                                            int64_t page_vecs, const int32_t* src, const int32_t* dst,
                                                            int64_t count_max, const int32_t* count, int pieces) {
  pdl_wait();
  const int64_t n = count ? min(static_cast<int64_t>(*count), count_max) : count_max;
  const int64_t units = n * planes * pieces;
  constexpr int kPiece = kCopyThreads * kCopyVecs;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t m = u / pieces;
    const int piece = static_cast<int>(u - m * pieces);
    const int64_t plane = m / n, i = m - plane * n;
    const int64_t a = src[i], b = dst[i];
    if (a < 0 || a >= num_pages || b < 0 || b >= num_pages) continue;
    const V* from = cache + (plane * num_pages + a) * page_vecs;
    V* to = cache + (plane * num_pages + b) * page_vecs;
    const int64_t v0 = static_cast<int64_t>(piece) * kPiece + threadIdx.x;
    V x[kCopyVecs];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k)
      if (v0 + k * kCopyThreads < page_vecs) x[k] = from[v0 + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k)
      if (v0 + k * kCopyThreads < page_vecs) to[v0 + k * kCopyThreads] = x[k];
  }
}

template <typename V>
cudaError_t copy_t(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                   const int32_t* dst, int64_t count_max, const int32_t* count, int num_sms, bool pdl,
                   cudaStream_t s) {
  const int64_t vecs = page_bytes / static_cast<int64_t>(sizeof(V));
  const int pieces = static_cast<int>((vecs + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs));
  const int64_t units = count_max * planes * pieces;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, static_cast<int64_t>(num_sms) * kCopyCtas));
  if (!pdl) {
    copy_kernel<V><<<grid, kCopyThreads, 0, s>>>(static_cast<V*>(cache), planes, num_pages, vecs, src, dst, count_max,
                                                 count, pieces);
    return cudaGetLastError();
  }
  return launch_pdl(copy_kernel<V>, dim3(grid), dim3(kCopyThreads), 0, s, 1, static_cast<V*>(cache), planes, num_pages,
                    vecs, src, dst, count_max, count, pieces);
}

// The widest vectors that pool and page allow.
cudaError_t copy_any(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                     const int32_t* dst, int64_t count_max, const int32_t* count, int num_sms, bool pdl,
                     cudaStream_t s) {
  if (count_max == 0 || planes == 0) return cudaSuccess;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(cache) | static_cast<uintptr_t>(page_bytes);
  if (bits % 16 == 0)
    return copy_t<uint4>(cache, planes, num_pages, page_bytes, src, dst, count_max, count, num_sms, pdl, s);
  if (bits % 4 == 0)
    return copy_t<uint32_t>(cache, planes, num_pages, page_bytes, src, dst, count_max, count, num_sms, pdl, s);
  return copy_t<uint8_t>(cache, planes, num_pages, page_bytes, src, dst, count_max, count, num_sms, pdl, s);
}

// ------------------------------------------------------------------ tables --

struct PagesArgs {
  const int32_t *table, *lens, *refs;
  int32_t *table_out, *lens_out, *refs_out;
  int64_t num_pages, table_stride;
  int seqs, width, page;
};

__device__ __forceinline__ int pages_for(int tokens, int page) {
  return tokens <= 0 ? 0 : (tokens - 1) / page + 1;
}
// Entries of sequence s that its length uses.
__device__ __forceinline__ int used_of(const PagesArgs& a, int s) {
  return min(pages_for(a.lens[s], a.page), a.width);
}
__device__ __forceinline__ bool in_pool(const PagesArgs& a, int p) { return p >= 0 && p < a.num_pages; }

// All threads of the cluster, as one row of them.
struct Team {
  int tid, threads, warp, warps, lane, rank, ctas;
  __device__ Team() {
    rank = blockIdx.x;  // one cluster to a grid
    ctas = gridDim.x;
    tid = rank * kMeta + threadIdx.x;
    threads = ctas * kMeta;
    warp = tid >> 5;
    warps = threads >> 5;
    lane = tid & 31;
  }
  // Global-memory writes before it are visible to the whole team after it.
  __device__ void sync() const {
    __threadfence();
    if (ctas == 1) {
      __syncthreads();
    } else {
      cluster_sync_all();
    }
  }
};

// Exclusive prefix of v over the CTA's threads; total in *sum. `red`: 33 ints.
__device__ __forceinline__ int block_prefix(int v, int* red, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = red[lane];
    int z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    red[lane] = z - w;
    if (lane == 31) red[32] = z;
  }
  __syncthreads();
  const int before = red[warp] + x - v;
  *sum = red[32];
  __syncthreads();
  return before;
}

// By one CTA: the lowest `want` free pages of refs, in order, to free_list.
// Returns how many there are. Eight pages to a thread and step; it stops at the
// step that has enough.
__device__ __forceinline__ int list_free(const int32_t* refs, int64_t num_pages, int want, int32_t* free_list, int* red) {
  int found = 0;
  for (int64_t base = 0; base < num_pages && found < want; base += kMeta * kPer) {
    const int64_t p0 = base + static_cast<int64_t>(threadIdx.x) * kPer;
    unsigned free_bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (p0 + k < num_pages && __ldcg(refs + p0 + k) <= 0) free_bits |= 1u << k;
    int sum;
    int at = found + block_prefix(__popc(free_bits), red, &sum);
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (free_bits >> k & 1) {
        if (at < want) free_list[at] = static_cast<int32_t>(p0 + k);
        ++at;
      }
    found += sum;
  }
  return min(found, want);
}

// Fork. Workspace: need (children), src, dst, free (children each).
__global__ void __launch_bounds__(kMeta) fork_kernel(PagesArgs a, const int32_t* __restrict__ parents, int children,
                                                     int32_t* missing, int32_t* need, int32_t* src, int32_t* dst,
                                                     int32_t* free_list) {
  __shared__ int red[33];
  const Team t;
  pdl_trigger();
  for (int64_t p = t.tid; p < a.num_pages; p += t.threads) a.refs_out[p] = a.refs[p];
  t.sync();
  // the old sequences' counts go, the new ones' come; a copied last page is left out for now
  for (int s = t.warp; s < a.seqs; s += t.warps)
    for (int i = t.lane, u = used_of(a, s); i < u; i += 32) {
      const int p = a.table[s * a.table_stride + i];
      if (in_pool(a, p)) atomicAdd(a.refs_out + p, -1);
    }
  for (int c = t.warp; c < children; c += t.warps) {
    const int par = parents[c];
    const bool some = par >= 0 && par < a.seqs;
    bool again = false;  // an earlier child has the same parent
    if (some)
      for (int j0 = 0; j0 < c && !again; j0 += 32)
        again = __any_sync(0xffffffffu, j0 + t.lane < c && parents[j0 + t.lane] == par);
    const int64_t cap = static_cast<int64_t>(a.width) * a.page;
    const int len = some ? max(0, static_cast<int>(min(static_cast<int64_t>(a.lens[par]), cap))) : 0;
    const int u = pages_for(len, a.page);
    const bool copy = again && len % a.page != 0;
    for (int i = t.lane; i < a.width; i += 32) {
      int p = i < u ? a.table[par * a.table_stride + i] : -1;
      if (!in_pool(a, p)) p = -1;
      if (copy && i == u - 1) {
        src[c] = p;
        p = -1;
      }
      if (p >= 0) atomicAdd(a.refs_out + p, 1);
      a.table_out[static_cast<int64_t>(c) * a.width + i] = p;
    }
    if (t.lane == 0) {
      a.lens_out[c] = len;
      need[c] = copy;
      if (!copy) src[c] = -1;
    }
  }
  t.sync();
  if (t.rank != 0) return;
  // one CTA: children that need a page, in order, meet the free pages, in order
  int want = 0;
  for (int c0 = 0; c0 < children; c0 += kMeta) {
    const int c = c0 + threadIdx.x;
    const int v = c < children && __ldcg(need + c) && __ldcg(src + c) >= 0;
    int sum;
    const int at = want + block_prefix(v, red, &sum);
    if (c < children) need[c] = v ? at : -1;
    want += sum;
  }
  const int got = list_free(a.refs_out, a.num_pages, want, free_list, red);
  __syncthreads();
  for (int c = threadIdx.x; c < children; c += kMeta) {
    const int at = need[c];
    int to = -1;
    if (at >= 0 && at < got) {
      to = free_list[at];
      a.refs_out[to] = 1;
      a.table_out[static_cast<int64_t>(c) * a.width + pages_for(a.lens_out[c], a.page) - 1] = to;
    }
    dst[c] = to;
  }
  if (threadIdx.x == 0) *missing = want - got;
}

// Length of a sequence of `old` tokens with `more` new ones, within what a length can be.
__device__ __forceinline__ int64_t grown(int old, int more) {
  return min(static_cast<int64_t>(old) + max(0, more), static_cast<int64_t>(INT32_MAX));
}

// Extend. Workspace: need (seqs), free (num_pages).
__global__ void __launch_bounds__(kMeta) extend_kernel(PagesArgs a, const int32_t* __restrict__ new_tokens,
                                                       int32_t* missing, int32_t* need, int32_t* free_list) {
  __shared__ int red[33];
  __shared__ int s_got;
  __shared__ unsigned long long s_lost;
  const Team t;
  for (int64_t p = t.tid; p < a.num_pages; p += t.threads) a.refs_out[p] = a.refs[p];
  for (int s = t.warp; s < a.seqs; s += t.warps) {
    const int u = used_of(a, s);
    for (int i = t.lane; i < a.width; i += 32) {
      const int p = i < u ? a.table[s * a.table_stride + i] : -1;
      a.table_out[static_cast<int64_t>(s) * a.width + i] = in_pool(a, p) ? p : -1;
    }
  }
  t.sync();
  if (t.rank != 0) return;
  if (threadIdx.x == 0) s_lost = 0;
  // first entry of the free list for every sequence, in order
  int64_t total = 0;
  __syncthreads();
  for (int s0 = 0; s0 < a.seqs; s0 += kMeta) {
    const int s = s0 + threadIdx.x;
    int more = 0;
    if (s < a.seqs) {
      const int old = max(0, a.lens[s]);
      const int64_t len = grown(old, new_tokens[s]);
      const int64_t to = len == 0 ? 0 : (len - 1) / a.page + 1;
      const int room = a.width - used_of(a, s);
      const int64_t grow = to - pages_for(old, a.page);
      more = static_cast<int>(min(grow, static_cast<int64_t>(max(0, room))));
      if (grow > more) atomicAdd(&s_lost, static_cast<unsigned long long>(grow - more));
    }
    int sum;
    const int at = block_prefix(more, red, &sum);
    if (s < a.seqs) need[s] = static_cast<int32_t>(min(total + at, static_cast<int64_t>(INT32_MAX)));
    total += sum;
  }
  const int want = static_cast<int>(min(total, a.num_pages));
  const int got = list_free(a.refs_out, a.num_pages, want, free_list, red);
  if (threadIdx.x == 0) s_got = got;
  __syncthreads();
  for (int s = threadIdx.x >> 5; s < a.seqs; s += kMeta / 32) {
    const int first = need[s], u = used_of(a, s);
    const int old = max(0, a.lens[s]);
    const int64_t len = grown(old, new_tokens[s]);
    const int64_t to = len == 0 ? 0 : (len - 1) / a.page + 1;
    const int more = static_cast<int>(min(to - pages_for(old, a.page), static_cast<int64_t>(max(0, a.width - u))));
    const int have = max(0, min(more, s_got - first));
    for (int i = t.lane; i < have; i += 32) {
      const int p = free_list[first + i];
      a.refs_out[p] = 1;
      a.table_out[static_cast<int64_t>(s) * a.width + u + i] = p;
    }
    if (t.lane == 0) a.lens_out[s] = static_cast<int32_t>(min(len, static_cast<int64_t>(u + have) * a.page));
  }
  if (threadIdx.x == 0) {
    const int64_t lost = total - got + static_cast<int64_t>(s_lost);
    *missing = static_cast<int32_t>(min(lost, static_cast<int64_t>(INT32_MAX)));
  }
}

__global__ void __launch_bounds__(kMeta) release_kernel(PagesArgs a, const uint8_t* __restrict__ drop) {
  const Team t;
  for (int64_t p = t.tid; p < a.num_pages; p += t.threads) a.refs_out[p] = a.refs[p];
  t.sync();
  for (int s = t.warp; s < a.seqs; s += t.warps) {
    const bool gone = drop[s] != 0;
    const int u = used_of(a, s);
    for (int i = t.lane; i < a.width; i += 32) {
      int p = i < u ? a.table[s * a.table_stride + i] : -1;
      if (!in_pool(a, p)) p = -1;
      if (gone && p >= 0) atomicAdd(a.refs_out + p, -1);
      a.table_out[static_cast<int64_t>(s) * a.width + i] = gone ? -1 : p;
    }
    if (t.lane == 0) a.lens_out[s] = gone ? 0 : a.lens[s];
  }
}

// Compact. Workspace: counts (3 * kMaxCluster), src and dst (num_pages/2 + 1
// each), number of moves.
__global__ void __launch_bounds__(kMeta) compact_kernel(PagesArgs a, int32_t* remap, int32_t* live, int32_t* counts,
                                                        int32_t* src, int32_t* dst, int32_t* moves) {
  __shared__ int red[33];
  const Team t;
  pdl_trigger();
  // a CTA's share of the pages: whole steps of kMeta * kPer
  const int64_t steps = (a.num_pages + kMeta * kPer - 1) / (kMeta * kPer);
  const int64_t per = (steps + t.ctas - 1) / t.ctas;
  const int64_t lo = min(t.rank * per, steps) * kMeta * kPer, hi = min(min((t.rank + 1) * per, steps) * kMeta * kPer, a.num_pages);
  const auto live_bits = [&](int64_t p0) {
    unsigned b = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (p0 + k < hi && a.refs[p0 + k] > 0) b |= 1u << k;
    return b;
  };
  int n_live = 0, sum;
  {
    int mine = 0;
    for (int64_t p0 = lo + threadIdx.x * kPer; p0 < hi; p0 += kMeta * kPer) mine += __popc(live_bits(p0));
    block_prefix(mine, red, &sum);
    if (threadIdx.x == 0) counts[t.rank] = sum;
  }
  t.sync();
  for (int r = 0; r < t.ctas; ++r) n_live += __ldcg(counts + r);
  // pages before the end of the compact pool that are free, and pages behind it that are live
  const auto split = [&](int64_t p0, unsigned b, unsigned* hole, unsigned* mover) {
    unsigned before = 0, within = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (p0 + k < n_live) before |= 1u << k;
      if (p0 + k < hi) within |= 1u << k;
    }
    *hole = ~b & before & within;
    *mover = b & ~before & within;
  };
  {
    int h = 0, m = 0;
    for (int64_t p0 = lo + threadIdx.x * kPer; p0 < hi; p0 += kMeta * kPer) {
      unsigned hole, mover;
      split(p0, live_bits(p0), &hole, &mover);
      h += __popc(hole);
      m += __popc(mover);
    }
    block_prefix(h, red, &sum);
    if (threadIdx.x == 0) counts[kMaxCluster + t.rank] = sum;
    block_prefix(m, red, &sum);
    if (threadIdx.x == 0) counts[2 * kMaxCluster + t.rank] = sum;
  }
  t.sync();
  int holes = 0, movers = 0, all = 0;
  for (int r = 0; r < t.ctas; ++r) {
    if (r < t.rank) {
      holes += __ldcg(counts + kMaxCluster + r);
      movers += __ldcg(counts + 2 * kMaxCluster + r);
    }
    all += __ldcg(counts + 2 * kMaxCluster + r);
  }
  for (int64_t base = lo; base < hi; base += kMeta * kPer) {
    const int64_t p0 = base + threadIdx.x * kPer;
    unsigned hole, mover;
    const unsigned b = live_bits(p0);
    split(p0, b, &hole, &mover);
    int ah = holes + block_prefix(__popc(hole), red, &sum);
    holes += sum;
    int am = movers + block_prefix(__popc(mover), red, &sum);
    movers += sum;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (p0 + k >= hi) break;
      const int p = static_cast<int>(p0 + k);
      if (hole >> k & 1) dst[ah++] = p;
      if (mover >> k & 1) src[am++] = p;
      // (a hole's count is written when its page is known)
      if (!(hole >> k & 1)) a.refs_out[p] = p < n_live ? a.refs[p] : 0;
      if (!(mover >> k & 1)) remap[p] = b >> k & 1 ? p : -1;
    }
  }
  t.sync();
  for (int i = t.tid; i < all; i += t.threads) {
    const int from = __ldcg(src + i), to = __ldcg(dst + i);
    remap[from] = to;
    a.refs_out[to] = a.refs[from];
  }
  if (t.tid == 0) {
    *moves = all;
    *live = n_live;
  }
  t.sync();
  for (int s = t.warp; s < a.seqs; s += t.warps)
    for (int i = t.lane, u = used_of(a, s); i < a.width; i += 32) {
      const int p = i < u ? a.table[s * a.table_stride + i] : -1;
      a.table_out[static_cast<int64_t>(s) * a.width + i] = in_pool(a, p) ? __ldcg(remap + p) : -1;
    }
}

// ------------------------------------------- small pools, in shared memory --
//
// Up to kSmallPages pages, one CTA: counts, lists and the map of pages live in
// shared memory, so that the phases are apart by a CTA barrier where those
// above send every count through the L2. (16 beams over 1021 pages: 5 us where
// fork_kernel takes 10; 24 sequences over 1501 pages: 6 us where compact_kernel
// takes 14.)

// A thread has the pages threadIdx.x + k * kMeta.

// Exclusive prefix over the kPer * 32 entries of `counts` (of page blocks (k,
// warp), in page order), by warp 0, in place; the total to *sum. Two numbers
// below 2^15 may share an entry.
__device__ __forceinline__ void scan_blocks(int* counts, int* sum) {
  if (threadIdx.x < 32) {
    int v[kPer], s = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      v[i] = s;
      s += counts[threadIdx.x * kPer + i];
    }
    int x = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (static_cast<int>(threadIdx.x) >= o) x += y;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) counts[threadIdx.x * kPer + i] = v[i] + x - s;
    if (threadIdx.x == 31) *sum = x;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kMeta) compact_small_kernel(PagesArgs a, int32_t* remap, int32_t* live, int32_t* src,
                                                              int32_t* dst, int32_t* moves) {
  extern __shared__ __align__(16) int32_t s_remap[];  // kSmallPages, then the lists
  int32_t* s_src = s_remap + kSmallPages;
  int32_t* s_dst = s_src + kSmallPages / 2;
  __shared__ int counts[kPer * 32];
  __shared__ int total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pages = static_cast<int>(a.num_pages);
  pdl_trigger();
  int refs[kPer];
  unsigned alive[kPer], hole[kPer], mover[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int p = k * kMeta + tid;
    refs[k] = p < pages ? a.refs[p] : 0;
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    alive[k] = __ballot_sync(0xffffffffu, refs[k] > 0);
    if (lane == 0) counts[k * 32 + warp] = __popc(alive[k]);
  }
  __syncthreads();
  scan_blocks(counts, &total);
  const int n = total;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int p = k * kMeta + tid;
    hole[k] = __ballot_sync(0xffffffffu, p < n && refs[k] <= 0);
    mover[k] = __ballot_sync(0xffffffffu, p >= n && refs[k] > 0);
    if (lane == 0) counts[k * 32 + warp] = __popc(hole[k]) | __popc(mover[k]) << 16;
  }
  __syncthreads();
  scan_blocks(counts, &total);
  const int all = total & 0xffff;
  const unsigned below = (1u << lane) - 1;
  const auto hole_at = [&](int k) { return (counts[k * 32 + warp] & 0xffff) + __popc(hole[k] & below); };
  const auto mover_at = [&](int k) { return (counts[k * 32 + warp] >> 16) + __popc(mover[k] & below); };
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int p = k * kMeta + tid;
    if (hole[k] >> lane & 1) s_dst[hole_at(k)] = p;
    if (mover[k] >> lane & 1) s_src[mover_at(k)] = p;
  }
  __syncthreads();
  for (int i = tid; i < all; i += kMeta) {
    src[i] = s_src[i];
    dst[i] = s_dst[i];
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int p = k * kMeta + tid;
    if (p >= pages) continue;
    const int to = mover[k] >> lane & 1 ? s_dst[mover_at(k)] : refs[k] > 0 ? p : -1;
    remap[p] = to;
    s_remap[p] = to;
    a.refs_out[p] = p >= n ? 0 : hole[k] >> lane & 1 ? a.refs[s_src[hole_at(k)]] : refs[k];
  }
  if (tid == 0) {
    *moves = all;
    *live = n;
  }
  __syncthreads();
  for (int s = warp; s < a.seqs; s += kMeta / 32)
    for (int i = lane, u = used_of(a, s); i < a.width; i += 32) {
      const int p = i < u ? a.table[s * a.table_stride + i] : -1;
      a.table_out[static_cast<int64_t>(s) * a.width + i] = in_pool(a, p) ? s_remap[p] : -1;
    }
}

// At most kMeta children of at most kMeta sequences. Workspace: src, dst.
__global__ void __launch_bounds__(kMeta) fork_small_kernel(PagesArgs a, const int32_t* __restrict__ parents, int children,
                                                           int32_t* missing, int32_t* src, int32_t* dst) {
  extern __shared__ __align__(16) int32_t s_refs[];  // kSmallPages
  __shared__ int counts[kPer * 32], red[33];
  __shared__ int s_first[kMeta];    // first child of each sequence
  __shared__ int s_free[kMeta];     // lowest free pages
  __shared__ int s_from[kMeta];     // page that a child copies, -1: none
  __shared__ int total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, pages = static_cast<int>(a.num_pages);
  pdl_trigger();
  const int par = tid < children ? parents[tid] : -1;
  const bool some = par >= 0 && par < a.seqs;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int p = k * kMeta + tid;
    if (p < pages) s_refs[p] = a.refs[p];
  }
  s_first[tid] = INT32_MAX;
  s_from[tid] = -1;
  __syncthreads();
  if (some) atomicMin(&s_first[par], tid);
  for (int s = warp; s < a.seqs; s += kMeta / 32)
    for (int i = lane, u = used_of(a, s); i < u; i += 32) {
      const int p = a.table[s * a.table_stride + i];
      if (in_pool(a, p)) atomicAdd(&s_refs[p], -1);
    }
  __syncthreads();
  const int64_t cap = static_cast<int64_t>(a.width) * a.page;
  for (int c = warp; c < children; c += kMeta / 32) {
    const int q = parents[c];
    const bool known = q >= 0 && q < a.seqs;
    const int len = known ? max(0, static_cast<int>(min(static_cast<int64_t>(a.lens[q]), cap))) : 0;
    const int u = pages_for(len, a.page);
    const bool copy = known && s_first[q] != c && len % a.page != 0;
    for (int i = lane; i < a.width; i += 32) {
      int p = i < u ? a.table[q * a.table_stride + i] : -1;
      if (!in_pool(a, p)) p = -1;
      if (copy && i == u - 1) {
        s_from[c] = p;
        p = -1;
      }
      if (p >= 0) atomicAdd(&s_refs[p], 1);
      a.table_out[static_cast<int64_t>(c) * a.width + i] = p;
    }
    if (lane == 0) a.lens_out[c] = len;
  }
  __syncthreads();
  // children that need a page, in order, meet the free pages, in order
  unsigned open[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int p = k * kMeta + tid;
    open[k] = __ballot_sync(0xffffffffu, p < pages && s_refs[p] <= 0);
    if (lane == 0) counts[k * 32 + warp] = __popc(open[k]);
  }
  const int from = tid < children ? s_from[tid] : -1;
  int want;
  const int at = block_prefix(from >= 0, red, &want);
  scan_blocks(counts, &total);
  const int got = min(want, total);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = counts[k * 32 + warp] + __popc(open[k] & ((1u << lane) - 1));
    if ((open[k] >> lane & 1) && r < got) s_free[r] = k * kMeta + tid;
  }
  __syncthreads();
  if (tid < children) {
    const int to = from >= 0 && at < got ? s_free[at] : -1;
    src[tid] = from;
    dst[tid] = to;
    if (to >= 0) {
      s_refs[to] = 1;
      const int len = static_cast<int>(min(static_cast<int64_t>(a.lens[par]), cap));
      a.table_out[static_cast<int64_t>(tid) * a.width + pages_for(len, a.page) - 1] = to;
    }
  }
  if (tid == 0) *missing = want - got;
  __syncthreads();
  for (int p = tid; p < pages; p += kMeta) a.refs_out[p] = s_refs[p];
}

PagesArgs args_of(const hc_pages_t& p) {
  return PagesArgs{p.page_table, p.lens, p.refs, p.page_table_out, p.lens_out, p.refs_out, p.num_pages, p.table_stride,
                   p.seqs, p.max_pages, p.page_size};
}

// CTAs of a table kernel: one for small pools (a CTA barrier costs less than a
// cluster's), else enough for 16 table entries or pages to a thread.
unsigned meta_ctas(int64_t num_pages, int64_t entries) {
  const int64_t per = static_cast<int64_t>(kMeta) * 16;
  const int64_t want = (num_pages + entries + per - 1) / per;
  unsigned n = 1;
  while (n < kMaxCluster && n < want) n *= 2;
  return n;
}

// Whether one CTA with everything in shared memory serves a pool: as many pages
// as that holds, and few enough table entries (64 to a thread) that a cluster's
// further CTAs would not pay for its barriers.
bool small_pool(int64_t num_pages, int64_t entries) { return num_pages <= kSmallPages && entries <= kMeta * 64; }

template <typename... KArgs, typename... Args>
cudaError_t launch_meta(void (*kernel)(KArgs...), unsigned ctas, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kMeta);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace

// 4 lists of `seqs` (fork) or one of seqs and one of pages (extend), or two of
// half the pages (compact), and the small counters.
size_t pages_workspace(int64_t num_pages, int32_t seqs) {
  return align_up((256 + 4 * static_cast<size_t>(seqs) + static_cast<size_t>(num_pages) + 8) * 4, 256);
}

cudaError_t launch_page_copy(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                             const int32_t* dst, int64_t count, int num_sms, cudaStream_t s) {
  return copy_any(cache, planes, num_pages, page_bytes, src, dst, count, nullptr, num_sms, false, s);
}

cudaError_t launch_page_fork(const hc_pages_t& p, const int32_t* parents, int32_t children, int32_t* missing,
                             void* cache, int64_t planes, int64_t page_bytes, void* ws, int num_sms, cudaStream_t s) {
  int32_t* w = static_cast<int32_t*>(ws);
  int32_t *need = w, *src = w + children, *dst = w + 2 * static_cast<int64_t>(children),
          *free_list = w + 3 * static_cast<int64_t>(children);
  const int64_t entries = static_cast<int64_t>(p.seqs + children) * p.max_pages;
  cudaError_t e;
  if (small_pool(p.num_pages, entries) && children <= kMeta && p.seqs <= kMeta) {
    constexpr size_t smem = kSmallPages * 4;
    e = ensure_smem<fork_small_kernel>(smem);
    if (e == cudaSuccess) e = launch_meta(fork_small_kernel, 1, smem, s, args_of(p), parents, children, missing, src, dst);
  } else {
    e = launch_meta(fork_kernel, meta_ctas(p.num_pages, entries), 0, s, args_of(p), parents, children, missing, need, src,
                    dst, free_list);
  }
  if (e != cudaSuccess) return e;
  return copy_any(cache, planes, p.num_pages, page_bytes, src, dst, children, nullptr, num_sms, true, s);
}

cudaError_t launch_page_extend(const hc_pages_t& p, const int32_t* new_tokens, int32_t* missing, void* ws,
                               int num_sms, cudaStream_t s) {
  (void)num_sms;
  int32_t* w = static_cast<int32_t*>(ws);
  const unsigned ctas = meta_ctas(p.num_pages, static_cast<int64_t>(p.seqs) * p.max_pages);
  return launch_meta(extend_kernel, ctas, 0, s, args_of(p), new_tokens, missing, w, w + p.seqs);
}

cudaError_t launch_page_release(const hc_pages_t& p, const uint8_t* drop, int num_sms, cudaStream_t s) {
  (void)num_sms;
  const unsigned ctas = meta_ctas(p.num_pages, static_cast<int64_t>(p.seqs) * p.max_pages);
  return launch_meta(release_kernel, ctas, 0, s, args_of(p), drop);
}

cudaError_t launch_page_compact(const hc_pages_t& p, int32_t* remap, int32_t* live, void* cache, int64_t planes,
                                int64_t page_bytes, void* ws, int num_sms, cudaStream_t s) {
  int32_t* w = static_cast<int32_t*>(ws);
  const int64_t most = p.num_pages / 2 + 1;  // moves: holes and movers are disjoint
  int32_t *counts = w, *moves = w + 64, *src = w + 128, *dst = src + most;
  const int64_t entries = static_cast<int64_t>(p.seqs) * p.max_pages;
  cudaError_t e;
  if (small_pool(p.num_pages, entries)) {
    constexpr size_t smem = 2 * kSmallPages * 4;
    e = ensure_smem<compact_small_kernel>(smem);
    if (e == cudaSuccess) e = launch_meta(compact_small_kernel, 1, smem, s, args_of(p), remap, live, src, dst, moves);
  } else {
    e = launch_meta(compact_kernel, meta_ctas(p.num_pages, entries), 0, s, args_of(p), remap, live, counts, src, dst, moves);
  }
  if (e != cudaSuccess) return e;
  return copy_any(cache, planes, p.num_pages, page_bytes, src, dst, p.num_pages / 2, moves, num_sms, true, s);
}

}  // namespace hc
