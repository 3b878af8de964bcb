// Attention over a paged cache for few rows: sequences whose new
// tokens and grouped heads make at most 16 rows to a key head, single tokens
// above all.
//
// Bound: bytes. Every key and value is read once and used by at most 16 rows, 16
// multiply-adds to the byte at most, so what counts is to keep enough loads in
// flight (some 44 bytes/ns and SM, about 45 KB at a microsecond's latency).
// Each warp runs for itself: blocks of 16 keys, every fourth of the split's,
// come by 16-byte cp.async into a ring of its own, two blocks deep, so that
// no barrier stands between the loads of one warp and the arithmetic of
// another; three CTAs of four warps to an SM have up to 192 KB on their way (a
// ring of three blocks leaves room for two CTAs: 112 us where this takes 104, of
// four for one: 146). The products are warp-level MMAs (m16n8k16): a tile of 16
// rows is what they are made for, where a tcgen05 tile would be seven eighths
// empty and its tensor-memory round trips would lie on the path of every block.
//
// Measured: two contexts of 130002 and 34402 tokens, 32 heads of 128 on 8, fp16:
// 104 us, 6.5 TB/s, 97% of the measured copy bandwidth; 61 ragged contexts of up
// to 8192 in bf16: 232 us, 6.1 TB/s, 91%; one of 700, 20 heads on 4: 8.3 us, the latency
// of its chain of loads.
//
// Work: where every sequence has one new token (no cu_q) and there are too few of
// them to fill half the GPU, the kernel splits them itself, by their lengths: with
// T CTAs, two for each SM, which all run at once, and as many extra pieces as
// rounding up may make, all are cut into pieces of
//   L = sum of keys * kv_heads / (T - seqs * kv_heads)
// keys, so that they fill the GPU once, evenly, whatever the lengths are. Every
// warp works that out for itself from kv_lens, 32 sequences at a time. (Against
// pieces that the host chose by the longest, with a ring of three blocks: two
// contexts of 130002 and 34402 tokens, 8 key heads, 121 -> 112 us; one of 30002, 4
// key heads, 35 -> 21 us; eight of up to 4002, 25 -> 17 us. With more sequences
// the host's splits are as good, and 64 contexts of up to 8192 took 231 us where
// these took 240.) Contexts of up to kClusterKeys, where eight CTAs to each tile
// still run at once, go to clusters of eight, which join their sums through
// shared memory: one kernel and no workspace (one context of 700, 20 heads on 4:
// 8.6 us where pieces take 10.7, of 2002 10.6 against 12.6; of 4002 14.7 against
// 12.2).
//
// Mathematics: the running maximum and sum of a softmax, held per warp, with the
// sums of values in registers; they are rescaled only when a block raises the
// maximum. The warps' results are joined once at the end:
//   M = max_w m_w,  out = sum_w 2^(m_w - M) o_w / sum_w 2^(m_w - M) l_w.
// The product with the values takes its weights in T, the operands' type. Up to eight
// rows to a key head leave half of the MMA's sixteen free, and there goes what the
// rounding leaves of each weight: for nothing, a weight keeps twice the bits, and
// what is off in a result is its own rounding (64 contexts in bf16: 1.66e-3 against
// 64 bits, where rounded weights gave 1.95e-3; an MMA of its own for the rest would
// take 3 to 4% more time, so from nine rows on weights are rounded). The sum of
// weights is taken before.
#include <type_traits>

#include "hc_async.cuh"
#include "hc_attn.cuh"
#include "hc_attn_internal.h"
#include "hc_mma.cuh"

namespace hc {
namespace {

constexpr int kWarps = 4;
constexpr int kBlock = 16;  // keys of a block
constexpr int kStages = 2;
constexpr int kShortest = 128;  // keys that are worth a piece
constexpr int kMaxPieces = 512; // of a sequence
constexpr int kClusterKeys = 2560;  // the longest context that a cluster takes

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a pair of numbers rounded to T leaves of the two, in T again.
template <typename T>
__device__ __forceinline__ uint32_t pack2_rest(float x, float y, uint32_t packed);
template <>
__device__ __forceinline__ uint32_t pack2_rest<__half>(float x, float y, uint32_t packed) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&packed));
  return pack2<__half>(x - f.x, y - f.y);
}
template <>
__device__ __forceinline__ uint32_t pack2_rest<__nv_bfloat16>(float x, float y, uint32_t packed) {
  return pack2<__nv_bfloat16>(x - __uint_as_float(packed << 16), y - __uint_as_float(packed & 0xffff0000u));
}

// 16-byte chunk `c` of row `r` of a block of D-element rows: chunks are permuted
// by the row's low three bits, so that the eight rows of an 8x8 matrix lie in
// eight different groups of banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return static_cast<uint32_t>(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// Pieces of a batch of single tokens, one tile to a sequence.
struct Pieces {
  int len;          // keys of a piece
  int s, z;         // sequence and piece of the unit asked for; s = -1: there is no such unit
  int unit0, count; // the sequence's first unit, and its pieces
};

// Keys of a sequence's one tile, from its first block on (as tile_at has them).
__device__ __forceinline__ int64_t keys_of(const AttnArgs& a, int s) {
  const int64_t n = kv_len_of(a.b, s), lo = a.window > 0 && n > a.window ? n - a.window : 0;
  return n - (lo & -static_cast<int64_t>(a.g.align));
}
__device__ __forceinline__ int pieces_of(int64_t keys, int len) {
  return keys <= len ? 1 : static_cast<int>(quotient(keys + len - 1, len));
}

// Place of row r of a unit among the partial results.
__device__ __forceinline__ int64_t piece_row(const AttnArgs& a, int kvh, int unit, int r) {
  return (static_cast<int64_t>(kvh) * a.units + unit) * 16 + r;
}

// By a full warp: the piece that is unit `unit`, or with `seq` >= 0 the units of that sequence.
__device__ __forceinline__ Pieces find_pieces(const AttnArgs& a, int unit, int seq) {
  const int lane = threadIdx.x & 31, seqs = a.b.seqs;
  const int64_t early = lane < seqs ? keys_of(a, lane) : 0;  // of the first 32 sequences
  int64_t total = early, most = early;
  for (int s = lane + 32; s < seqs; s += 32) {
    const int64_t k = keys_of(a, s);
    total += k;
    most = k > most ? k : most;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    const int64_t other = __shfl_xor_sync(0xffffffffu, most, o);
    most = other > most ? other : most;
  }
  Pieces p;
  int64_t len = quotient(total * a.kv_heads + a.spare_ctas - 1, a.spare_ctas);
  const int64_t least = (most + kMaxPieces - 1) / kMaxPieces;
  len = len < kShortest ? kShortest : len;
  len = len < least ? least : len;
  // (2^30 keys to a piece are more than the memory of a GPU holds)
  p.len = static_cast<int>(len < (1 << 30) ? (len + kBlock - 1) / kBlock * kBlock : 1 << 30);
  int before = 0;
  p.s = -1;
  for (int s0 = 0; s0 < seqs; s0 += 32) {
    const int n = s0 + lane < seqs ? pieces_of(s0 == 0 ? early : keys_of(a, s0 + lane), p.len) : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int first = before + x - n;
    const unsigned hit = __ballot_sync(0xffffffffu, seq >= 0 ? s0 + lane == seq : unit >= first && unit < first + n);
    if (hit != 0) {
      const int at = __ffs(hit) - 1;
      p.s = s0 + at;
      p.unit0 = __shfl_sync(0xffffffffu, first, at);
      p.count = __shfl_sync(0xffffffffu, n, at);
      p.z = unit - p.unit0;
      return p;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  return p;
}

// How a sequence's keys are shared out: slots along x and splits along z
// (hc_attn.cuh); pieces of single-token sequences along x, as above; or a cluster
// of kCluster CTAs along x to each single-token sequence.
enum Share { kBySplit, kByPiece, kByCluster };
constexpr int kCluster = 8;

// What a CTA has to do: tile, split, piece or rank z, and its keys [k0, k1).
template <int SHARE>
__device__ __forceinline__ bool find_work(const AttnArgs& a, AttnTile* t, int* z, int64_t* k0, int64_t* k1) {
  if (SHARE == kByPiece) {
    const Pieces p = find_pieces(a, blockIdx.x, -1);
    if (p.s < 0) return false;
    tile_at(a, a.g, p.s, 0, t);
    t->splits = p.count;
    *z = p.z;
    *k0 = t->base + static_cast<int64_t>(p.z) * p.len;
    *k1 = p.z == p.count - 1 ? t->hi : *k0 + p.len;
    return true;
  }
  if (SHARE == kByCluster) {
    tile_at(a, a.g, blockIdx.x / kCluster, 0, t);
    *z = blockIdx.x % kCluster;
    const int64_t len = (t->hi - t->base + kCluster * kBlock - 1) / (kCluster * kBlock) * kBlock;
    *k0 = t->base + *z * len;
    *k0 = *k0 < t->hi ? *k0 : t->hi;
    *k1 = *k0 + len < t->hi ? *k0 + len : t->hi;
    return true;
  }
  tile_of_slot(a, blockIdx.x, t);
  if (t->rows == 0 || *z >= t->splits) return false;
  split_range(a.g, *t, *z, k0, k1);
  return true;
}

__device__ __forceinline__ float4 peer_load4(const void* p, int rank) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(mapa_shared(smem_addr(p), rank)));
  return x;
}
__device__ __forceinline__ float2 peer_load2(const void* p, int rank) {
  float2 x;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(x.x), "=f"(x.y)
               : "r"(mapa_shared(smem_addr(p), rank)));
  return x;
}

// Floats of shared memory for a tile's sums on their way out: each warp's, and, in a cluster, the CTA's with its maxima and sums
// of weights.
template <int D>
constexpr int sum_floats(bool cluster) {
  return kWarps * 16 * (D + 8) + (cluster ? 16 * D + 32 : 0);
}

// Joins the warps' sums `all` ([warp][16 rows][D + 8], each scaled to the largest
// maximum) of a tile's rows, and writes them as partial results or as the result.
// The CTAs of a cluster join theirs through one another's shared memory, each for
// its share of the rows' features.
template <typename T, int D, int SHARE>
__device__ __forceinline__ void write_rows(const AttnArgs& a, const AttnTile& t, int z, int kvh, float* all,
                                           const float (*s_m)[16], const float (*s_l)[16]) {
  constexpr int kPitch = D + 8;
  constexpr int kPerRow = D / 4;  // threads of a row, four features each
  const auto write = [&](int r, int d, float4 x, float top, float sum) {
    int64_t token;
    int head;
    row_owner(a, t, kvh, r, &token, &head);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    T* dst = static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs + d;
    stf(dst, x.x * inv);
    stf(dst + 1, x.y * inv);
    stf(dst + 2, x.z * inv);
    stf(dst + 3, x.w * inv);
    if (d == 0 && a.lse) a.lse[token * a.heads + head] = sum == 0.0f ? neg_inf() : top * kLn2 + logf(sum);
  };
  float* const cta_sums = all + kWarps * 16 * kPitch;
  float2* const cta_ml = reinterpret_cast<float2*>(cta_sums + 16 * D);
  for (int u = threadIdx.x; u < t.rows * kPerRow; u += kWarps * 32) {
    const int r = u / kPerRow, d = (u - r * kPerRow) * 4;
    float top = neg_inf(), sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_l[w][r] * (s_m[w][r] == neg_inf() ? 1.0f : exp2f(s_m[w][r] - top));
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(all + (w * 16 + r) * kPitch + d);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    if (SHARE == kByCluster) {
      *reinterpret_cast<float4*>(cta_sums + r * D + d) = x;
      if (d == 0) cta_ml[r] = make_float2(top, sum);
    } else if (t.splits > 1) {
      int64_t at;
      if (SHARE == kByPiece) {
        at = piece_row(a, kvh, blockIdx.x, r);
      } else {
        int64_t token;
        int head;
        row_owner(a, t, kvh, r, &token, &head);
        at = part_index(a, z, token, head);
      }
      *reinterpret_cast<float4*>(a.part_o + at * D + d) = x;
      if (d == 0) a.part_ml[at] = make_float2(top, sum);
    } else {
      write(r, d, x, top, sum);
    }
  }
  if (SHARE == kByCluster) {
    cluster_sync_all();
    for (int u = z * kWarps * 32 + threadIdx.x; u < t.rows * kPerRow; u += kCluster * kWarps * 32) {
      const int r = u / kPerRow, d = (u - r * kPerRow) * 4;
      float2 ml[kCluster];
      float4 y[kCluster];
#pragma unroll
      for (int k = 0; k < kCluster; ++k) {
        ml[k] = peer_load2(cta_ml + r, k);
        y[k] = peer_load4(cta_sums + r * D + d, k);
      }
      float top = neg_inf(), sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kCluster; ++k) top = fmaxf(top, ml[k].x);
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kCluster; ++k) {
        // (no weights: sums of zero, or NaN from NaN scores)
        const float w = ml[k].x == neg_inf() ? 1.0f : exp2f(ml[k].x - top);
        sum += ml[k].y * w;
        x.x = fmaf(y[k].x, w, x.x);
        x.y = fmaf(y[k].y, w, x.y);
        x.z = fmaf(y[k].z, w, x.z);
        x.w = fmaf(y[k].w, w, x.w);
      }
      write(r, d, x, top, sum);
    }
    cluster_sync_all();  // (no CTA leaves while another reads its memory)
  }
}

template <typename T, int D, int SHARE>
__global__ void __launch_bounds__(kWarps * 32, 3) rows_kernel(AttnArgs a) {
  constexpr int kChunks = D / 8;                 // 16-byte chunks of a row
  constexpr int kHalf = kBlock * D * 2;          // bytes of a block's keys
  constexpr int kStage = 2 * kHalf;              // and of its values
  constexpr int kRowsPer = 32 / kChunks;         // rows that a warp copies at once
  constexpr int kCopies = kBlock / kRowsPer;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int kvh = blockIdx.y;
  int z = blockIdx.z;
  pdl_trigger();
  if (SHARE == kBySplit && a.clears && blockIdx.x == gridDim.x - 1) clear_unowned<T>(a, z * gridDim.y + kvh, gridDim.y * gridDim.z);
  AttnTile t;
  int64_t k0, k1;
  if (!find_work<SHARE>(a, &t, &z, &k0, &k1)) return;
  const T* kp = static_cast<const T*>(a.k) + kvh * a.c_hs;
  const T* vp = static_cast<const T*>(a.v) + kvh * a.c_hs;
  const int blocks = k1 > k0 ? static_cast<int>((k1 - k0 + kBlock - 1) / kBlock) : 0;
  const uint32_t base = smem_addr(ring) + warp * (kStages * kStage);

  // place of key (lane & 15) of block b in the pool, -1: no such key
  const auto place_of = [&](int b) -> int64_t {
    const int64_t j = k0 + static_cast<int64_t>(b) * kBlock + (lane & 15);
    if (b >= blocks || j < t.lo || j >= k1) return -1;
    const uint32_t i = static_cast<uint32_t>(j) / static_cast<uint32_t>(a.b.page_size);
    const int page = page_of(a.b, t.s, i);
    return page < 0 ? -1 : page * a.c_ps + (static_cast<uint32_t>(j) - i * a.b.page_size) * a.c_ts;
  };
  const auto fetch = [&](int64_t place, int stage) {
    const uint32_t to = base + stage * kStage;
    const int c = lane % kChunks;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int r = i * kRowsPer + lane / kChunks;
      const int64_t at = __shfl_sync(0xffffffffu, place, r);
      const int64_t off = (at < 0 ? 0 : at) + c * 8;
      const uint32_t bytes = at < 0 ? 0 : 16;
      cp_async16_zfill(to + chunk_at<D>(r, c), kp + off, bytes);
      cp_async16_zfill(to + kHalf + chunk_at<D>(r, c), vp + off, bytes);
    }
  };

  // the ring's first blocks, then the queries while those are on their way
  int64_t place = place_of(warp);
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    const int b = warp + i * kWarps;
    const int64_t next = place_of(b + kWarps);
    if (b < blocks) fetch(place, i);
    cp_async_commit();
    place = next;
  }
  uint32_t qf[D / 16][4];
  {
    const T* rows[2] = {nullptr, nullptr};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (g + 8 * i < t.rows) {
        int64_t token;
        int head;
        row_owner(a, t, kvh, g + 8 * i, &token, &head);
        rows[i] = static_cast<const T*>(a.q) + token * a.q_ts + head * a.q_hs;
      }
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const T* src = rows[i & 1];
        qf[ks][i] = src ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + (i >> 1) * 8 + q4 * 2) : 0u;
      }
  }
  // keys that this thread's two rows see, relative to k0: [from, to)
  int from[2], to[2], all_from = 0, all_to = 0;
  const auto rel = [&](int64_t j) {
    const int64_t d = j - k0, n = k1 - k0;
    return static_cast<int>(d < 0 ? 0 : d > n ? n : d);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t p = row_position(t, t.row0 + g + 8 * i, a.group);
    const bool real = g + 8 * i < t.rows;
    to[i] = real ? rel(p + 1) : 0;
    from[i] = real && a.window > 0 ? rel(p - a.window + 1) : 0;
  }
  all_to = rel(row_position(t, t.row0, a.group) + 1);  // seen by every row: [all_from, all_to)
  if (a.window > 0) all_from = rel(row_position(t, t.row0 + t.rows - 1, a.group) - a.window + 1);
  const bool uneven = row_position(t, t.row0, a.group) != row_position(t, t.row0 + t.rows - 1, a.group);

  // Up to eight rows leave the upper half of the product's tile free for what rounding to T leaves of their weights.
  const bool spare = t.rows <= 8;
  const ScoreMap map = score_map(a.scale, a.softcap);
  float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.0f, 0.0f};
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;

  int stage = 0;
  for (int b = warp; b < blocks; b += kWarps) {
    {
      const int ahead = b + (kStages - 1) * kWarps;
      const int64_t next = place_of(ahead + kWarps);
      if (ahead < blocks) fetch(place, stage == 0 ? kStages - 1 : stage - 1);
      cp_async_commit();
      place = next;
    }
    cp_async_wait_group<kStages - 1>();
    __syncwarp();
    const uint32_t ks_at = base + stage * kStage, vs_at = ks_at + kHalf;
    // scores of 16 rows and 16 keys, as two 16 x 8 tiles
    float s[2][4] = {};
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4(ks_at + chunk_at<D>(((lane >> 4) << 3) + (lane & 7), 2 * ks + ((lane >> 3) & 1)), b0, b1, b2, b3);
      Mma<T>::run4(s[0], qf[ks], b0, b1);
      Mma<T>::run4(s[1], qf[ks], b2, b3);
    }
    const int j0 = b * kBlock;
    const bool whole = j0 >= all_from && j0 + kBlock <= all_to;
    const auto map_all = [&](auto exponent) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = exponent(s[n][e]);
    };
    if (map.cap == 0.0f) {
      map_all([&](float x) { return x * map.mul; });
    } else {
      bool far = false;
      map_all([&](float x) {
        far |= cap_far(map, x);
        return x;
      });
      if (__any_sync(0xffffffffu, far)) {
        map_all([&](float x) { return map_score(map, x); });
      } else {  // (the same bits)
        map_all([&](float x) { return cap_near(map, x); });
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!whole) {
          const int j = j0 + 8 * n + 2 * q4 + (e & 1), i = e >> 1;
          if (j < from[i] || j >= to[i]) s[n][e] = neg_inf();
        }
      }
    float top[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float now = fmaxf(m[i], top[i]);
        f[i] = now == neg_inf() ? 1.0f : ex2(m[i] - now);
        m[i] = now;
        l[i] *= f[i];
      }
      if (spare) f[1] = f[0];
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        o[d][0] *= f[0];
        o[d][1] *= f[0];
        o[d][2] *= f[1];
        o[d][3] *= f[1];
      }
    }
    float ref[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) ref[i] = m[i] == neg_inf() ? 0.0f : m[i];
    uint32_t p[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = ex2(s[n][e] - ref[e >> 1]);
        l[e >> 1] += s[n][e];
      }
      p[2 * n] = pack2<T>(s[n][0], s[n][1]);
      p[2 * n + 1] = spare ? pack2_rest<T>(s[n][0], s[n][1], p[2 * n]) : pack2<T>(s[n][2], s[n][3]);
    }
    const auto load_values = [&](int d, uint32_t(&v)[4]) {
      ldsm_x4_trans(vs_at + chunk_at<D>(lane & 15, 2 * d + (lane >> 4)), v[0], v[1], v[2], v[3]);
    };
    // Keys that only some of the rows see: for the others their weight is zero, which only a finite value takes to zero.
    bool care = false;
    if (SHARE == kBySplit && uneven && !whole) {  // (else all rows are one token's)
      bool bad = false;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t v[4];
        load_values(d, v);
        bad |= not_finite2<T>(v[0]) || not_finite2<T>(v[1]) || not_finite2<T>(v[2]) || not_finite2<T>(v[3]);
      }
      care = __any_sync(0xffffffffu, bad);
    }
    if (!care) {
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t v[4];
        load_values(d, v);
        Mma<T>::run4(o[2 * d], p, v[0], v[1]);
        Mma<T>::run4(o[2 * d + 1], p, v[2], v[3]);
      }
    } else {
      // row by row, with the values that the row does not see at zero
      for (int r = 0; r < t.rows; ++r) {
        const int owner = (r & 7) * 4;
        const int f0 = __shfl_sync(0xffffffffu, from[0], owner), f1 = __shfl_sync(0xffffffffu, from[1], owner);
        const int t0 = __shfl_sync(0xffffffffu, to[0], owner), t1 = __shfl_sync(0xffffffffu, to[1], owner);
        const int lo = (r < 8 ? f0 : f1) - j0 - 2 * q4, hi = (r < 8 ? t0 : t1) - j0 - 2 * q4;
        const uint32_t m0 = (0 >= lo && 0 < hi ? 0xffffu : 0u) | (1 >= lo && 1 < hi ? 0xffff0000u : 0u);
        const uint32_t m1 = (8 >= lo && 8 < hi ? 0xffffu : 0u) | (9 >= lo && 9 < hi ? 0xffff0000u : 0u);
        const bool mine = g == (r & 7);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t v[4];
          load_values(d, v);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float (&sums)[4] = o[2 * d + n];
            float y[4] = {sums[0], sums[1], sums[2], sums[3]};  // (from the sums on: the bits of the row are those of the product above)
            Mma<T>::run4(y, p, v[2 * n] & m0, v[2 * n + 1] & m1);
            if (mine && r < 8) {
              sums[0] = y[0];
              sums[1] = y[1];
            }
            if (mine && (r >= 8 || spare)) {
              sums[2] = y[2];
              sums[3] = y[3];
            }
          }
        }
      }
    }
    __syncwarp();
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_async_wait_group<0>();

  if (spare) {
#pragma unroll
    for (int d = 0; d < D / 8; ++d) {
      // (an infinite value is in the first sum as it should be; its product with a rest, of either sign or zero, is nothing)
      if (isfinite(o[d][2])) o[d][0] += o[d][2];
      if (isfinite(o[d][3])) o[d][1] += o[d][3];
    }
  }
  // join the four lanes of a row, then the warps
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    if (q4 == 0) {
      s_m[warp][g + 8 * i] = m[i];
      s_l[warp][g + 8 * i] = l[i];
    }
  }
  __syncthreads();  // (every warp is done with its ring)
  float f[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float top = neg_inf();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][g + 8 * i]);
    f[i] = m[i] == neg_inf() ? 1.0f : ex2(m[i] - top);  // (no weights: sums of zero, or NaN from NaN scores)
  }
  constexpr int kPitch = D + 8;  // floats; rows g and g + 1 lie 8 banks apart
  float* sums = reinterpret_cast<float*>(ring) + warp * 16 * kPitch;
#pragma unroll
  for (int d = 0; d < D / 8; ++d) {
    *reinterpret_cast<float2*>(sums + g * kPitch + d * 8 + q4 * 2) = make_float2(o[d][0] * f[0], o[d][1] * f[0]);
    *reinterpret_cast<float2*>(sums + (g + 8) * kPitch + d * 8 + q4 * 2) = make_float2(o[d][2] * f[1], o[d][3] * f[1]);
  }
  __syncthreads();
  write_rows<T, D, SHARE>(a, t, z, kvh, reinterpret_cast<float*>(ring), s_m, s_l);
}

// The same for float32 and at most 8 rows, on the CUDA cores. A key's or a value's row
// goes straight from global memory to registers, D / 32 features to a lane (512
// bytes side by side for a head of 128), 32 / R keys at a time, the values on
// their way while the keys are worked on and the next keys while the values
// are. Each lane forms its features' part of the block's 32 scores; a butterfly
// that halves the scores a lane keeps at each of its five steps leaves each
// lane with one whole score. Weights go back to all lanes by shuffles. All sums are
// float32. Bound by its instructions, some 140 for a key and a value of 1 KB with
// eight rows. One context of 100001 tokens, 20 heads on 4: 188 us, 2.2 TB/s
// (341 us by the general kernel); 32 of up to 8001: 452 us against 488; 64 of up to 2001,
// 32 heads on 8: 360 us.
template <int D, int R, int SHARE>
__global__ void __launch_bounds__(kWarps * 32, 3) f32_rows_kernel(AttnArgs a) {
  constexpr int V = D / 32, kKeys = 32 / R;  // features of a lane; keys of a block
  struct alignas(4 * V) Vec {
    float e[V];
  };
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kvh = blockIdx.y;
  int z = blockIdx.z;
  pdl_trigger();
  AttnTile t;
  int64_t k0, k1;
  if (!find_work<SHARE>(a, &t, &z, &k0, &k1)) return;
  const float* kp = static_cast<const float*>(a.k) + kvh * a.c_hs + lane * V;
  const float* vp = static_cast<const float*>(a.v) + kvh * a.c_hs + lane * V;
  const int blocks = k1 > k0 ? static_cast<int>((k1 - k0 + kKeys - 1) / kKeys) : 0;

  // place of key lane % kKeys of block b in the pool, -1: no such key
  const auto place_of = [&](int b) -> int64_t {
    const int64_t j = k0 + static_cast<int64_t>(b) * kKeys + lane % kKeys;
    if (b >= blocks || j < t.lo || j >= k1) return -1;
    const uint32_t i = static_cast<uint32_t>(j) / static_cast<uint32_t>(a.b.page_size);
    const int page = page_of(a.b, t.s, i);
    return page < 0 ? -1 : page * a.c_ps + (static_cast<uint32_t>(j) - i * a.b.page_size) * a.c_ts;
  };
  const auto fetch = [&](Vec* x, const float* base, int64_t place) {
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      const int64_t at = __shfl_sync(0xffffffffu, place, j);
      if (at >= 0) {
        x[j] = *reinterpret_cast<const Vec*>(base + at);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) x[j].e[e] = 0.0f;
      }
    }
  };
  Vec keys[kKeys], values[kKeys];
  int64_t place = place_of(warp), next = place_of(warp + kWarps);
  fetch(keys, kp, place);
  float q[R][V], o[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int e = 0; e < V; ++e) q[r][e] = o[r][e] = 0.0f;
    if (r < t.rows) {
      int64_t token;
      int head;
      row_owner(a, t, kvh, r, &token, &head);
      const Vec x = *reinterpret_cast<const Vec*>(static_cast<const float*>(a.q) + token * a.q_ts + head * a.q_hs + lane * V);
#pragma unroll
      for (int e = 0; e < V; ++e) q[r][e] = x.e[e];
    }
  }
  // this lane's score of a block: row `mine`, key my_key; and the keys that the row sees, relative to k0
  const int mine = lane / kKeys, my_key = lane % kKeys;
  int from = 0, to = 0;
  {
    const auto rel = [&](int64_t j) {
      const int64_t d = j - k0, n = k1 - k0;
      return static_cast<int>(d < 0 ? 0 : d > n ? n : d);
    };
    const int64_t p = row_position(t, t.row0 + mine, a.group);
    to = mine < t.rows ? rel(p + 1) : 0;
    from = mine < t.rows && a.window > 0 ? rel(p - a.window + 1) : 0;
  }
  float m = neg_inf(), l = 0.0f;  // of row `mine`, l over this lane's keys

  for (int b = warp; b < blocks; b += kWarps) {
    fetch(values, vp, place);
    float s[32];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        float x = q[r][0] * keys[j].e[0];
#pragma unroll
        for (int e = 1; e < V; ++e) x = fmaf(q[r][e], keys[j].e[e], x);
        s[r * kKeys + j] = x;
      }
    fetch(keys, kp, next);
    place = next;
    next = place_of(b + 2 * kWarps);
#pragma unroll
    for (int step = 0; step < 5; ++step) {
      const int n = 16 >> step, bit = n;
      const bool upper = lane & bit;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i >= n) break;
        const float give = upper ? s[i] : s[i + n], have = upper ? s[i + n] : s[i];
        s[i] = have + __shfl_xor_sync(0xffffffffu, give, bit);
      }
    }
    float x = s[0] * a.scale;
    if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
    const int at = b * kKeys + my_key;
    x = at >= from && at < to ? x * kLog2e : neg_inf();
    float top = x;
#pragma unroll
    for (int bit = 1; bit < kKeys; bit *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, bit));
    if (__any_sync(0xffffffffu, top > m)) {
      const float now = fmaxf(m, top);
      const float f = now == neg_inf() ? 1.0f : exp2f(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float x = __shfl_sync(0xffffffffu, f, r * kKeys);
#pragma unroll
        for (int e = 0; e < V; ++e) o[r][e] *= x;
      }
    }
    const float weight = exp2f(x - (m == neg_inf() ? 0.0f : m));
    l += weight;
    // (all rows are one token's: what it does not see has come as zeros)
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        const float w = __shfl_sync(0xffffffffu, weight, r * kKeys + j);
#pragma unroll
        for (int e = 0; e < V; ++e) o[r][e] = fmaf(w, values[j].e[e], o[r][e]);
      }
  }
#pragma unroll
  for (int bit = 1; bit < kKeys; bit *= 2) l += __shfl_xor_sync(0xffffffffu, l, bit);
  if (my_key == 0) {
    s_m[warp][mine] = m;
    s_l[warp][mine] = l;
  }
  __syncthreads();
  constexpr int kPitch = D + 8;
  float* sums = reinterpret_cast<float*>(ring) + warp * 16 * kPitch;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float top = neg_inf();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
    const float f = s_m[warp][r] == neg_inf() ? 1.0f : exp2f(s_m[warp][r] - top);
    Vec x;
#pragma unroll
    for (int e = 0; e < V; ++e) x.e[e] = o[r][e] * f;
    *reinterpret_cast<Vec*>(sums + r * kPitch + lane * V) = x;
  }
  __syncthreads();
  write_rows<float, D, SHARE>(a, t, z, kvh, reinterpret_cast<float*>(ring), s_m, s_l);
}

// Joins the pieces of every sequence that has more than one (as combine_kernel of
// hc_attn.cu does splits), a CTA to a row: all weights first, then each warp
// adds every eighth piece. The pieces are worked out while the other kernel still
// runs, from the caller's lengths alone, which were complete before that kernel
// began (its launch waits for everything before it). Worked out after the wait, or left
// by the other kernel and read then, they cost 2 us: eight contexts of 4001, 20.6 -> 22.6.
template <typename T, int D>
__global__ void __launch_bounds__(256) rows_join_kernel(AttnArgs a) {
  __shared__ float s_w[kMaxPieces];
  __shared__ float s_red[8][2];
  __shared__ float s_o[8][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, s = blockIdx.x, head = blockIdx.y;
  const int kvh = head / a.group, r = head - kvh * a.group;
  const Pieces p = find_pieces(a, 0, s);
  pdl_wait();  // (in every thread, whatever it finds: later kernels on the stream count on this one's end alone)
  if (p.count == 1) return;
  const int64_t first = piece_row(a, kvh, p.unit0, r);  // the next piece's row is 16 on
  float top = neg_inf(), sum = 0.0f;
  for (int i = tid; i < p.count; i += 256) top = fmaxf(top, a.part_ml[first + i * 16].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_red[warp][0] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = fmaxf(top, s_red[w][0]);
  for (int i = tid; i < p.count; i += 256) {
    const float2 ml = a.part_ml[first + i * 16];
    const float w = ml.x == neg_inf() ? (ml.y == 0.0f ? 0.0f : 1.0f) : exp2f(ml.x - top);  // (NaN scores alone: m = -inf, l = NaN)
    s_w[i] = w;
    sum += ml.y * w;
  }
  sum = warp_sum(sum);
  if (lane == 0) s_red[warp][1] = sum;
  __syncthreads();
  sum = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) sum += s_red[w][1];
  if (lane < D / 4) {
    const float* src = a.part_o + first * D + lane * 4;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = warp; i < p.count; i += 8) {
      const float4 y = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(i) * 16 * D);
      const float w = s_w[i];
      x.x = fmaf(y.x, w, x.x);
      x.y = fmaf(y.y, w, x.y);
      x.z = fmaf(y.z, w, x.z);
      x.w = fmaf(y.w, w, x.w);
    }
    *reinterpret_cast<float4*>(&s_o[warp][lane * 4]) = x;
  }
  __syncthreads();
  if (tid < D) {
    float x = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) x += s_o[w][tid];
    stf(static_cast<T*>(a.out) + s * a.o_ts + head * a.o_hs + tid, sum == 0.0f ? 0.0f : x / sum);
  }
  if (tid == 0 && a.lse) a.lse[static_cast<int64_t>(s) * a.heads + head] = sum == 0.0f ? neg_inf() : top * kLn2 + logf(sum);
}

template <int SHARE, auto Kernel>
cudaError_t launch_kernel(const AttnArgs& a, int64_t slots, size_t smem, cudaStream_t s) {
  const cudaError_t e = ensure_smem<Kernel>(smem);
  if (e != cudaSuccess) return e;
  if (SHARE == kByCluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.b.seqs * kCluster, a.kv_heads);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, Kernel, a);
  }
  const dim3 grid = SHARE == kByPiece ? dim3(a.units, a.kv_heads) : dim3(static_cast<unsigned>(slots), a.kv_heads, a.g.splits);
  Kernel<<<grid, kWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int D, int SHARE>
cudaError_t launch_share(const AttnArgs& a, int64_t slots, cudaStream_t s) {
  constexpr size_t ring = static_cast<size_t>(kWarps) * kStages * kBlock * D * 4;
  constexpr size_t sums = static_cast<size_t>(sum_floats<D>(SHARE == kByCluster)) * 4;
  if constexpr (std::is_same<T, float>::value) {
    return a.group <= 4 ? launch_kernel<SHARE, f32_rows_kernel<D, 4, SHARE>>(a, slots, sums, s)
                        : launch_kernel<SHARE, f32_rows_kernel<D, 8, SHARE>>(a, slots, sums, s);
  } else {
    return launch_kernel<SHARE, rows_kernel<T, D, SHARE>>(a, slots, ring > sums ? ring : sums, s);
  }
}

template <typename T, int D>
cudaError_t launch_t(const AttnArgs& a, int64_t slots, cudaStream_t s) {
  if (a.clusters) return launch_share<T, D, kByCluster>(a, slots, s);
  if (a.units == 0) return launch_share<T, D, kBySplit>(a, slots, s);
  const cudaError_t e = launch_share<T, D, kByPiece>(a, slots, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(rows_join_kernel<T, D>, dim3(a.b.seqs, a.heads), dim3(256), 0, s, 1, a);
}

}  // namespace

bool attn_rows_supported(int dtype, int dim, bool single, int group, bool aligned) {
  return aligned && (dim == 64 || dim == 128) && (dtype != HC_F32 || (single && group <= 8));
}

RowsSchedule attn_rows_schedule(int64_t seqs, int kv_heads, int64_t keys, int num_sms) {
  const int64_t tiles = seqs * kv_heads, wave = 2 * static_cast<int64_t>(num_sms);
  if (keys <= kShortest || tiles * 2 > wave) return RowsSchedule{0, 0, false};
  if (keys <= kClusterKeys && tiles * kCluster <= wave) return RowsSchedule{0, 0, true};
  return RowsSchedule{static_cast<int>(wave - tiles), static_cast<int>((wave - tiles) / kv_heads + seqs), false};
}

cudaError_t launch_attn_rows(const AttnArgs& a, int dtype, int64_t slots, cudaStream_t s) {
  if (dtype == HC_F32) return a.dim == 64 ? launch_t<float, 64>(a, slots, s) : launch_t<float, 128>(a, slots, s);
  if (dtype == HC_F16) return a.dim == 64 ? launch_t<__half, 64>(a, slots, s) : launch_t<__half, 128>(a, slots, s);
  return a.dim == 64 ? launch_t<__nv_bfloat16, 64>(a, slots, s) : launch_t<__nv_bfloat16, 128>(a, slots, s);
}

}  // namespace hc
