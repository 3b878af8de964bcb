// Attention over a paged cache in float32 (heads of 64 or 128, aligned rows), on
// the tensor cores at float32's precision.
//
// Mathematics: a float32 x is cut into parts of fewer bits that sum to it
// exactly, and a product into the MMAs of its parts that matter, with fp32
// accumulation:
//   three bf16 of 8 bits each (tile_kernel), x y = x0 y0 + x0 y1 + x1 y0 +
//     x1 y1 + x0 y2 + x2 y0, and at most 2^-23 |x y| left out;
//   a tf32 of 11 bits and the rest, of which the MMA reads 11 bits more
//     (rows_kernel), x y = hi hi + hi lo + lo hi, and at most 3 * 2^-22 |x y|.
// Scores, weights and sums of values keep float32's accuracy: what is left out is
// below the dim * 2^-24 of a sum in float32. Softmax as in hc_attn.cu, with
// CUDA's accurate exponential and tanh. An infinite key or value takes part in the
// product of the first parts alone (its rest would be NaN, and so would a zero part
// times infinity), so each has its first part a second time, zero if infinite,
// for the corrections.
//
// Bound: for many rows the warp-level MMAs (an m16n8k16 takes 8 cycles of a
// quarter SM, so six for a product make 170 multiply-adds a cycle and SM, where
// the CUDA cores have 128 and reach a third of that for want of operands);
// for few rows, bytes.
//
// tile_kernel: a tile of 64 rows, 16 to a warp. Blocks of 16 keys go from global
// memory to registers, are cut into parts, once for the four warps, and stored
// in shared memory in the layout that ldmatrix reads without conflicts; while a
// block is multiplied, the next is cut and the one after is on its way.
// rows_kernel, for sequences of at most 16 rows: all warps have the same rows, and
// each its own blocks of keys in a cp.async ring of its own (as in
// hc_attn_rows.cu); their results are joined at the end.
#include "hc_async.cuh"
#include "hc_attn.cuh"
#include "hc_attn_internal.h"
#include "hc_mma.cuh"

namespace hc {
namespace {

constexpr int kWarps = 4;

template <int D>
struct RowsCfg {
  // rows lie 4 banks apart, so that the MMA operands' loads (8 rows by 4
  // neighbours, or 8 neighbours by rows two apart) touch 32 banks
  static constexpr int kPitch = D + 4;
  static constexpr int kKeys = 16;  // keys of a block
  static constexpr int kStages = 3;
  static constexpr int kRows = 16;
  static constexpr int kBlock = 2 * kKeys * kPitch;  // floats of a block's keys and values
  static constexpr int kRing = kWarps * kStages * kBlock;
  static constexpr int kSums = kWarps * 16 * (D + 8);  // (joined in the ring's place)
  static constexpr size_t kSmem = static_cast<size_t>(kRows * kPitch + (kRing > kSums ? kRing : kSums)) * 4;
};

struct Split {
  uint32_t hi, lo;
};
__device__ __forceinline__ Split split(float x) {
  const uint32_t hi = __float_as_uint(x) & 0xffffe000u;
  return Split{hi, __float_as_uint(x - __uint_as_float(hi))};
}
// The same for keys and values, which may be infinite: such a number takes part in the product of the upper halves alone, for
// its rest would be NaN, and so would a lower half of zero times infinity. `cor` is the upper half for the correction.
struct SplitAny {
  uint32_t hi, cor, lo;
};
__device__ __forceinline__ SplitAny split_any(float x) {
  const uint32_t hi = __float_as_uint(x) & 0xffffe000u;
  const float lo = x - __uint_as_float(hi);
  const bool fine = lo == lo;
  return SplitAny{hi, fine ? hi : 0u, fine ? __float_as_uint(lo) : 0u};
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) f32_rows_kernel(AttnArgs a) {
  using C = RowsCfg<D>;
  constexpr int kKeys = C::kKeys, kPitch = C::kPitch, kTiles = kKeys / 8;
  extern __shared__ __align__(128) float smem[];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int z = blockIdx.z, kvh = blockIdx.y;
  float* const queries = smem;
  float* const ring = smem + C::kRows * kPitch + warp * C::kStages * C::kBlock;
  pdl_trigger();
  AttnTile t;
  tile_of_slot(a, blockIdx.x, &t);
  if (t.rows == 0 || z >= t.splits) return;
  int64_t k0, k1;
  split_range(a.g, t, z, &k0, &k1);
  const float* kp = static_cast<const float*>(a.k) + kvh * a.c_hs;
  const float* vp = static_cast<const float*>(a.v) + kvh * a.c_hs;
  const int blocks = k1 > k0 ? static_cast<int>((k1 - k0 + kKeys - 1) / kKeys) : 0;

  // Block b into a stage: the lanes take a row's 16-byte pieces side by side; a row that does not exist is zeros.
  constexpr int kPieces = D / 4, kAtOnce = 32 / kPieces;
  static_assert(kAtOnce >= 1, "a row at a time at least");
  const int piece = lane % kPieces, row_of = lane / kPieces;
  const auto bring = [&](int b, int stage) {
    if (b >= blocks) return;
    float* to = ring + stage * C::kBlock;
#pragma unroll
    for (int i = 0; i < kKeys / kAtOnce; ++i) {
      const int r = i * kAtOnce + row_of;
      const int64_t j = k0 + static_cast<int64_t>(b) * kKeys + r;
      int64_t at = -1;
      if (j >= t.lo && j < k1) {
        const uint32_t e = static_cast<uint32_t>(j) / static_cast<uint32_t>(a.b.page_size);
        const int page = page_of(a.b, t.s, e);
        if (page >= 0) at = page * a.c_ps + (static_cast<uint32_t>(j) - e * a.b.page_size) * a.c_ts;
      }
      const int64_t off = (at < 0 ? 0 : at) + piece * 4;
      const uint32_t bytes = at < 0 ? 0 : 16;
      cp_async16_zfill(smem_addr(to + r * kPitch + piece * 4), kp + off, bytes);
      cp_async16_zfill(smem_addr(to + (kKeys + r) * kPitch + piece * 4), vp + off, bytes);
    }
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) {
    bring(warp + i * kWarps, i);
    cp_async_commit();
  }
  // queries, rows past the last as zeros
  for (int r = warp; r < C::kRows; r += kWarps) {
    const float* src = nullptr;
    if (r < t.rows) {
      int64_t token;
      int head;
      row_owner(a, t, kvh, r, &token, &head);
      src = static_cast<const float*>(a.q) + token * a.q_ts + head * a.q_hs;
    }
    for (int d = lane; d < D; d += 32) queries[r * kPitch + d] = src ? src[d] : 0.0f;
  }
  __syncthreads();
  const float* const qa = queries + g * kPitch + q4;

  // keys that this thread's two rows see, relative to k0: [from, to)
  int from[2], to[2], all_from = 0, all_to = 0;
  const auto rel = [&](int64_t j) {
    const int64_t d = j - k0, n = k1 - k0;
    return static_cast<int>(d < 0 ? 0 : d > n ? n : d);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i;
    const int64_t p = row_position(t, t.row0 + r, a.group);
    to[i] = r < t.rows ? rel(p + 1) : 0;
    from[i] = r < t.rows && a.window > 0 ? rel(p - a.window + 1) : 0;
  }
  all_to = rel(row_position(t, t.row0, a.group) + 1);  // seen by every row: [all_from, all_to)
  if (a.window > 0) all_from = rel(row_position(t, t.row0 + t.rows - 1, a.group) - a.window + 1);

  float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.0f, 0.0f};
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;

  int stage = 0;
  for (int b = warp; b < blocks; b += kWarps) {
    cp_async_wait_group<C::kStages - 2>();
    __syncwarp();
    bring(b + (C::kStages - 1) * kWarps, stage == 0 ? C::kStages - 1 : stage - 1);
    cp_async_commit();
    const float* keys = ring + stage * C::kBlock;
    const float* values = keys + kKeys * kPitch;
    stage = stage + 1 == C::kStages ? 0 : stage + 1;
    float s[kTiles][4] = {}, c[kTiles][4] = {};  // products of the upper halves, and the corrections
#pragma unroll 4
    for (int ks = 0; ks < D; ks += 8) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Split x = split(qa[(i & 1) * 8 * kPitch + ks + (i >> 1) * 4]);
        hi[i] = x.hi;
        lo[i] = x.lo;
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        const float* kb = keys + (n * 8 + g) * kPitch + ks + q4;
        const SplitAny x = split_any(kb[0]), y = split_any(kb[4]);
        mma_tf32(c[n], lo, x.cor, y.cor);
        mma_tf32(s[n], hi, x.hi, y.hi);
        mma_tf32(c[n], hi, x.lo, y.lo);
      }
    }
    const int j0 = b * kKeys;
    const bool whole = j0 >= all_from && j0 + kKeys <= all_to;
    float top[2] = {neg_inf(), neg_inf()};
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = (s[n][e] + c[n][e]) * a.scale;
        if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
        x *= kLog2e;
        const int j = j0 + 8 * n + 2 * q4 + (e & 1), i = e >> 1;
        if (!whole && (j < from[i] || j >= to[i])) x = neg_inf();
        s[n][e] = x;
        top[i] = fmaxf(top[i], x);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float now = fmaxf(m[i], top[i]);
        f[i] = now == neg_inf() ? 1.0f : exp2f(m[i] - now);
        m[i] = now;
        l[i] *= f[i];
      }
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        o[d][0] *= f[0];
        o[d][1] *= f[0];
        o[d][2] *= f[1];
        o[d][3] *= f[1];
      }
    }
    const float ref[2] = {m[0] == neg_inf() ? 0.0f : m[0], m[1] == neg_inf() ? 0.0f : m[1]};
    // The scores' places (rows g, g + 8; keys 2 q4, 2 q4 + 1) are those of the second product's A operand (columns q4, q4 + 4) if
    // its column q4 stands for key 2 q4 and q4 + 4 for 2 q4 + 1.
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = exp2f(s[n][e] - ref[e >> 1]);
        l[e >> 1] += w;
        const Split x = split(w);
        const int i = (e >> 1) | ((e & 1) << 1);
        hi[i] = x.hi;
        lo[i] = x.lo;
      }
      const float* vb = values + (n * 8 + 2 * q4) * kPitch + g;
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        const SplitAny x = split_any(vb[d * 8]), y = split_any(vb[kPitch + d * 8]);
        mma_tf32(o[d], lo, x.cor, y.cor);
        mma_tf32(o[d], hi, x.lo, y.lo);
        mma_tf32(o[d], hi, x.hi, y.hi);
      }
    }
    __syncwarp();
  }
  cp_async_wait_group<0>();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }

  // a row's four features to the partial results, or divided to out
  const auto write = [&](int r, int d, float4 x, float top, float sum) {
    int64_t token;
    int head;
    row_owner(a, t, kvh, r, &token, &head);
    if (t.splits > 1) {
      const int64_t at = part_index(a, z, token, head);
      *reinterpret_cast<float4*>(a.part_o + at * D + d) = x;
      if (d == 0) a.part_ml[at] = make_float2(top, sum);
    } else {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      float* dst = static_cast<float*>(a.out) + token * a.o_ts + head * a.o_hs + d;
      dst[0] = x.x * inv;
      dst[1] = x.y * inv;
      dst[2] = x.z * inv;
      dst[3] = x.w * inv;
      if (d == 0 && a.lse) a.lse[token * a.heads + head] = sum == 0.0f ? neg_inf() : top * kLn2 + logf(sum);
    }
  };
  if (q4 == 0)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      s_m[warp][g + 8 * i] = m[i];
      s_l[warp][g + 8 * i] = l[i];
    }
  __syncthreads();  // (every warp is done with its ring)
  float f[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float top = neg_inf();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][g + 8 * i]);
    f[i] = m[i] == neg_inf() ? 1.0f : exp2f(m[i] - top);
  }
  constexpr int kSumPitch = D + 8;
  float* const all = smem + C::kRows * kPitch;
  float* const sums = all + warp * 16 * kSumPitch;
#pragma unroll
  for (int d = 0; d < D / 8; ++d) {
    *reinterpret_cast<float2*>(sums + g * kSumPitch + d * 8 + q4 * 2) = make_float2(o[d][0] * f[0], o[d][1] * f[0]);
    *reinterpret_cast<float2*>(sums + (g + 8) * kSumPitch + d * 8 + q4 * 2) = make_float2(o[d][2] * f[1], o[d][3] * f[1]);
  }
  __syncthreads();
  for (int u = threadIdx.x; u < t.rows * kPieces; u += kWarps * 32) {
    const int r = u / kPieces, d = (u - r * kPieces) * 4;
    float top = neg_inf(), sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_l[w][r] * (s_m[w][r] == neg_inf() ? 1.0f : exp2f(s_m[w][r] - top));
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(all + (w * 16 + r) * kSumPitch + d);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    write(r, d, x, top, sum);
  }
}

// ------------------------------------------------------------------- tiles --

constexpr int kTileRows = 16 * kWarps;
constexpr int kTileKeys = 16;

template <int D>
struct TileCfg {
  static constexpr int kRow = D * 2;                             // bytes of a row of one part
  static constexpr int kPart = kTileKeys * kRow;                 // a block's keys (or values), one part
  static constexpr int kBlock = 8 * kPart;                       // keys and values, parts 0, 0 again, 1, 2
  static constexpr int kQueries = 3 * kTileRows * kRow;
  static constexpr size_t kSmem = kQueries + 2 * kBlock;
  static constexpr int kPieces = D / 4;                          // 16-byte pieces of a row in float32
  static constexpr int kAtOnce = kWarps * 32 / kPieces;          // rows that the CTA loads at once
  static constexpr int kLoads = kTileKeys / kAtOnce;
};

// Byte of 16-byte chunk c of row r among rows of D 16-bit elements: chunks are
// permuted by the row's low three bits, so that the eight rows of an 8x8 matrix lie
// in different banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return static_cast<uint32_t>(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// Parts of two floats as pairs of bf16. The parts are cut off, not rounded, so
// that three of 8 bits are all 24 bits, and no part overflows.
struct Parts {
  uint32_t p0, p1, p2;
};
__device__ __forceinline__ uint32_t upper_pair(uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x7632); }
__device__ __forceinline__ Parts cut(float x, float y) {
  const uint32_t x0 = __float_as_uint(x), y0 = __float_as_uint(y);
  const float x1 = x - __uint_as_float(x0 & 0xffff0000u), y1 = y - __uint_as_float(y0 & 0xffff0000u);
  const float x2 = x1 - __uint_as_float(__float_as_uint(x1) & 0xffff0000u);
  const float y2 = y1 - __uint_as_float(__float_as_uint(y1) & 0xffff0000u);
  return Parts{upper_pair(x0, y0), upper_pair(__float_as_uint(x1), __float_as_uint(y1)),
               upper_pair(__float_as_uint(x2), __float_as_uint(y2))};
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2) f32_tile_kernel(AttnArgs a) {
  using C = TileCfg<D>;
  using M = Mma<__nv_bfloat16>;
  extern __shared__ __align__(128) unsigned char tile_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int z = blockIdx.z, kvh = blockIdx.y;
  pdl_trigger();
  AttnTile t;
  tile_of_slot(a, blockIdx.x, &t);
  if (t.rows == 0 || z >= t.splits) return;
  int64_t k0, k1;
  split_range(a.g, t, z, &k0, &k1);
  const float* kp = static_cast<const float*>(a.k) + kvh * a.c_hs;
  const float* vp = static_cast<const float*>(a.v) + kvh * a.c_hs;
  const int blocks = k1 > k0 ? static_cast<int>((k1 - k0 + kTileKeys - 1) / kTileKeys) : 0;
  unsigned char* const parts = tile_smem + C::kQueries;

  // This thread's pieces of block b's keys and values, on their way; then cut and stored.
  float4 held[2][C::kLoads];
  const int piece = threadIdx.x % C::kPieces, row_of = threadIdx.x / C::kPieces;
  const auto load = [&](int b) {
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      held[0][i] = held[1][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int64_t j = k0 + static_cast<int64_t>(b) * kTileKeys + i * C::kAtOnce + row_of;
      if (j < t.lo || j >= k1) continue;
      const uint32_t e = static_cast<uint32_t>(j) / static_cast<uint32_t>(a.b.page_size);
      const int page = page_of(a.b, t.s, e);
      if (page < 0) continue;
      const int64_t at = page * a.c_ps + (static_cast<uint32_t>(j) - e * a.b.page_size) * a.c_ts + piece * 4;
      held[0][i] = *reinterpret_cast<const float4*>(kp + at);
      held[1][i] = *reinterpret_cast<const float4*>(vp + at);
    }
  };
  const auto store = [&](unsigned char* to) {
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      const uint32_t at = chunk_at<D>(i * C::kAtOnce + row_of, piece >> 1) + (piece & 1) * 8;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        float4 x = held[kind][i];
        unsigned char* dst = to + kind * 4 * C::kPart + at;
        const auto put = [&](int part, uint32_t lo, uint32_t hi) {
          *reinterpret_cast<uint2*>(dst + part * C::kPart) = make_uint2(lo, hi);
        };
        put(0, upper_pair(__float_as_uint(x.x), __float_as_uint(x.y)), upper_pair(__float_as_uint(x.z), __float_as_uint(x.w)));
        x.x = isinf(x.x) ? 0.0f : x.x;
        x.y = isinf(x.y) ? 0.0f : x.y;
        x.z = isinf(x.z) ? 0.0f : x.z;
        x.w = isinf(x.w) ? 0.0f : x.w;
        const Parts lo = cut(x.x, x.y), hi = cut(x.z, x.w);
        put(1, lo.p0, hi.p0);
        put(2, lo.p1, hi.p1);
        put(3, lo.p2, hi.p2);
      }
    }
  };
  if (blocks > 0) load(0);
  // queries: a warp cuts its own 16 rows (those past the last are zeros)
  const int row0 = warp * 16;
  for (int i = lane; i < 16 * C::kPieces; i += 32) {
    const int r = row0 + i / C::kPieces, c = i % C::kPieces;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (r < t.rows) {
      int64_t token;
      int head;
      row_owner(a, t, kvh, r, &token, &head);
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + token * a.q_ts + head * a.q_hs + c * 4);
    }
    const Parts lo = cut(x.x, x.y), hi = cut(x.z, x.w);
    unsigned char* dst = tile_smem + chunk_at<D>(r, c >> 1) + (c & 1) * 8;
    *reinterpret_cast<uint2*>(dst) = make_uint2(lo.p0, hi.p0);
    *reinterpret_cast<uint2*>(dst + kTileRows * C::kRow) = make_uint2(lo.p1, hi.p1);
    *reinterpret_cast<uint2*>(dst + 2 * kTileRows * C::kRow) = make_uint2(lo.p2, hi.p2);
  }
  if (blocks > 0) store(parts);
  if (blocks > 1) load(1);
  __syncthreads();

  // keys that this thread's two rows see, relative to k0: [from, to)
  int from[2], to[2], all_from = 0, all_to = 0;
  const auto rel = [&](int64_t j) {
    const int64_t d = j - k0, n = k1 - k0;
    return static_cast<int>(d < 0 ? 0 : d > n ? n : d);
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row0 + g + 8 * i;
    const int64_t p = row_position(t, t.row0 + r, a.group);
    to[i] = r < t.rows ? rel(p + 1) : 0;
    from[i] = r < t.rows && a.window > 0 ? rel(p - a.window + 1) : 0;
  }
  if (row0 + 15 < t.rows) {  // seen by all of the warp's rows: [all_from, all_to)
    all_to = rel(row_position(t, t.row0 + row0, a.group) + 1);
    if (a.window > 0) all_from = rel(row_position(t, t.row0 + row0 + 15, a.group) - a.window + 1);
  }

  float m[2] = {neg_inf(), neg_inf()}, l[2] = {0.0f, 0.0f};
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
  const uint32_t q_at = smem_addr(tile_smem), parts_at = smem_addr(parts);

  for (int b = 0; b < blocks; ++b) {
    const uint32_t k_at = parts_at + (b & 1) * C::kBlock, v_at = k_at + 4 * C::kPart;
    // the next block into the other buffer (all warps are done with it), the one after on its way
    if (b + 1 < blocks) store(parts + ((b + 1) & 1) * C::kBlock);
    if (b + 2 < blocks) load(b + 2);
    if (row0 < t.rows) {
      float s[2][4] = {}, c[2][4] = {};  // first parts' products, and the corrections
#pragma unroll 2
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t q[3][4], k[4][4];
#pragma unroll
        for (int i = 0; i < 3; ++i)
          ldsm_x4(q_at + i * kTileRows * C::kRow + chunk_at<D>(row0 + (lane & 15), 2 * ks + (lane >> 4)), q[i][0], q[i][1], q[i][2],
                  q[i][3]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ldsm_x4(k_at + i * C::kPart + chunk_at<D>(((lane >> 4) << 3) + (lane & 7), 2 * ks + ((lane >> 3) & 1)), k[i][0], k[i][1],
                  k[i][2], k[i][3]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          M::run4(c[n], q[2], k[1][2 * n], k[1][2 * n + 1]);
          M::run4(s[n], q[0], k[0][2 * n], k[0][2 * n + 1]);
          M::run4(c[n], q[0], k[3][2 * n], k[3][2 * n + 1]);
          M::run4(c[n], q[1], k[2][2 * n], k[2][2 * n + 1]);
          M::run4(c[n], q[1], k[1][2 * n], k[1][2 * n + 1]);
          M::run4(c[n], q[0], k[2][2 * n], k[2][2 * n + 1]);
        }
      }
      const int j0 = b * kTileKeys;
      const bool whole = j0 >= all_from && j0 + kTileKeys <= all_to;
      float top[2] = {neg_inf(), neg_inf()};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = (s[n][e] + c[n][e]) * a.scale;
          if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
          x *= kLog2e;
          const int j = j0 + 8 * n + 2 * q4 + (e & 1), i = e >> 1;
          if (!whole && (j < from[i] || j >= to[i])) x = neg_inf();
          s[n][e] = x;
          top[i] = fmaxf(top[i], x);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float now = fmaxf(m[i], top[i]);
          f[i] = now == neg_inf() ? 1.0f : exp2f(m[i] - now);
          m[i] = now;
          l[i] *= f[i];
        }
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          o[d][0] *= f[0];
          o[d][1] *= f[0];
          o[d][2] *= f[1];
          o[d][3] *= f[1];
        }
      }
      const float ref[2] = {m[0] == neg_inf() ? 0.0f : m[0], m[1] == neg_inf() ? 0.0f : m[1]};
      uint32_t p[3][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = exp2f(s[n][2 * i] - ref[i]), y = exp2f(s[n][2 * i + 1] - ref[i]);
          l[i] += x + y;
          const Parts w = cut(x, y);
          p[0][2 * n + i] = w.p0;
          p[1][2 * n + i] = w.p1;
          p[2][2 * n + i] = w.p2;
        }
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          ldsm_x4_trans(v_at + i * C::kPart + chunk_at<D>(lane & 15, 2 * d + (lane >> 4)), v[i][0], v[i][1], v[i][2], v[i][3]);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float(&y)[4] = o[2 * d + n];
          M::run4(y, p[2], v[1][2 * n], v[1][2 * n + 1]);
          M::run4(y, p[0], v[3][2 * n], v[3][2 * n + 1]);
          M::run4(y, p[1], v[2][2 * n], v[2][2 * n + 1]);
          M::run4(y, p[1], v[1][2 * n], v[1][2 * n + 1]);
          M::run4(y, p[0], v[2][2 * n], v[2][2 * n + 1]);
          M::run4(y, p[0], v[0][2 * n], v[0][2 * n + 1]);
        }
      }
    }
    __syncthreads();
  }
  if (row0 >= t.rows) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
  }
  // pairs of lanes trade two features, so that each has four of one of the two rows
  const bool odd = q4 & 1;
  const int r = row0 + g + 8 * odd;
  const float top = odd ? m[1] : m[0], sum = odd ? l[1] : l[0];
  const float inv = t.splits > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
  int64_t token = 0;
  int head = 0;
  if (r < t.rows) row_owner(a, t, kvh, r, &token, &head);
  const int64_t at = part_index(a, z, token, head);
  float* dst = t.splits > 1 ? a.part_o + at * D : static_cast<float*>(a.out) + token * a.o_ts + head * a.o_hs;
  const bool wide = t.splits > 1 || (((a.o_ts | a.o_hs) & 3) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0);
#pragma unroll
  for (int d = 0; d < D / 8; ++d) {
    const float2 mine = odd ? make_float2(o[d][2], o[d][3]) : make_float2(o[d][0], o[d][1]);
    const float2 give = odd ? make_float2(o[d][0], o[d][1]) : make_float2(o[d][2], o[d][3]);
    const float2 got = make_float2(__shfl_xor_sync(0xffffffffu, give.x, 1), __shfl_xor_sync(0xffffffffu, give.y, 1));
    const float4 x = odd ? make_float4(got.x * inv, got.y * inv, mine.x * inv, mine.y * inv)
                         : make_float4(mine.x * inv, mine.y * inv, got.x * inv, got.y * inv);
    if (r >= t.rows) continue;
    float* y = dst + d * 8 + (q4 >> 1) * 4;
    if (wide) {
      *reinterpret_cast<float4*>(y) = x;
    } else {
      y[0] = x.x;
      y[1] = x.y;
      y[2] = x.z;
      y[3] = x.w;
    }
  }
  if (r < t.rows && q4 < 2) {
    if (t.splits > 1) {
      a.part_ml[at] = make_float2(top, sum);
    } else if (a.lse) {
      a.lse[token * a.heads + head] = sum == 0.0f ? neg_inf() : top * kLn2 + logf(sum);
    }
  }
}

template <int D>
cudaError_t launch_t(const AttnArgs& a, int64_t slots, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(slots), a.kv_heads, a.g.splits);
  if (a.g.rows == 16) {
    constexpr size_t smem = RowsCfg<D>::kSmem;
    const cudaError_t e = ensure_smem<f32_rows_kernel<D>>(smem);
    if (e != cudaSuccess) return e;
    f32_rows_kernel<D><<<grid, kWarps * 32, smem, s>>>(a);
  } else {
    constexpr size_t smem = TileCfg<D>::kSmem;
    const cudaError_t e = ensure_smem<f32_tile_kernel<D>>(smem);
    if (e != cudaSuccess) return e;
    f32_tile_kernel<D><<<grid, kWarps * 32, smem, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

bool attn_f32_supported(int dtype, int dim, bool aligned) {
  return aligned && dtype == HC_F32 && (dim == 64 || dim == 128);
}

cudaError_t launch_attn_f32(const AttnArgs& a, int64_t slots, cudaStream_t s) {
  return a.dim == 64 ? launch_t<64>(a, slots, s) : launch_t<128>(a, slots, s);
}

}  // namespace hc
