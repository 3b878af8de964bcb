// Attention over a paged cache in float32 for many rows (heads of 64 or 128,
// aligned rows), on the tensor cores at float32's precision.
//
// Mathematics: a float32 x is cut into three bf16 of 8 bits each that sum to it
// exactly, and a product into the MMAs of its parts that matter,
//   x y = x0 y0 + x0 y1 + x1 y0 + x1 y1 + x0 y2 + x2 y0
// with fp32 accumulation. What is left out, x1 y2 + x2 y1 + x2 y2, is below 2^-21 |x y|
// (the parts are cut off, so that x1 may come near 2^-7 of x and x2 near 2^-15; its sign
// is that of x y), an eighth of the dim * 2^-24 of a float32 sum's bound at a head of 64.
// An MMA cuts its sums off rather than rounding
// them, so a block's values are summed by MMAs from zero and added to the running
// sums by a rounded addition (sums run through the MMAs were 1.7e-6 off on the case
// below, these are 5e-7, plain float32 sums 9e-7). Softmax as in hc_attn.cu, with
// CUDA's accurate exponential and tanh. An infinite key or value takes part in the
// product of the first parts alone (its rest would be NaN, and so would a zero part
// times infinity), so each has its first part a second time, zero if infinite,
// for the corrections.
//
// Work: a tile of 64 rows, 16 to a warp. Blocks of 16 keys go from global
// memory to registers, are cut into parts, once for the four warps, and stored
// in shared memory in the layout that ldmatrix reads without conflicts; while a
// block is multiplied, the next is cut and the one after is on its way.
//
// Bound: the warp-level MMAs, of which an m16n8k16 takes 8 cycles of a quarter
// SM, so that six for a product make 170 multiply-adds a cycle and SM (the CUDA
// cores have 128, and reached a third of that for want of operands). Three chunks
// of up to 131 tokens, 20 heads of 128, behind up to 901: 112 us; 1000 tokens
// behind 2000: 745 us, 34 TFLOP/s, 38% of the MMAs' rate; the rest is cutting and
// waiting, with two CTAs of four warps to an SM.
#include "hc_async.cuh"
#include "hc_attn.cuh"
#include "hc_attn_internal.h"
#include "hc_mma.cuh"

namespace hc {
namespace {

constexpr int kWarps = 4;

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

// Infinite and NaN values at keys that only some of a tile's rows see go into the
// products as zeros (a weight of zero must meet a finite value), and a bit stands
// for each key that has any; the rows that see such a key read its value again at
// the end and add what is not finite there, where any weight above zero gives the
// same.
struct OddValues {
  static constexpr int kSide = 96;  // keys where the rows' views begin, or end: 64 rows' and a block's rest
  static constexpr int kWords = 2 * kSide / 32;
  int any, lower, all_from, all_to;  // (keys are relative to the split's first, k0)
  uint32_t k0;
  uint32_t keys[kWords];  // keys with such values: from `lower` on, and from all_to on
};
__device__ __noinline__ float4 odd_taken(OddValues& s, float4 x, int key) {
  const int at = key < s.all_from ? min(key - s.lower, OddValues::kSide - 1)
                                  : OddValues::kSide + min(key - s.all_to, OddValues::kSide - 1);
  atomicOr(&s.keys[at >> 5], 1u << (at & 31));
  s.any = 1;
  return make_float4(isfinite(x.x) ? x.x : 0.0f, isfinite(x.y) ? x.y : 0.0f, isfinite(x.z) ? x.z : 0.0f,
                     isfinite(x.w) ? x.w : 0.0f);
}
__device__ __forceinline__ void set_odd_aside(OddValues& s, float4& x, int key) {
  if (key < s.all_from || key >= s.all_to) x = odd_taken(s, x, key);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2) f32_tile_kernel(AttnArgs a) {
  using C = TileCfg<D>;
  using M = Mma<__nv_bfloat16>;
  extern __shared__ __align__(128) unsigned char tile_smem[];
  __shared__ OddValues aside;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int z = blockIdx.z, kvh = blockIdx.y;
  pdl_trigger();
  if (a.clears && blockIdx.x == gridDim.x - 1) clear_unowned<float>(a, z * gridDim.y + kvh, gridDim.y * gridDim.z);
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
  const auto store = [&](int b) {
    unsigned char* const to = parts + (b & 1) * C::kBlock;
#pragma unroll
    for (int i = 0; i < C::kLoads; ++i) {
      const uint32_t at = chunk_at<D>(i * C::kAtOnce + row_of, piece >> 1) + (piece & 1) * 8;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        float4 x = held[kind][i];
        unsigned char* dst = to + kind * 4 * C::kPart + at;
        if (kind == 1 && !(isfinite(x.x) && isfinite(x.y) && isfinite(x.z) && isfinite(x.w)))
          set_odd_aside(aside, x, b * kTileKeys + i * C::kAtOnce + row_of);
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
  {
    // keys that all of the tile's rows see, relative to k0
    const int64_t first = row_position(t, t.row0, a.group), last = row_position(t, t.row0 + t.rows - 1, a.group);
    const auto rel = [&](int64_t j) { return static_cast<int>(max(min(j - k0, k1 - k0), int64_t{0})); };
    if (threadIdx.x < OddValues::kWords) aside.keys[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
      aside.any = 0;
      aside.k0 = static_cast<uint32_t>(k0);
      aside.lower = rel(t.lo);
      aside.all_from = a.window > 0 ? rel(last - a.window + 1) : 0;
      aside.all_to = rel(first + 1);
    }
    __syncthreads();
  }
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
  if (blocks > 0) store(0);
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
    if (b + 1 < blocks) store(b + 1);
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
          float y[4] = {};
          M::run4(y, p[2], v[1][2 * n], v[1][2 * n + 1]);
          M::run4(y, p[0], v[3][2 * n], v[3][2 * n + 1]);
          M::run4(y, p[1], v[2][2 * n], v[2][2 * n + 1]);
          M::run4(y, p[1], v[1][2 * n], v[1][2 * n + 1]);
          M::run4(y, p[0], v[2][2 * n], v[2][2 * n + 1]);
          M::run4(y, p[0], v[0][2 * n], v[0][2 * n + 1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[2 * d + n][e] += y[e];
        }
      }
    }
    __syncthreads();
  }
  if (row0 >= t.rows) return;
  if (aside.any != 0) {
    for (int side = 0; side < 2; ++side)
      for (int w = 0; w < OddValues::kWords / 2; ++w)
        for (uint32_t bits = aside.keys[side * (OddValues::kWords / 2) + w]; bits != 0; bits &= bits - 1) {
          const int key = (side == 0 ? aside.lower : aside.all_to) + 32 * w + __ffs(bits) - 1;
          const uint32_t j = static_cast<uint32_t>(aside.k0 + key), e = j / static_cast<uint32_t>(a.b.page_size);
          const int page = page_of(a.b, t.s, e);
          if (page < 0) continue;
          const float* v = static_cast<const float*>(a.v) + page * a.c_ps + (j - e * a.b.page_size) * a.c_ts + kvh * a.c_hs + q4 * 2;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (key < from[i] || key >= to[i]) continue;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
              const float2 x = *reinterpret_cast<const float2*>(v + d * 8);
              if (!isfinite(x.x)) o[d][2 * i] += x.x;
              if (!isfinite(x.y)) o[d][2 * i + 1] += x.y;
            }
          }
        }
  }
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
  constexpr size_t smem = TileCfg<D>::kSmem;
  const cudaError_t e = ensure_smem<f32_tile_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  f32_tile_kernel<D><<<dim3(static_cast<unsigned>(slots), a.kv_heads, a.g.splits), kWarps * 32, smem, s>>>(a);
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
