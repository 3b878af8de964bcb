// Attention of new tokens over a paged cache (include/hc_paged.h): the choice
// of kernels, the general kernel, and the kernel that joins splits.
//
// General kernel, for what the specialised ones do not take (heads other than 64
// and 128, operands off 16-byte boundaries, odd page sizes and scales of zero or
// below for chunks in 16 bits, several tokens of few rows in float32): every type,
// head size, page size, stride and alignment, fp32 arithmetic on the CUDA cores. A CTA holds `ROWS` rows of
// queries in shared memory and passes once over the split's keys in steps of
// kKeys: scores into shared memory, running maximum m and sum l of each row
//   m' = max(m, max_j s_j),  l' = l 2^(m - m') + sum_j 2^(s_j - m')
// with s in base-2 exponents, and the sums of values scaled alike in
// registers. 16 rows to a tile where a sequence has no more than that (single
// tokens), else 64. Bound, for many rows, by the loads of its operands from shared
// memory (a 16-byte load takes four cycles of the SM for 16 multiply-adds of
// each of 32 threads): three chunks of up to 131 tokens of 20 heads behind up to
// 901, heads of 96 in bf16 163 us, 14 TFLOP/s, of 256 371 us, 16 TFLOP/s; heads of
// 128 in float32, if it is made to take them, 158 us, 19 TFLOP/s.
#include <algorithm>
#include <type_traits>

#include "hc_async.cuh"
#include "hc_attn_internal.h"
#include "hc_paged_internal.h"

namespace hc {
namespace {

constexpr int kThreads = 256;
constexpr int kKeys = 32;

// DP: head_dim padded to a multiple of 64. BUFS: buffers of keys and values, two
// where the next step's come by cp.async while this one is worked on.
template <int ROWS, int DP, int BUFS>
struct GeneralSmem {
  float q[ROWS][DP + 4];
  float k[BUFS][kKeys][DP + 4];
  float v[BUFS][kKeys][DP];
  float p[ROWS][kKeys + 4];
  float alpha[ROWS];
  float m[ROWS], l[ROWS];
};

// Threads are 16 x 16: thread (ty, tx) forms the scores of rows ty + 16 i and
// keys tx, tx + 16, and the sums of rows ty + 16 i and features 4 tx + 64 c ..
// + 3. Keys j of a step belong to warp j % 8, which finds their places in the
// pool and copies their rows.
template <typename T, int ROWS, int DP, bool ASYNC>
__global__ void __launch_bounds__(kThreads) general_kernel(AttnArgs a) {
  constexpr int BUFS = ASYNC ? 2 : 1;
  extern __shared__ __align__(16) unsigned char raw[];
  auto& sm = *reinterpret_cast<GeneralSmem<ROWS, DP, BUFS>*>(raw);
  constexpr int RI = ROWS / 16, CI = DP / 64;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, lane = tid & 31;
  const int z = blockIdx.z, kvh = blockIdx.y;
  if (a.clears && blockIdx.x == gridDim.x - 1) clear_unowned<T>(a, z * gridDim.y + kvh, gridDim.y * gridDim.z);
  AttnTile t;
  tile_of_slot(a, blockIdx.x, &t);
  if (t.rows == 0 || z >= t.splits) return;
  int64_t k0, k1;
  split_range(a.g, t, z, &k0, &k1);
  const T* kp = static_cast<const T*>(a.k);
  const T* vp = static_cast<const T*>(a.v);

  const auto bring = [&](int64_t kb, int buf) {
    int64_t at[kKeys / 8];
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) {
      const int64_t j = kb + warp + 8 * i;
      at[i] = -1;
      if (j >= t.lo && j < k1) {
        const int page = page_of(a.b, t.s, j / a.b.page_size);
        if (page >= 0) at[i] = page * a.c_ps + j % a.b.page_size * a.c_ts + kvh * a.c_hs;
      }
    }
#pragma unroll
    for (int i = 0; i < kKeys / 8; ++i) {
      const int j = warp + 8 * i;
      if (ASYNC) {
#pragma unroll
        for (int d = lane * 4; d < DP; d += 128) {
          const bool in = at[i] >= 0 && d < a.dim;
          const int64_t off = in ? at[i] + d : 0;
          cp_async16_zfill(smem_addr(&sm.k[buf][j][d]), kp + off, in ? 16 : 0);
          cp_async16_zfill(smem_addr(&sm.v[buf][j][d]), vp + off, in ? 16 : 0);
        }
      } else {
#pragma unroll
        for (int d = lane; d < DP; d += 32) {
          const bool in = at[i] >= 0 && d < a.dim;
          sm.k[buf][j][d] = in ? ldf(kp + at[i] + d) : 0.0f;
          sm.v[buf][j][d] = in ? ldf(vp + at[i] + d) : 0.0f;
        }
      }
    }
  };
  if (ASYNC) {
    bring(k0, 0);
    cp_async_commit();
  }
  for (int r = warp; r < ROWS; r += kThreads / 32) {
    const T* src = nullptr;
    if (r < t.rows) {
      int64_t token;
      int head;
      row_owner(a, t, kvh, r, &token, &head);
      src = static_cast<const T*>(a.q) + token * a.q_ts + head * a.q_hs;
    }
    for (int d = lane; d < DP; d += 32) sm.q[r][d] = src != nullptr && d < a.dim ? ldf(src + d) : 0.0f;
  }
  if (tid < ROWS) {
    sm.m[tid] = neg_inf();
    sm.l[tid] = 0.0f;
  }
  float acc[RI][CI][4] = {};

  int buf = 0;
  for (int64_t kb = k0; kb < k1; kb += kKeys) {
    __syncthreads();
    if (ASYNC) {
      if (kb + kKeys < k1) bring(kb + kKeys, buf ^ 1);
      cp_async_commit();
      cp_async_wait_group1();
    } else {
      bring(kb, 0);
    }
    __syncthreads();
    float s[RI][2] = {};
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
      const float4 x = *reinterpret_cast<const float4*>(&sm.k[buf][tx][d]);
      const float4 y = *reinterpret_cast<const float4*>(&sm.k[buf][tx + 16][d]);
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(&sm.q[ty + 16 * i][d]);
        s[i][0] = fmaf(q.x, x.x, fmaf(q.y, x.y, fmaf(q.z, x.z, fmaf(q.w, x.w, s[i][0]))));
        s[i][1] = fmaf(q.x, y.x, fmaf(q.y, y.y, fmaf(q.z, y.z, fmaf(q.w, y.w, s[i][1]))));
      }
    }
    // running maximum and sum: the 16 threads of a row are half a warp
    bool masked = false;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int r = ty + 16 * i;
      const int64_t p = row_position(t, t.row0 + r, a.group);
      float top = neg_inf();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t j = kb + tx + 16 * c;
        float x = s[i][c] * a.scale;
        if (a.softcap > 0.0f) x = a.softcap * tanhf(x / a.softcap);
        x *= kLog2e;
        const bool seen = r < t.rows && j < k1 && j <= p && (a.window <= 0 || j > p - a.window);
        masked |= !seen;
        s[i][c] = seen ? x : neg_inf();
        top = fmaxf(top, s[i][c]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float old = sm.m[r];
      const float now = fmaxf(old, top);
      const float ref = now == neg_inf() ? 0.0f : now;  // nothing seen yet
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float w = exp2f(s[i][c] - ref);
        sum += w;
        sm.p[r][tx + 16 * c] = w;
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncwarp();
      if (tx == 0) {
        const float scale = exp2f(old - ref);
        sm.alpha[r] = scale;
        sm.m[r] = now;
        sm.l[r] = sm.l[r] * scale + sum;
      }
    }
    masked = __syncthreads_or(masked);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const float f = sm.alpha[ty + 16 * i];
#pragma unroll
      for (int c = 0; c < CI; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][c][e] *= f;
    }
    // four keys at a time, so that a row's weights come in one load
    const auto add_values = [&](auto skip_zeros) {
#pragma unroll 2
      for (int j0 = 0; j0 < kKeys; j0 += 4) {
        float4 w4[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) w4[i] = *reinterpret_cast<const float4*>(&sm.p[ty + 16 * i][j0]);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          float4 v[CI];
#pragma unroll
          for (int c = 0; c < CI; ++c) v[c] = *reinterpret_cast<const float4*>(&sm.v[buf][j0 + jj][4 * tx + 64 * c]);
#pragma unroll
          for (int i = 0; i < RI; ++i) {
            const float w = jj == 0 ? w4[i].x : jj == 1 ? w4[i].y : jj == 2 ? w4[i].z : w4[i].w;
            if (decltype(skip_zeros)::value && w == 0.0f) continue;
#pragma unroll
            for (int c = 0; c < CI; ++c) {
              acc[i][c][0] = fmaf(w, v[c].x, acc[i][c][0]);
              acc[i][c][1] = fmaf(w, v[c].y, acc[i][c][1]);
              acc[i][c][2] = fmaf(w, v[c].z, acc[i][c][2]);
              acc[i][c][3] = fmaf(w, v[c].w, acc[i][c][3]);
            }
          }
        }
      }
    };
    // a weight of zero adds nothing, whatever the value at a key that the row does not see
    if (masked) {
      add_values(std::true_type());
    } else {
      add_values(std::false_type());
    }
    if (ASYNC) buf ^= 1;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = ty + 16 * i;
    if (r >= t.rows) continue;
    int64_t token;
    int head;
    row_owner(a, t, kvh, r, &token, &head);
    const float l = sm.l[r], m = sm.m[r];
    if (t.splits > 1) {
      const int64_t at = part_index(a, z, token, head);
      for (int c = 0; c < CI; ++c)
        for (int e = 0; e < 4; ++e) {
          const int d = 4 * tx + 64 * c + e;
          if (d < a.dim) a.part_o[at * a.dim + d] = acc[i][c][e];
        }
      if (tx == 0) a.part_ml[at] = make_float2(m, l);
    } else {
      T* dst = static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs;
      const float f = l == 0.0f ? 0.0f : 1.0f / l;  // no weight at all: the row sees nothing
      for (int c = 0; c < CI; ++c)
        for (int e = 0; e < 4; ++e) {
          const int d = 4 * tx + 64 * c + e;
          if (d < a.dim) stf(dst + d, acc[i][c][e] * f);
        }
      if (tx == 0 && a.lse) a.lse[token * a.heads + head] = l == 0.0f ? neg_inf() : m * kLn2 + logf(l);
    }
  }
}

// Before its wait for the kernels whose splits it joins, the kernel below reads
// nothing but the caller's lengths and bounds. They are no work of those kernels,
// the first of which was launched to wait for everything before it, so they were
// complete, and written back, before it began. Read after the wait they
// lengthen the chain of loads: 46.3 -> 47.4 us for 64 contexts of 1000, 55.4 -> 57.6
// for 40 sequences of up to 3 new tokens behind 8000.
//
// Joins the splits of every row that has more than one: with M = max_z m_z,
//   out = sum_z 2^(m_z - M) o_z / sum_z 2^(m_z - M) l_z.
// WARPS warps to a row: all weights first, at once, then each warp adds every
// WARPS-th split, four loads in flight, and the warps' sums are added in order.
// One warp where the splits are few and the rows many, a CTA of eight where a
// row has many splits (two rows of 64 heads and 39 splits took 100 us with one
// warp to a row, one load after another). Bound by the latency of three loads
// in a row; the L2 holds the partial results.
constexpr int kMaxSplits = 256;

template <typename T, int WARPS>
__global__ void __launch_bounds__(kThreads) combine_kernel(AttnArgs a, AttnGeometry small, int64_t small_rows,
                                                           AttnGeometry large) {
  constexpr int kRows = kThreads / 32 / WARPS;  // rows of a CTA
  __shared__ float s_w[kRows][kMaxSplits];
  __shared__ float s_red[kRows][WARPS][2];
  __shared__ float s_o[WARPS > 1 ? WARPS : 1][WARPS > 1 ? 256 : 1];
  const int lane = threadIdx.x & 31, group = threadIdx.x / (32 * WARPS), tid = threadIdx.x % (32 * WARPS), warp = tid >> 5;
  const auto sync = [] {
    if (WARPS == 1) {
      __syncwarp();
    } else {
      __syncthreads();
    }
  };
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group;
  // (every thread waits for the kernels before, whatever it finds: later kernels on the stream count on this one's end alone)
  if (row >= a.tokens * a.heads) {
    pdl_wait();
    return;
  }
  const int64_t token = row / a.heads;
  const int head = static_cast<int>(row - token * a.heads);
  const int s = a.b.cu_q ? warp_last_le(a.b.seqs, token, [&](int i) { return first_row(a.b, i); })
                         : static_cast<int>(token);
  const int64_t first = first_row(a.b, s), all = (first_row(a.b, s + 1) - first) * a.group;
  const AttnGeometry& g = all <= small_rows ? small : large;
  AttnTile t;
  tile_at(a, g, s, ((token - first) * a.group + head % a.group) / g.rows, &t);
  pdl_wait();
  if (token < first || (token - first) * a.group >= all || t.rows == 0 || t.splits == 1) return;  // (some rows are no sequence's)
  const int64_t step = a.tokens * a.heads;  // from one split to the next
  const float2* ml = a.part_ml + row;
  float top = neg_inf();
  for (int z = tid; z < t.splits; z += 32 * WARPS) top = fmaxf(top, ml[z * step].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (WARPS > 1) {
    if (lane == 0) s_red[group][warp][0] = top;
    sync();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_red[group][w][0]);
  }
  float sum = 0.0f;
  for (int z = tid; z < t.splits; z += 32 * WARPS) {
    const float2 x = ml[z * step];
    const float w = x.x == neg_inf() ? (x.y == 0.0f ? 0.0f : 1.0f) : exp2f(x.x - top);  // (NaN scores alone: m = -inf, l = NaN)
    s_w[group][z] = w;
    sum += x.y * w;
  }
  sum = warp_sum(sum);
  if (WARPS > 1 && lane == 0) s_red[group][warp][1] = sum;
  sync();
  if (WARPS > 1) {
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += s_red[group][w][1];
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  T* dst = static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs;
  if (a.dim % 4 == 0) {
    for (int d = lane * 4; d < a.dim; d += 128) {
      const float* src = a.part_o + row * a.dim + d;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int z = warp; z < t.splits; z += WARPS) {
        const float4 y = *reinterpret_cast<const float4*>(src + z * step * a.dim);
        const float w = s_w[group][z];
        x.x = fmaf(y.x, w, x.x);
        x.y = fmaf(y.y, w, x.y);
        x.z = fmaf(y.z, w, x.z);
        x.w = fmaf(y.w, w, x.w);
      }
      if (WARPS > 1) {
        *reinterpret_cast<float4*>(&s_o[warp][d]) = x;
      } else {
        stf(dst + d, x.x * f);
        stf(dst + d + 1, x.y * f);
        stf(dst + d + 2, x.z * f);
        stf(dst + d + 3, x.w * f);
      }
    }
  } else {
    for (int d = lane; d < a.dim; d += 32) {
      float x = 0.0f;
#pragma unroll 4
      for (int z = warp; z < t.splits; z += WARPS) x = fmaf(a.part_o[(z * step + row) * a.dim + d], s_w[group][z], x);
      if (WARPS > 1) {
        s_o[warp][d] = x;
      } else {
        stf(dst + d, x * f);
      }
    }
  }
  if (WARPS > 1) {
    sync();
    for (int d = tid; d < a.dim; d += 32 * WARPS) {
      float x = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) x += s_o[w][d];
      stf(dst + d, x * f);
    }
  }
  if (tid == 0 && a.lse) a.lse[row] = sum == 0.0f ? neg_inf() : top * kLn2 + logf(sum);
}

// ------------------------------------------------------------------- host --

struct Plan {
  bool tile;           // all sequences by hc_attn_tile.cu; the rest does not matter then
  AttnGeometry small, large;
  bool use_large;      // sequences of more than kSmallRows rows go to the large tiles
  bool rows_kernel;    // small tiles by hc_attn_rows.cu
  RowsSchedule pieces; // which splits single-token sequences itself; units 0: the splits below
  bool f32_kernel;     // large tiles by hc_attn_f32.cu, and then no small ones
  int splits;          // the larger of the two
};

constexpr int kSmallRows = 16;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int64_t slots_of(const hc_paged_attention_t& a, int rows) {
  const int64_t group = a.heads / a.kv_heads;
  return a.tokens * group / rows + a.seqs;
}

// Keys of a split: the longest piece that still gives every SM `per_sm` CTAs,
// if all sequences were as long as the longest can be.
void set_splits(AttnGeometry* g, const hc_paged_attention_t& a, int64_t keys, int64_t tiles, int num_sms, int per_sm,
                int64_t shortest) {
  const int64_t want = std::max<int64_t>(1, ceil_div(static_cast<int64_t>(num_sms) * per_sm, tiles * a.kv_heads));
  int64_t len = std::max<int64_t>(shortest, ceil_div(keys, want));
  len = ceil_div(len, g->align) * g->align;
  g->split_len = static_cast<int>(std::min<int64_t>(len, int64_t{1} << 30));
  g->splits = static_cast<int>(std::max<int64_t>(1, ceil_div(keys + (a.window > 0 ? g->align : 0), g->split_len)));
  if (g->splits > kMaxSplits) {
    g->splits = kMaxSplits;
    g->split_len =
        static_cast<int>(std::min<int64_t>(ceil_div(ceil_div(keys, kMaxSplits), g->align) * g->align, int64_t{1} << 30));
  }
}

// Kernels for a call. Where no sequence has more than 16 rows (single tokens
// of up to 16 grouped heads), the small tiles serve all: they read keys at the
// rate of memory, and a tile of 256 rows would be empty. Anything longer goes
// to the tile kernel with all sequences of the batch, where type, head size and
// page size allow it; its single tokens cost it less than a second kernel.
// Otherwise small and large general tiles share the sequences.
Plan plan_of(const hc_paged_attention_t& a, bool aligned, int num_sms) {
  Plan p = {};
  const bool fast = !(a.flags & HC_FLAG_FORCE_GENERAL);
  const int64_t group = a.heads / a.kv_heads;
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
  const int64_t max_kv = a.max_kv > 0 ? std::min<int64_t>(a.max_kv, cap) : cap;
  const int64_t max_q = a.cu_q == nullptr ? 1 : a.max_q > 0 ? std::min<int64_t>(a.max_q, a.tokens) : a.tokens;
  const bool few = max_q * group <= kSmallRows;
  p.splits = 1;
  p.tile = !few && fast && attn_tile_supported(a.dtype, a.head_dim, a.page_size, a.scale, aligned);
  if (p.tile) return p;
  p.rows_kernel = fast && attn_rows_supported(a.dtype, a.head_dim, a.cu_q == nullptr, static_cast<int>(group), aligned);
  p.f32_kernel = fast && attn_f32_supported(a.dtype, a.head_dim, aligned);
  p.use_large = !few;
  p.small = AttnGeometry{kSmallRows, kKeys, 0, 0};
  p.large = AttnGeometry{64, kKeys, 0, 0};
  const auto keys_of = [&](int rows) {
    const int64_t span = ceil_div(rows, group) + 1;
    return a.window > 0 ? std::min<int64_t>(max_kv, a.window + span) : max_kv;
  };
  if (p.rows_kernel && few && a.cu_q == nullptr)
    p.pieces = attn_rows_schedule(a.seqs, a.kv_heads, keys_of(p.small.rows), num_sms);
  if (p.pieces.units > 0 || p.pieces.clusters) {
    p.small.split_len = 1 << 30;
    p.small.splits = 1;
    return p;
  }
  set_splits(&p.small, a, keys_of(p.small.rows), a.seqs, num_sms, 8, 128);
  set_splits(&p.large, a, keys_of(p.large.rows), std::max<int64_t>(1, a.tokens * group / 64), num_sms, 4, 128);
  p.splits = std::max(p.small.splits, p.use_large ? p.large.splits : 1);
  return p;
}

// Rows of partial results.
size_t part_rows(const hc_paged_attention_t& a, const Plan& p) {
  if (p.pieces.units > 0) return static_cast<size_t>(p.pieces.units) * a.kv_heads * kSmallRows;
  return p.splits <= 1 ? 0 : static_cast<size_t>(p.splits) * a.tokens * a.heads;
}

size_t part_bytes(const hc_paged_attention_t& a, const Plan& p) {
  const size_t rows = part_rows(a, p);
  return align_up(rows * 8, 256) + align_up(rows * a.head_dim * 4, 256);
}

AttnArgs args_of(const hc_paged_attention_t& a) {
  AttnArgs d = {};
  d.q = a.q;
  d.k = a.k_cache;
  d.v = a.v_cache;
  d.out = a.out;
  d.lse = a.lse;
  d.b = BatchView{a.page_table, a.kv_lens, a.cu_q, a.table_stride, a.num_pages, a.seqs, a.max_pages, a.page_size, a.tokens};
  d.tokens = a.tokens;
  d.q_ts = a.q_token_stride;
  d.q_hs = a.q_head_stride;
  d.o_ts = a.out_token_stride;
  d.o_hs = a.out_head_stride;
  d.c_ps = a.cache_page_stride;
  d.c_ts = a.cache_token_stride;
  d.c_hs = a.cache_head_stride;
  d.heads = a.heads;
  d.kv_heads = a.kv_heads;
  d.group = a.heads / a.kv_heads;
  d.dim = a.head_dim;
  d.window = a.window;
  d.scale = a.scale;
  d.softcap = a.softcap;
  return d;
}

template <typename T, int ROWS, int DP, bool ASYNC>
cudaError_t general_a(const AttnArgs& d, int64_t slots, cudaStream_t s) {
  constexpr size_t smem = sizeof(GeneralSmem<ROWS, DP, ASYNC ? 2 : 1>);
  const cudaError_t e = ensure_smem<general_kernel<T, ROWS, DP, ASYNC>>(smem);
  if (e != cudaSuccess) return e;
  general_kernel<T, ROWS, DP, ASYNC>
      <<<dim3(static_cast<unsigned>(slots), d.kv_heads, d.g.splits), kThreads, smem, s>>>(d);
  return cudaGetLastError();
}

// float32 needs no conversion on its way in, so aligned rows come asynchronously.
template <typename T, int ROWS, int DP>
cudaError_t general_t(const AttnArgs& d, bool aligned, int64_t slots, cudaStream_t s) {
  if constexpr (std::is_same<T, float>::value) {
    if (aligned && d.dim % 4 == 0) return general_a<T, ROWS, DP, true>(d, slots, s);
  }
  return general_a<T, ROWS, DP, false>(d, slots, s);
}

template <typename T, int ROWS>
cudaError_t general_d(const AttnArgs& d, bool aligned, int64_t slots, cudaStream_t s) {
  if (d.dim <= 64) return general_t<T, ROWS, 64>(d, aligned, slots, s);
  if (d.dim <= 128) return general_t<T, ROWS, 128>(d, aligned, slots, s);
  return general_t<T, ROWS, 256>(d, aligned, slots, s);
}

template <typename T>
cudaError_t launch_t(const hc_paged_attention_t& a, bool aligned, int num_sms, cudaStream_t s) {
  const Plan p = plan_of(a, aligned, num_sms);
  AttnArgs d = args_of(a);
  if (const size_t rows = part_rows(a, p)) {
    d.part_ml = static_cast<float2*>(a.workspace);
    d.part_o = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + align_up(rows * 8, 256));
  }
  if (p.tile) return launch_attn_tile(d, a.dtype, a.workspace, num_sms, s);
  // Sequences of at most small_rows rows go to the small tiles, the others to the large ones (hc_attn_f32.cu takes all of a batch
  // that has any longer). Where there are both kinds, a sequence's one small tile is the slot of its number.
  const int64_t small_rows = !p.use_large ? INT64_MAX : p.f32_kernel ? 0 : kSmallRows;
  cudaError_t e = cudaSuccess;
  if (small_rows > 0) {
    const int64_t slots = p.use_large ? a.seqs : slots_of(a, p.small.rows);
    d.g = p.small;
    d.min_rows = 1;
    d.max_rows = small_rows;
    d.slot_is_seq = p.use_large;
    d.clears = !p.use_large && a.cu_q != nullptr;
    d.spare_ctas = p.pieces.spare_ctas;
    d.units = p.pieces.units;
    d.clusters = p.pieces.clusters;
    e = p.rows_kernel ? launch_attn_rows(d, a.dtype, slots, s) : general_d<T, kSmallRows>(d, aligned, slots, s);
    if (e != cudaSuccess) return e;
  }
  if (p.use_large) {
    d.g = p.large;
    d.slot_is_seq = false;
    d.clears = a.cu_q != nullptr;
    d.min_rows = small_rows + 1;
    d.max_rows = INT64_MAX;
    const int64_t slots = slots_of(a, p.large.rows);
    e = p.f32_kernel ? launch_attn_f32(d, slots, s) : general_d<T, 64>(d, aligned, slots, s);
    if (e != cudaSuccess) return e;
  }
  if (p.splits > 1) {
    const int64_t rows = a.tokens * a.heads;
    if (p.splits > 8 && rows < 4096) {
      e = launch_pdl(combine_kernel<T, 8>, dim3(static_cast<unsigned>(rows)), dim3(kThreads), 0, s, 1, d, p.small,
                     small_rows, p.large);
    } else {
      e = launch_pdl(combine_kernel<T, 1>, dim3(static_cast<unsigned>(ceil_div(rows, kThreads / 32))), dim3(kThreads), 0, s,
                     1, d, p.small, small_rows, p.large);
    }
  }
  return e;
}

}  // namespace

size_t attention_workspace(const hc_paged_attention_t& a, bool aligned, int num_sms) {
  const Plan p = plan_of(a, aligned, num_sms);
  if (p.tile) return attn_tile_workspace(a.tokens, a.heads / a.kv_heads, a.seqs, a.head_dim, num_sms);
  return part_bytes(a, p);
}

cudaError_t launch_attention(const hc_paged_attention_t& a, bool aligned, int num_sms, cudaStream_t s) {
  switch (a.dtype) {
    case HC_F32: return launch_t<float>(a, aligned, num_sms, s);
    case HC_F16: return launch_t<__half>(a, aligned, num_sms, s);
    default: return launch_t<__nv_bfloat16>(a, aligned, num_sms, s);
  }
}

}  // namespace hc
