// Attention over a paged cache for many rows (fp16/bf16, heads of 64 or 128,
// pages that divide 128 keys or are whole multiples of them): chunks of a
// prompt, and batches that mix chunks with single tokens.
//
// Mathematics: per tile of rows, over key blocks j of 128,
//   S = Q K_j^T;  P = 2^(S c - m);  l += sum P;  O += P V_j
// with the running maximum m of each row. O is rescaled (O, l *= 2^(m - m'))
// only when a row's maximum has risen by more than 8 (a factor of 256) above
// the m in use: weights up to 2^8 are as precise in either type as weights up to
// one, so most blocks touch O with nothing but the MMA. P is rounded to T for its
// product (the tensor core's operands are 16 bits, and a second product with what
// the rounding leaves would add half to the MMAs' time); l sums the weights before
// that. So a result is off by 2.3e-3 of its size against 64 bits in bf16 (2.9e-4 in
// fp16) where its own rounding is 1.7e-3 (2.1e-4).
//
// Bound: the tensor cores, 4 * head_dim flops for each pair of row and key.
// One CTA per SM holds two tiles, A and B, of 128 rows. Both products run on
// tcgen05: S = Q K^T from shared memory into tensor memory (128 columns for
// each tile), and O += P V with P read from tensor memory, where it takes the
// place of the S it came from (the MMAs of one thread run in the order of their
// issue, so QK(j+1) does not overtake PV(j)). The MMA warp issues PV_A(j), QK_A(j+1),
// PV_B(j), QK_B(j+1) in turn, so that while the softmax warps of one tile work,
// the tensor core has the other tile's two products to do (with a warp for each
// tile the two fell into step, and products and softmax took turns). Two warpgroups do
// the softmax, a thread to a row (no exchange between lanes); one warp copies
// keys and values by TMA, a box per page and 64 features, into a ring. Of the
// 168 * 384 registers that the CTA starts with, the softmax threads take 216
// each, so that a row's 128 scores stay in them, and the others 72
// (2 * 128 * 216 + 128 * 72 = 384 * 168).
//
// Measured: 2047 tokens behind 28001, 32 heads of 128 on 8, bf16: 643 us call after
// call, where it meets the power limit (1.51 PFLOP/s, 79% of the measured burst rate
// and 87% of the sustained one; 640 to 680 from one GPU to the next), 567 us for a few
// calls from rest (1.71 PFLOP/s, 89% of burst); with scores capped at 50 875 us. 17
// sequences of 1 to 301 tokens, window 1000, scores capped at 30, 20 heads of 64 on 4,
// fp16: 66 us, of which some 15 are plan, start and joining; a block of keys takes a
// tile pair of 64 features about 1.7 us then, the capped scores' multiply-adds and
// exponentials of two warps to a scheduler (47 us without the cap, 107 where scores
// pass 3/5 of it).
//
// Work: all tiles' key blocks, for all key heads, laid end to end with four
// units before each tile for its queries and results, are cut into equal runs,
// one for each SM (hc_attn.cuh's slots give the tiles, plan_kernel their prefix
// sums); a cut among those units moves to the tile's start. A tile that a cut goes through is written as partial
// sums by every CTA that has a piece of it and joined by join_kernel; at most
// two pieces to a CTA are of that kind. So a long prompt, many short ones and one
// short chunk over a long context all fill the GPU, without a choice of split.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "hc_async.cuh"
#include "hc_attn_internal.h"
#include "hc_tc.cuh"

namespace hc {
namespace {

constexpr int kRows = 128;        // rows of a tile, an MMA's M
constexpr int kPair = 2 * kRows;  // rows of a CTA's two tiles
constexpr int kKeys = 128;        // keys of a block, N of the first product
constexpr int kThreads = 384;     // two softmax warpgroups, and one of the other warps
constexpr int kLoadWarp = 8, kMmaWarp = 9, kFixWarp = 10;  // (and 11 plans)
constexpr int kSegs = 4;          // segments at hand
constexpr int kSegUsers = 11;     // warps that read them
constexpr int kTileCost = 4;      // what a tile costs beside its key blocks (queries in, results out), in blocks
constexpr float kLazy = 8.0f;     // rise of a row's maximum (base-2) that O is rescaled for

__device__ unsigned int g_tile_wait_timeouts = 0;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;             // boxes of 64 features
  static constexpr int kHalf = kKeys * 128;          // bytes of one such box of 128 rows
  static constexpr int kSlot = kHalves * kHalf;      // a block's keys or values
  static constexpr int kSlots = D == 128 ? 4 : 6;
  static constexpr int kQ = kHalves * kRows * 128;   // one tile's queries
  static constexpr int kStage = 8 * 32 * 128;        // results on their way out, 128 bytes of each row
  static constexpr int kSmem = 2 * kQ + kSlots * kSlot + kStage + 1024;
};

// A tile that a cut goes through, for the kernel that joins its pieces.
struct JoinTile {
  AttnTile t;
  int kv_head, pieces;  // pieces of the CTAs from this one on; 0: none to join here
};

struct Work {
  const AttnTile* tiles;  // tile of each slot
  const int64_t* prefix;  // units of the tiles before each slot, per key head; [slots] = all (4 million tokens of 16 grouped heads have 2^32)
  int slots, ctas;
  JoinTile* joins;        // of each CTA, the tile that its run ends in, if that is the first cut in it
  float2* part_ml;        // [2 * ctas][kPair]
  float* part_o;          // [2 * ctas][kPair][dim]
};

// --------------------------------------------------------------- schedule --

__device__ __forceinline__ int64_t blocks_of(const AttnTile& t) {
  const int64_t n = (t.hi - t.base + kKeys - 1) / kKeys;
  return n < 1 ? 1 : n;  // a tile that sees nothing still writes its zeros
}

// The tile of every slot, and the units of all before it.
__global__ void __launch_bounds__(1024) plan_kernel(AttnArgs a, int64_t* prefix, AttnTile* tiles, int slots) {
  __shared__ int64_t red[33];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < slots; i += 1024) prefix[i] = 0;
  __syncthreads();
  for (int s = warp; s < a.b.seqs; s += 32) {
    const int64_t first = first_row(a.b, s), next = first_row(a.b, s + 1);
    const int64_t lo = first * a.group / kPair + s, hi = next * a.group / kPair + s + 1;
    for (int64_t i = lo + lane; i < hi; i += 32) {
      AttnTile t;
      tile_at(a, a.g, s, i - lo, &t);
      if (i < slots) tiles[i] = t;
      if (i < slots) prefix[i] = t.rows == 0 ? 0 : kTileCost + static_cast<int>(blocks_of(t));
    }
  }
  __syncthreads();
  // exclusive prefix in place, 1024 slots at a time
  int64_t before = 0;
  for (int i0 = 0; i0 <= slots; i0 += 1024) {
    const int i = i0 + threadIdx.x;
    const int64_t v = i < slots ? prefix[i] : 0;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    if (warp == 0) {
      const int64_t w = red[lane];
      int64_t z = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, z, o);
        if (lane >= o) z += y;
      }
      red[lane] = z - w;
      if (lane == 31) red[32] = z;
    }
    __syncthreads();
    if (i <= slots) prefix[i] = before + red[warp] + x - v;
    before += red[32];
    __syncthreads();
  }
}

// The run of units that CTA c has, out of all: [start(c), start(c + 1)).
struct Run {
  int64_t per_head, all;
  int ctas;
  __device__ Run(const Work& w, int kv_heads) {
    per_head = w.prefix[w.slots];
    all = per_head * kv_heads;
    const int64_t most = all / (kTileCost + 1);  // a tile of one block to a CTA, where there is no more
    ctas = static_cast<int>(most < 1 ? 1 : most < w.ctas ? most : w.ctas);
  }
  __device__ int64_t start(int c) const { return all * c / ctas; }
};

// A CTA's piece of one tile pair: blocks [j0, j1) of its n; none: the run's end.
struct Segment {
  AttnTile t;
  int kv_head, j0, j1, n;
  int all_from, all_to;  // keys that every row of the pair sees, from the tile's first block on
  int64_t at;            // unit of the tile's first block
};
// Whether a block of keys holds some that not every row of the tile pair sees.
__device__ __forceinline__ bool at_edge(const Segment& g, int j) {
  return j * kKeys < g.all_from || (j + 1) * kKeys > g.all_to;
}

// The segment that unit u of all lies in, of a run that ends at u1 (full warps).
__device__ __forceinline__ void segment_at(const Work& w, const Run& run, int64_t u, int64_t u1,
                                           Segment* g) {
  const int h = static_cast<int>(u / run.per_head);
  const int64_t v = u - h * run.per_head;
  const int slot = warp_last_le(w.slots, v, [&](int i) { return w.prefix[i]; });
  g->t = w.tiles[slot];
  g->kv_head = h;
  g->at = h * run.per_head + w.prefix[slot] + kTileCost;
  g->n = static_cast<int>(w.prefix[slot + 1] - w.prefix[slot]) - kTileCost;
  const int64_t from = u - g->at, to = u1 - g->at;
  g->j0 = from < 0 ? 0 : static_cast<int>(from);
  g->j1 = to < 0 ? 0 : to < g->n ? static_cast<int>(to) : g->n;
}

// What is to be joined of the tile that cut c + 1 goes through, if that is the first cut in it (full warps).
__device__ __forceinline__ JoinTile join_at(const Work& w, const Run& run, int c) {
  JoinTile j = {};
  if (c + 1 < run.ctas) {
    Segment g;
    segment_at(w, run, run.start(c + 1), run.all, &g);
    if (g.j0 > 0 && run.start(c) <= g.at) {
      j.t = g.t;
      j.kv_head = g.kv_head;
      for (j.pieces = 1; c + j.pieces < run.ctas && run.start(c + j.pieces) < g.at + g.n;) ++j.pieces;
    }
  }
  return j;
}

// Blocks of tile x (0: A, 1: B) of a pair: those up to the last key its last row sees.
__device__ __forceinline__ int tile_rows(const AttnTile& t, int x) {
  const int r = t.rows - x * kRows;
  return r < 0 ? 0 : r < kRows ? r : kRows;
}
__device__ __forceinline__ int tile_blocks(const AttnArgs& a, const AttnTile& t, int x) {
  const int rows = tile_rows(t, x);
  if (rows == 0) return 0;
  const int64_t end = row_position(t, t.row0 + x * kRows + rows - 1, a.group) + 1;
  const int64_t n = (end - t.base + kKeys - 1) / kKeys;
  return n < 1 ? 1 : static_cast<int>(n);
}

// ------------------------------------------------------------ tensor memory --

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Marks registers that an asynchronous load filled as written here, after its wait.
__device__ __forceinline__ void landed32(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                   "+r"(r[i + 6]), "+r"(r[i + 7]));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], issued by one thread; A holds pairs of
// 16-bit elements of a row in each 32-bit column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
  return d;
}
__device__ __forceinline__ float min3(float x, float y, float z) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
  return d;
}
// x * y + z on two floats at once.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return d;
}
// Scores inside a cap: map_score's polynomial in x, scale / c worked into its
// coefficients: five operations on pairs of floats that leave the exponential
// unit to the softmax. A score of minus infinity, which stands for a key that
// is not seen, stays one: the highest coefficient is positive. Where a
// coefficient may have lost its precision below float32's normal range, or pass
// the range, scores go through map_score: with |x| <= 1.8e4 what is lost of the
// smallest (2^-149 x^8) is below 1e-7 of scale.
struct CapPoly {
  float c[5];
  float most;  // largest |x|
  bool all;    // that is, all that have |y| <= kCapTurn
};
__device__ __forceinline__ CapPoly cap_poly(float scale, float softcap) {
  const float k = scale / softcap, k2 = k * k, k4 = k2 * k2, c = scale * kLog2e;
  const bool fits = scale >= 1e-4f && scale <= 1e4f && k <= 1e3f;
  return CapPoly{{c * kCap0, c * k2 * kCap1, c * k4 * kCap2, c * k4 * k2 * kCap3, fmaxf(c * k4 * k4 * kCap4, 1e-45f)},
                 fits ? fminf(kCapTurn / k, 1.8e4f) : -1.0f,
                 fits && kCapTurn / k <= 1.8e4f};
}
__device__ __forceinline__ float2 cap_factor(const CapPoly& p, float2 x) {
  const auto twice = [](float v) { return make_float2(v, v); };
  const float2 u = fma2(x, x, twice(0.0f));
  float2 y = fma2(twice(p.c[4]), u, twice(p.c[3]));
  y = fma2(y, u, twice(p.c[2]));
  y = fma2(y, u, twice(p.c[1]));
  return fma2(y, u, twice(p.c[0]));
}

// Any score, less `ref`: the bits of fma2(x, cap_factor(x), -ref) where that holds.
template <bool ALL>  // poly.all
__device__ __forceinline__ float cap_exponent(const CapPoly& p, const ScoreMap& m, float x, float ref) {
  const float near = fmaf(x, cap_factor(p, make_float2(x, x)).x, -ref);
  const float far = (ALL ? cap_beyond(m, x * m.k) : map_score(m, x)) - ref;
  return fabsf(x) <= p.most ? near : far;
}

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

// ----------------------------------------------------------------- kernel --

// Infinite or NaN values at keys that only some of a tile's rows see. The copy of the
// values that the product reads has zeros in their place (a weight of zero must
// meet a finite value), and a bit stands for each key that has any; the rows that
// see such a key read its value again at the end and add what is not finite there,
// where any weight above zero gives the same infinity or NaN.
constexpr int kOddBlocks = 8;  // of a tile: its rows' views begin within three blocks, and end within three
struct OddValues {
  int any, blocks;
  int block[kOddBlocks];               // blocks that not all rows see
  uint32_t keys[kOddBlocks][4];        // and their keys with such values
};

struct Bars {
  uint64_t q_full[2];   // a tile's queries lie in shared memory
  uint64_t s_full[2];   // its scores lie in tensor memory
  uint64_t p_full[2];   // its weights do, and O may be added to
  uint64_t o_done[2];   // the product with the values is done
  uint64_t kv_full[8], kv_empty[8];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t odd_full[kSegs];  // a segment's odd values are all listed
  uint64_t edge[8];     // values that not all rows see have landed and are yet to be cleaned
  uint32_t tmem;
};

// A wait that gave up ends its role's loop; the other roles' next waits give
// up in turn, and the rows of the tile at hand become NaN.
#define HC_WAIT(bar, parity)                                                                         \
  do {                                                                                               \
    if (!__all_sync(0xffffffffu, mbar_wait((bar), (parity), &g_tile_wait_timeouts))) return false;   \
  } while (0)

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

template <typename T, int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ Work w,
                const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using C = Cfg<D>;
  extern __shared__ unsigned char raw[];
  __shared__ Bars bars;
  __shared__ Segment segs[kSegs];
  __shared__ OddValues odd[kSegs];
  unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  unsigned char* const ring = smem + 2 * C::kQ;
  // (through a shuffle the compiler knows that a warp's threads agree on it, and keeps what follows from it in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars.q_full[x], kRows);
      mbar_init(&bars.s_full[x], 1);
      mbar_init(&bars.p_full[x], 4);  // a warp each
      mbar_init(&bars.o_done[x], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars.seg_full[i], 1);
      mbar_init(&bars.seg_empty[i], kSegUsers);
      mbar_init(&bars.odd_full[i], 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&bars.kv_full[i], 1);
      mbar_init(&bars.kv_empty[i], 1);
      mbar_init(&bars.edge[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars.tmem, 512);
    tmem_relinquish();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&k_map);
    tma_prefetch_desc(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_wait();
  pdl_trigger();  // (after the wait: join_kernel may read the plan before its own)
  // tensor memory: S (and P) of A and B, then O of A and B
  constexpr uint32_t kO = 2 * kKeys;

  // Segment i of this CTA's run, worked out by the plan warp ahead of the others
  // (a chain of loads through the schedule and the batch that nobody else waits for).
  const auto done_with = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.seg_empty[i % kSegs]);
  };
#define HC_SEGMENT(i) HC_WAIT(&bars.seg_full[(i) % kSegs], ((i) / kSegs) & 1)

  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kLoadWarp) {
      // ---- copies: for each segment K(j0), V(j0), K(j0+1), ... ----
      const int page = a.b.page_size;
      const int box = page < kKeys ? page : kKeys;       // tokens of a copy
      const int boxes = kKeys / box * C::kHalves;        // copies of a block's keys
      int slot = 0;
      uint32_t round = 0;
      const auto copy_all = [&]() -> bool {
        for (int seg = 0;; ++seg) {
          HC_SEGMENT(seg);
          const Segment& g = segs[seg % kSegs];
          if (g.j1 <= g.j0) return true;
          for (int j = g.j0; j < g.j1; ++j) {
            const int64_t key0 = g.t.base + static_cast<int64_t>(j) * kKeys;
            // pages of this lane's copies; a box without a key that any row sees lies outside the pool, and reads zeros
            int at[2] = {-1, -1};
            int off[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int b = (lane + 32 * i) / C::kHalves;
              const int64_t key = key0 + b * box;
              if (lane + 32 * i < boxes && key < g.t.hi && key + box > g.t.lo) {
                const uint32_t e = static_cast<uint32_t>(key) / static_cast<uint32_t>(page);
                at[i] = page_of(a.b, g.t.s, e);
                off[i] = static_cast<int>(static_cast<uint32_t>(key) - e * page);
              }
            }
            for (int kind = 0; kind < 2; ++kind) {
              HC_WAIT(&bars.kv_empty[slot], (round & 1) ^ 1);
              uint64_t* const full = kind == 1 && at_edge(g, j) ? &bars.edge[slot] : &bars.kv_full[slot];
              if (lane == 0) mbar_arrive_expect_tx(full, C::kSlot);
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int e = lane + 32 * i;
                if (e < boxes) {
                  const int h = e % C::kHalves, b = e / C::kHalves;
                  tma_load_4d(smem_addr(ring + slot * C::kSlot + h * C::kHalf) + b * box * 128, kind ? &v_map : &k_map,
                              h * 64, off[i], g.kv_head, at[i] < 0 ? static_cast<int>(a.b.num_pages) : at[i],
                              full);
                }
              }
              if (++slot == C::kSlots) {
                slot = 0;
                ++round;
              }
            }
          }
          done_with(seg);
        }
      };
      const bool ok = copy_all();
      // the CTA keeps its memory until the last copies have landed and the last products have read them
      for (int i = 0; i < C::kSlots; ++i) {
        const uint32_t used = i < slot ? round : round - 1;
        if (i < slot || round > 0) {
          mbar_wait(&bars.kv_full[i], used & 1, nullptr);
          if (ok) mbar_wait(&bars.kv_empty[i], used & 1, &g_tile_wait_timeouts);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---- products ----
      constexpr uint32_t kQk = idesc_f16(std::is_same<T, __nv_bfloat16>::value, kRows, kKeys, false, false);
      constexpr uint32_t kPv = idesc_f16(std::is_same<T, __nv_bfloat16>::value, kRows, D, false, true);
      const uint64_t q_desc = smem_desc_sw128(smem_addr(smem), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_addr(ring), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_addr(ring), C::kHalf, 1024);
      int slot = 0;
      uint32_t round = 0, q_seen[2] = {0, 0}, p_seen[2] = {0, 0};
      const auto advance = [&] {
        if (++slot == C::kSlots) {
          slot = 0;
          ++round;
        }
      };
      // (descriptors count addresses in 16 bytes)
      const auto issue_qk = [&](int x, int k_slot) {
        const uint64_t q = q_desc + static_cast<uint32_t>(x * (C::kQ / 16));
        const uint64_t k = k_desc + static_cast<uint32_t>(k_slot * (C::kSlot / 16));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t o = ((ks / 4) * C::kHalf + (ks % 4) * 32) / 16;
          mma_f16(tmem + x * kKeys, q + o, k + o, kQk, ks > 0);
        }
        mma_commit(&bars.s_full[x]);
      };
      const auto issue_pv = [&](int x, int v_slot, bool add) {
        const uint64_t v = v_desc + static_cast<uint32_t>(v_slot * (C::kSlot / 16));
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          mma_f16_ts(tmem + kO + x * D, tmem + x * kKeys + ks * 8, v + ks * (2048 / 16), kPv, add || ks > 0);
        mma_commit(&bars.o_done[x]);
      };
      const auto multiply_all = [&]() -> bool {
        for (int seg = 0;; ++seg) {
          HC_SEGMENT(seg);
          const Segment& g = segs[seg % kSegs];
          const int j0 = g.j0, j1 = g.j1;
          if (j1 <= j0) return true;
          const int ends[2] = {min(tile_blocks(a, g.t, 0), j1), min(tile_blocks(a, g.t, 1), j1)};
          done_with(seg);
          HC_WAIT(&bars.kv_full[slot], round & 1);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (j0 < ends[x]) {
              HC_WAIT(&bars.q_full[x], q_seen[x] & 1);
              ++q_seen[x];
              tc_fence_after();
              if (elect_one()) issue_qk(x, slot);
              __syncwarp();
            }
          if (elect_one()) mma_commit(&bars.kv_empty[slot]);
          __syncwarp();
          advance();
          HC_WAIT(&bars.kv_full[slot], round & 1);
          for (int j = j0; j < j1; ++j) {
            // block j's values are there, block j+1's keys and values are waited for while products are queued
            const int v_slot = slot;
            advance();
            const int k_slot = slot;
            const uint32_t k_round = round;
            const bool more = j + 1 < j1;
            if (more) advance();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (j < ends[x]) {
                HC_WAIT(&bars.p_full[x], p_seen[x] & 1);
                ++p_seen[x];
                tc_fence_after();
                if (elect_one()) issue_pv(x, v_slot, j > j0);
              }
              if (x == 1 && elect_one()) mma_commit(&bars.kv_empty[v_slot]);
              __syncwarp();
              if (more) {
                if (x == 0) HC_WAIT(&bars.kv_full[k_slot], k_round & 1);
                if (j + 1 < ends[x] && elect_one()) issue_qk(x, k_slot);
                if (x == 1 && elect_one()) mma_commit(&bars.kv_empty[k_slot]);
                __syncwarp();
                if (x == 1) HC_WAIT(&bars.kv_full[slot], round & 1);
              }
            }
          }
        }
      };
      multiply_all();
    } else if (warp == kFixWarp) {
      // ---- values that not all rows see: zeros for those that none sees, and for what is not finite ----
      int slot = 0;
      uint32_t edges = 0;  // parity of each slot's edge barrier
      const auto fix_all = [&]() -> bool {
        for (int seg = 0;; ++seg) {
          HC_SEGMENT(seg);
          const Segment& g = segs[seg % kSegs];
          if (g.j1 <= g.j0) return true;
          OddValues& list = odd[seg % kSegs];
          if (lane == 0) list.any = list.blocks = 0;
          int blocks = 0;
          __syncwarp();
          for (int j = g.j0; j < g.j1; ++j) {
            const int v_slot = slot + 1 == C::kSlots ? 0 : slot + 1;
            slot = v_slot + 1 == C::kSlots ? 0 : v_slot + 1;
            const int64_t key0 = g.t.base + static_cast<int64_t>(j) * kKeys;
            if (!at_edge(g, j)) continue;
            HC_WAIT(&bars.edge[v_slot], edges >> v_slot & 1);
            edges ^= 1u << v_slot;
            uint32_t* const odd_keys = list.keys[min(blocks, kOddBlocks - 1)];
            if (lane < 4) odd_keys[lane] = 0;
            if (lane == 0) list.block[min(blocks, kOddBlocks - 1)] = j;
            ++blocks;
            __syncwarp();
            // rows of the block: none sees those before lo and from hi on, not all those before sure_lo and from sure_hi on
            const auto in_block = [&](int64_t key) { return static_cast<int>(max(min(key, static_cast<int64_t>(kKeys)), int64_t{0})); };
            const int lo = in_block(g.t.lo - key0), hi = in_block(g.t.hi - key0);
            const int sure_lo = in_block(g.all_from - j * kKeys), sure_hi = max(in_block(g.all_to - j * kKeys), sure_lo);
            constexpr int kPer = 8 * C::kHalves;  // 16-byte chunks of a row
            const int rows = sure_lo + kKeys - sure_hi;
            const auto place = [&](int e, int* r) {
              const int i = e / kPer, c = e & 7, h = (e >> 3) % C::kHalves;
              *r = i < sure_lo ? i : sure_hi + (i - sure_lo);
              return reinterpret_cast<uint4*>(ring + v_slot * C::kSlot + h * C::kHalf + *r * 128 + ((c ^ (*r & 7)) << 4));
            };
            // a half whose exponent is all ones carries into its sign's place
            constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
            constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
            uint32_t carry = 0;
#pragma unroll 8
            for (int e = lane; e < rows * kPer; e += 32) {
              int r;
              uint4* const at = place(e, &r);
              if (r < lo || r >= hi) {
                *at = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 v = *at;
                carry |= (v.x & kExp) + kOne | (v.y & kExp) + kOne | (v.z & kExp) + kOne | (v.w & kExp) + kOne;
              }
            }
            if (__any_sync(0xffffffffu, carry & 0x80008000u)) {
              for (int e = lane; e < rows * kPer; e += 32) {
                int r;
                uint4* const at = place(e, &r);
                const uint4 v = *at;
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const uint32_t half = w[i / 2] >> (16 * (i & 1)) & 0xffffu;
                  if (!not_finite2<T>(half)) continue;
                  list.any = 1;
                  atomicOr(&odd_keys[r >> 5], 1u << (r & 31));
                  w[i / 2] &= (i & 1) ? 0xffffu : 0xffff0000u;
                }
                *at = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.kv_full[v_slot]);
          }
          __syncwarp();
          if (lane == 0) {
            list.blocks = min(blocks, kOddBlocks);
            mbar_arrive(&bars.odd_full[seg % kSegs]);
          }
          done_with(seg);
        }
      };
      fix_all();
    } else {
      // ---- the run's segments, one after another ----
      const Run run(w, a.kv_heads);
      const auto plan_all = [&]() -> bool {
        const bool mine = static_cast<int>(blockIdx.x) < run.ctas;
        int64_t u = mine ? run.start(blockIdx.x) : 0;
        const int64_t u1 = mine ? run.start(blockIdx.x + 1) : 0;
        for (int seg = 0;; ++seg) {
          Segment g = {};
          if (u < u1) {
            segment_at(w, run, u, u1, &g);
            const int64_t first = row_position(g.t, g.t.row0, a.group) - g.t.base;
            const int64_t last = row_position(g.t, g.t.row0 + g.t.rows - 1, a.group) - g.t.base;
            g.all_to = static_cast<int>(first + 1 < 0 ? 0 : first + 1);
            g.all_from = static_cast<int>(a.window <= 0 || last - a.window + 1 < 0 ? 0 : last - a.window + 1);
          }
          HC_WAIT(&bars.seg_empty[seg % kSegs], ((seg / kSegs) & 1) ^ 1);
          if (lane == 0) {
            segs[seg % kSegs] = g;
            mbar_arrive(&bars.seg_full[seg % kSegs]);
          }
          __syncwarp();
          if (g.j1 <= g.j0) return true;
          u = g.at + g.n;
        }
      };
      plan_all();
      const JoinTile join = join_at(w, run, blockIdx.x);
      if (lane == 0) w.joins[blockIdx.x] = join;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // ---- softmax: warpgroup x has tile x, a thread to a row ----
    const int x = warp >> 2, row = threadIdx.x & (kRows - 1);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);  // this warp's 32 lanes
    const uint32_t s_at = lanes + x * kKeys, o_at = lanes + kO + x * D;
    const ScoreMap map = score_map(a.scale, a.softcap);
    const CapPoly poly = cap_poly(a.scale, CAP ? a.softcap : 1.0f);
    uint32_t s_seen = 0, o_seen = 0;
    // Queries of a segment's tile: a warp copies its 32 rows, whole rows side by side, and hands them over when they have landed.
    const auto fetch_q = [&](const Segment& sg) {
      if (sg.j0 >= min(tile_blocks(a, sg.t, x), sg.j1)) return false;
      int64_t at = -1;
      if (row < tile_rows(sg.t, x)) {
        int64_t token;
        int head;
        row_owner(a, sg.t, sg.kv_head, x * kRows + row, &token, &head);
        at = token * a.q_ts + head * a.q_hs;
      }
      constexpr int kChunks = D / 8, kAtOnce = 32 / kChunks;
      const int c = lane % kChunks;
      const uint32_t dst = smem_addr(smem + x * C::kQ + (c >> 3) * (kRows * 128));
#pragma unroll
      for (int i = 0; i < 32; i += kAtOnce) {
        const int from = i + lane / kChunks, r = (warp & 3) * 32 + from;
        const int64_t off = __shfl_sync(0xffffffffu, at, from);
        cp_async16_zfill(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                         static_cast<const T*>(a.q) + (off < 0 ? 0 : off) + c * 8, off < 0 ? 0 : 16);
      }
      cp_async_commit();
      return true;
    };
    const auto hand_q = [&] {
      cp_async_wait_all();
      fence_async_smem();
      mbar_arrive(&bars.q_full[x]);
    };
    // 128 bytes of each of the warp's rows, held a row to a lane, to where `place` says (element offset, -1: nowhere): through
    // shared memory, so that a store writes four rows' 128 bytes and not 16 bytes of 32 rows.
    unsigned char* const stage = ring + C::kSlots * C::kSlot + warp * (32 * 128);
    const auto write_out = [&](const uint32_t* y, unsigned char* base, int64_t place, bool wide) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
            make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      __syncwarp();
      const int c = lane & 7;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const int r = i + (lane >> 3);
        const int64_t off = __shfl_sync(0xffffffffu, place, r);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
        if (off < 0) continue;
        unsigned char* dst = base + off + c * 16;
        if (wide) {
          *reinterpret_cast<uint4*>(dst) = v;
        } else {
          const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            reinterpret_cast<uint16_t*>(dst)[e] = static_cast<uint16_t>(w4[e / 2] >> (16 * (e & 1)));
        }
      }
      __syncwarp();
    };
    float m = neg_inf(), l = 0.0f;
    int seg = 0;
    const auto softmax_all = [&]() -> bool {
      HC_SEGMENT(0);
      if (fetch_q(segs[0])) hand_q();
      for (;; ++seg) {
        const Segment& g = segs[seg % kSegs];
        if (g.j1 <= g.j0) return true;
        const int end = min(tile_blocks(a, g.t, x), g.j1);
        const int rows = tile_rows(g.t, x);
        // keys that this row sees, from the tile's first block on: [from, to); those that every row sees: [all_from, all_to)
        int from = 0, to = 0, all_from = 0, all_to = 0;
        if (rows > 0) {
          const int64_t r0 = g.t.row0 + x * kRows;
          const int64_t p0 = row_position(g.t, r0, a.group) - g.t.base, p1 = row_position(g.t, r0 + rows - 1, a.group) - g.t.base;
          const int64_t p = row_position(g.t, r0 + row, a.group) - g.t.base;
          const auto cut = [](int64_t v) { return static_cast<int>(v < 0 ? 0 : v); };
          // (rows past the last are computed along and never written; they are not masked)
          to = row < rows ? cut(p + 1) : INT32_MAX;
          from = row < rows && a.window > 0 ? cut(p - a.window + 1) : 0;
          all_to = cut(p0 + 1);
          all_from = a.window > 0 ? cut(p1 - a.window + 1) : 0;
        }
        m = neg_inf();
        l = 0.0f;
        for (int j = g.j0; j < end; ++j) {
          uint32_t s[kKeys];
          HC_WAIT(&bars.s_full[x], s_seen & 1);
          ++s_seen;
          tc_fence_after();
          const auto load_scores = [&] {
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) tmem_ld32(s_at + c, s + c);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) landed32(s + c);
          };
          load_scores();
          float* f = reinterpret_cast<float*>(s);
          // largest (and, to see whether all are inside the cap, smallest) score
          float tops[4], lows[4];
          const auto extremes = [&] {
#pragma unroll
            for (int i = 0; i < 4; ++i) tops[i] = fmaxf(f[2 * i], f[2 * i + 1]);
#pragma unroll
            for (int c = 8; c < kKeys; c += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) tops[i] = max3(tops[i], f[c + 2 * i], f[c + 2 * i + 1]);
            return fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
          };
          const int j0 = j * kKeys;
          const bool masked = j0 < all_from || j0 + kKeys > all_to;
          // (a bit for each key, so that a score costs one test: with two comparisons a score, the
          // batch of 17 sequences above took 79 us and not 71)
          const auto mask = [&] {
            const int lo = from - j0, hi = to - j0;
#pragma unroll
            for (int h = 0; h < kKeys; h += 32) {
              const int below = min(max(lo - h, 0), 32), upto = min(max(hi - h, 0), 32);
              const uint32_t seen = upto > below ? 0xffffffffu >> (32 - (upto - below)) << below : 0u;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(seen >> c & 1)) f[h + c] = neg_inf();
            }
          };
          // Whether a warp's scores are all well inside the cap chooses between two ways to the same bits: scores that a row
          // does not see have a say in it.
          bool inside = false;
          float top = 0.0f;
          if (CAP) {
            top = extremes();
#pragma unroll
            for (int i = 0; i < 4; ++i) lows[i] = fminf(f[2 * i], f[2 * i + 1]);
#pragma unroll
            for (int c = 8; c < kKeys; c += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) lows[i] = min3(lows[i], f[c + 2 * i], f[c + 2 * i + 1]);
            const float low = fminf(fminf(lows[0], lows[1]), fminf(lows[2], lows[3]));
            inside = poly.most > 0.0f && !__any_sync(0xffffffffu, fmaxf(top, -low) > poly.most);
          }
          if (masked) mask();
          if (!CAP || masked) top = extremes();
          if (!CAP) {
            top *= map.mul;
          } else if (inside) {
            top = fmaf(top, cap_factor(poly, make_float2(top, top)).x, 0.0f);
          } else if (top != neg_inf()) {
            top = cap_exponent<false>(poly, map, top, 0.0f);
          }
          if (j == g.j0) {
            m = top;
          } else if (const bool rise = top > m + kLazy || (m == neg_inf() && top > m); __any_sync(0xffffffffu, rise)) {
            const float now = rise ? top : m;  // (each row by its own scores)
            const float scale = now == neg_inf() ? 1.0f : ex2(m - now);
            m = now;
            l *= scale;
            // O holds the products up to block j-1
            HC_WAIT(&bars.o_done[x], (o_seen - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(o_at + c, o);
              tmem_wait_ld();
              landed32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * scale);
              tmem_st32(o_at + c, o);
            }
            tmem_wait_st();
          }
          const float ref = m == neg_inf() ? 0.0f : m;
          if (CAP && !inside) {
            // (32 at a time from tensor memory and back, in a loop: all 128 in registers spill)
            const auto exponents = [&](auto all) {
#pragma unroll 1
              for (int c = 0; c < kKeys; c += 32) {
                uint32_t y[32];
                tmem_ld32(s_at + c, y);
                tmem_wait_ld();
                landed32(y);
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(cap_exponent<decltype(all)::value>(poly, map, __uint_as_float(y[i]), ref));
                tmem_st32(s_at + c, y);
              }
            };
            if (poly.all) {
              exponents(std::true_type());
            } else {
              exponents(std::false_type());
            }
            tmem_wait_st();
            load_scores();
            if (masked) mask();
          }
          const float2 mul2 = make_float2(map.mul, map.mul), ref2 = make_float2(-ref, -ref);
          float2 sum0 = make_float2(0.0f, 0.0f), sum1 = sum0;
          const auto weights = [&](auto exponent) {
#pragma unroll
            for (int h = 0; h < kKeys; h += 64) {
              uint32_t p[32];
#pragma unroll
              for (int c = 0; c < 64; c += 4) {
                const float2 v0 = make_float2(f[h + c], f[h + c + 1]), v1 = make_float2(f[h + c + 2], f[h + c + 3]);
                float2 y0 = exponent(v0), y1 = exponent(v1);
                y0 = make_float2(ex2(y0.x), ex2(y0.y));
                y1 = make_float2(ex2(y1.x), ex2(y1.y));
                sum0 = add2(sum0, y0);
                sum1 = add2(sum1, y1);
                p[c / 2] = pack2<T>(y0.x, y0.y);
                p[c / 2 + 1] = pack2<T>(y1.x, y1.y);
              }
              tmem_st32(s_at + h / 2, p);
            }
          };
          if (!CAP) {
            weights([&](float2 v) { return fma2(v, mul2, ref2); });
          } else if (inside) {
            weights([&](float2 v) { return fma2(v, cap_factor(poly, v), ref2); });
          } else {
            weights([&](float2 v) { return v; });
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.p_full[x]);
          sum0 = add2(sum0, sum1);
          l += sum0.x + sum0.y;
          ++o_seen;
        }
        // the tile's scores are all formed, so its queries make room for the next segment's
        HC_SEGMENT(seg + 1);
        const bool fetched = fetch_q(segs[(seg + 1) % kSegs]);
        const bool some = end > g.j0;
        if (some) {
          HC_WAIT(&bars.o_done[x], (o_seen - 1) & 1);
          tc_fence_after();
        }
        if (fetched) hand_q();
        // what is to be added to features c .. c + 31 of this row's sums
        HC_WAIT(&bars.odd_full[seg % kSegs], (seg / kSegs) & 1);
        const OddValues& list = odd[seg % kSegs];
        const bool odds = list.any != 0;
        const auto add_odd = [&](int c, uint32_t* o) {
          for (int b = 0; b < list.blocks; ++b)
            for (int w = 0; w < 4; ++w) {
              const int k0 = list.block[b] * kKeys + 32 * w, lo = max(from - k0, 0), hi = min(to - k0, 32);
              uint32_t keys = lo < hi ? list.keys[b][w] & (0xffffffffu >> (32 - (hi - lo)) << lo) : 0u;
              for (; keys != 0; keys &= keys - 1) {
                const uint32_t key = static_cast<uint32_t>(g.t.base + k0 + __ffs(keys) - 1), e = key / static_cast<uint32_t>(a.b.page_size);
                const int page = page_of(a.b, g.t.s, e);
                if (page < 0) continue;
                const T* v = static_cast<const T*>(a.v) + page * a.c_ps + (key - e * a.b.page_size) * a.c_ts + g.kv_head * a.c_hs + c;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float x = ldf(v + i);
                  if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
                }
              }
            }
        };
        if (rows > 0) {
          const bool partial = g.j0 > 0 || g.j1 < g.n;
          const bool real = row < rows;
          if (partial) {
            const int64_t at = (2 * static_cast<int64_t>(blockIdx.x) + (g.j0 > 0 ? 0 : 1)) * kPair + x * kRows + row;
            w.part_ml[at] = some ? make_float2(m, l) : make_float2(neg_inf(), 0.0f);
            if (some) {
#pragma unroll
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(o_at + c, o);
                tmem_wait_ld();
                landed32(o);
                if (odds) add_odd(c, o);
                write_out(o, reinterpret_cast<unsigned char*>(w.part_o), real ? (at * D + c) * 4 : -1, true);
              }
            }
          } else {
            int64_t token = 0;
            int head = 0;
            if (real) row_owner(a, g.t, g.kv_head, x * kRows + row, &token, &head);
            const int64_t at = token * a.o_ts + head * a.o_hs;
            const bool wide = ((a.o_ts | a.o_hs) & 7) == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int c = 0; c < D; c += 64) {
              uint32_t y[32];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t o[32];
                tmem_ld32(o_at + c + 32 * h, o);
                tmem_wait_ld();
                landed32(o);
                if (odds) add_odd(c + 32 * h, o);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  y[16 * h + i] = pack2<T>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
              }
              write_out(y, static_cast<unsigned char*>(a.out), real ? (at + c) * 2 : -1, wide);
            }
            if (real && a.lse) a.lse[token * a.heads + head] = l == 0.0f ? neg_inf() : m * kLn2 + logf(l);
          }
          tc_fence_before();  // O has been read before the next segment's weights let it be written
        }
        done_with(seg);
      }
    };
    if (!softmax_all()) {
      const Segment& g = segs[seg % kSegs];
      const float nan = __int_as_float(0x7fffffff);
      for (int i = 0; i < 2; ++i)
        w.part_ml[(2 * static_cast<int64_t>(blockIdx.x) + i) * kPair + x * kRows + row] = make_float2(0.0f, nan);
      if (mbar_test(&bars.seg_full[seg % kSegs], (seg / kSegs) & 1) && g.j1 > g.j0 && row < tile_rows(g.t, x)) {
        int64_t token;
        int head;
        row_owner(a, g.t, g.kv_head, x * kRows + row, &token, &head);
        for (int d = 0; d < D; ++d) stf(static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs + d, nan);
      }
    }
  }
#undef HC_SEGMENT
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of the tiles that cuts go through: kJoinRows rows to a CTA. First
// every row's weights, 2^(m_i - M) / sum, eight threads to a row; then the sums, a
// thread to four features. Bound by the latency of its chain of loads (what is to be
// joined, then maxima and sums, then partial results), so a CTA has many rows in
// flight at once.
constexpr int kJoinRows = 32;
constexpr int kMaxCtas = 160;

template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(AttnArgs a, Work w) {
  __shared__ float s_w[kJoinRows][kMaxCtas + 1];
  pdl_wait();  // (in every thread, before anything is read or left: later kernels on the stream count on this one's end alone)
  const int c0 = blockIdx.x;
  const JoinTile g = w.joins[c0];
  const int pieces = g.pieces;
  const int row0 = blockIdx.y * kJoinRows;
  const int rows = min(g.t.rows - row0, kJoinRows);
  // piece 0 is the last of its CTA's segments, the others are the first of theirs
  const auto index = [&](int i, int r) { return (2 * static_cast<int64_t>(c0 + i) + (i == 0 ? 1 : 0)) * kPair + row0 + r; };
  if (c0 == static_cast<int>(gridDim.x) - 1) clear_unowned<T>(a, blockIdx.y, gridDim.y);  // (no cut lies behind the last CTA's run)
  if (pieces == 0 || rows <= 0) return;
  {
    const int r = threadIdx.x >> 3, e = threadIdx.x & 7;
    float top = neg_inf(), sum = 0.0f;
    if (r < rows)
      for (int i = e; i < pieces; i += 8) top = fmaxf(top, w.part_ml[index(i, r)].x);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (r < rows)
      for (int i = e; i < pieces; i += 8) {
        const float2 ml = w.part_ml[index(i, r)];
        // (scores that are all NaN: m = -inf, l = NaN)
        const float f = ml.x == neg_inf() ? (ml.y == 0.0f ? 0.0f : 1.0f) : exp2f(ml.x - top);
        s_w[r][i] = f;
        sum += ml.y * f;
      }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (r < rows) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      for (int i = e; i < pieces; i += 8) s_w[r][i] *= inv;
      if (e == 0 && a.lse) {
        int64_t token;
        int head;
        row_owner(a, g.t, g.kv_head, row0 + r, &token, &head);
        a.lse[token * a.heads + head] = sum == 0.0f ? neg_inf() : top * kLn2 + logf(sum);
      }
    }
  }
  __syncthreads();
  constexpr int kPer = D / 4;          // threads of a row
  constexpr int kAtOnce = 256 / kPer;  // rows at once
  const int d = threadIdx.x % kPer * 4;
#pragma unroll
  for (int r0 = 0; r0 < kJoinRows; r0 += kAtOnce) {
    const int r = r0 + threadIdx.x / kPer;
    if (r >= rows) continue;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < pieces; ++i) {
      const float f = s_w[r][i];
      if (f == 0.0f) continue;  // (a piece without a key of this row has no sums)
      const float4 y = *reinterpret_cast<const float4*>(w.part_o + index(i, r) * D + d);
      o.x = fmaf(y.x, f, o.x);
      o.y = fmaf(y.y, f, o.y);
      o.z = fmaf(y.z, f, o.z);
      o.w = fmaf(y.w, f, o.w);
    }
    int64_t token;
    int head;
    row_owner(a, g.t, g.kv_head, row0 + r, &token, &head);
    T* dst = static_cast<T*>(a.out) + token * a.o_ts + head * a.o_hs + d;
    stf(dst, o.x);
    stf(dst + 1, o.y);
    stf(dst + 2, o.z);
    stf(dst + 3, o.w);
  }
}

// ------------------------------------------------------------------- host --

// The pool as (features, tokens of a page, key heads, pages), boxes of 64
// features and a page's tokens (128 at most) of one head.
bool make_pool_map(CUtensorMap* m, const void* base, bool bf16, const AttnArgs& a) {
  auto fn = tmap_encoder();
  if (fn == nullptr) return false;
  // strides of axes with one entry are never used, but must be valid
  const int64_t row = a.dim, ts = a.b.page_size > 1 ? a.c_ts : row, hs = a.kv_heads > 1 ? a.c_hs : row,
                ps = a.b.num_pages > 1 ? a.c_ps : row;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(a.b.page_size),
                              static_cast<cuuint64_t>(a.kv_heads), static_cast<cuuint64_t>(a.b.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ts) * 2, static_cast<cuuint64_t>(hs) * 2,
                                 static_cast<cuuint64_t>(ps) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(std::min(a.b.page_size, kKeys)), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(base),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool CAP>
cudaError_t launch_t(const AttnArgs& a, const Work& w, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  constexpr size_t smem = Cfg<D>::kSmem;
  cudaError_t e = ensure_smem<tile_kernel<T, D, CAP>>(smem);
  if (e != cudaSuccess) return e;
  plan_kernel<<<1, 1024, 0, s>>>(a, const_cast<int64_t*>(w.prefix), const_cast<AttnTile*>(w.tiles), w.slots);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_pdl(tile_kernel<T, D, CAP>, dim3(w.ctas), dim3(kThreads), smem, s, 1, a, w, k, v);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_kernel<T, D>, dim3(w.ctas, kPair / kJoinRows), dim3(256), 0, s, 1, a, w);
}

template <typename T>
cudaError_t launch_d(const AttnArgs& a, const Work& w, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
  if (a.dim == 64)
    return a.softcap > 0.0f ? launch_t<T, 64, true>(a, w, k, v, s) : launch_t<T, 64, false>(a, w, k, v, s);
  return a.softcap > 0.0f ? launch_t<T, 128, true>(a, w, k, v, s) : launch_t<T, 128, false>(a, w, k, v, s);
}

size_t prefix_bytes(int64_t slots) { return align_up(static_cast<size_t>(slots + 1) * 8, 256); }
size_t tiles_bytes(int64_t slots) { return align_up(static_cast<size_t>(slots) * sizeof(AttnTile), 256); }
size_t joins_bytes(int num_sms) { return align_up(static_cast<size_t>(num_sms) * sizeof(JoinTile), 256); }

int64_t slots_of(int64_t tokens, int group, int seqs) { return tokens * group / kPair + seqs; }

}  // namespace

unsigned int read_tile_wait_timeouts(bool reset) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_tile_wait_timeouts, sizeof(v)) != cudaSuccess) return 0xffffffffu;
  if (reset) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_tile_wait_timeouts, &z, sizeof(z));
  }
  return v;
}

bool attn_tile_supported(int dtype, int dim, int page, float scale, bool aligned) {
  return aligned && (dtype == HC_F16 || dtype == HC_BF16) && (dim == 64 || dim == 128) && scale > 0.0f && page >= 8 &&
         (kKeys % page == 0 || page % kKeys == 0) && tmap_encoder() != nullptr;
}

size_t attn_tile_workspace(int64_t tokens, int group, int seqs, int dim, int num_sms) {
  const size_t rows = 2 * static_cast<size_t>(num_sms) * kPair;
  const int64_t slots = slots_of(tokens, group, seqs);
  return prefix_bytes(slots) + tiles_bytes(slots) + joins_bytes(num_sms) + align_up(rows * 8, 256) + rows * dim * 4;
}

cudaError_t launch_attn_tile(const AttnArgs& args, int dtype, void* workspace, int num_sms, cudaStream_t s) {
  AttnArgs a = args;
  a.g = AttnGeometry{kPair, kKeys, 1 << 30, 1};
  Work w;
  w.slots = static_cast<int>(slots_of(a.tokens, a.group, a.b.seqs));
  w.ctas = std::min(num_sms, kMaxCtas);
  char* p = static_cast<char*>(workspace);
  w.prefix = reinterpret_cast<const int64_t*>(p);
  p += prefix_bytes(w.slots);
  w.tiles = reinterpret_cast<const AttnTile*>(p);
  p += tiles_bytes(w.slots);
  w.joins = reinterpret_cast<JoinTile*>(p);
  p += joins_bytes(num_sms);
  w.part_ml = reinterpret_cast<float2*>(p);
  p += align_up(2 * static_cast<size_t>(num_sms) * kPair * 8, 256);
  w.part_o = reinterpret_cast<float*>(p);
  CUtensorMap k, v;
  const bool bf16 = dtype == HC_BF16;
  if (!make_pool_map(&k, a.k, bf16, a) || !make_pool_map(&v, a.v, bf16, a)) return cudaErrorInvalidValue;
  return bf16 ? launch_d<__nv_bfloat16>(a, w, k, v, s) : launch_d<__half>(a, w, k, v, s);
}

}  // namespace hc
