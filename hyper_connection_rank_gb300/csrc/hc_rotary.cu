// Rotary positions, alone and fused with the write of a batch's new tokens
// into the paged cache (include/hc_paged.h).
//
// Mathematics: pair (a, b) of a head at position p turns by p * inv_freq. The
// angle is wanted modulo one turn, and fp32 has lost it long before p reaches
// the lengths in use (at p = 10^5 an fp32 angle is off by up to 0.004 rad).
// So the frequency becomes a 64-bit fraction of a turn, u = 2^64 * frac(
// inv_freq / 2 pi), and p * u modulo 2^64 is the exact fraction of a turn after
// p tokens (negative p wrap the right way); its upper 32 bits, as a signed
// number of half turns in [-1, 1), go to sincospif. What is left is u's own
// rounding (2^-53 relative) and one fp32 rounding of the half turns.
//
// Bound: bytes; every element is read and written once. A CTA of 128 threads
// serves a token; its sines and cosines are formed once in shared memory (rot_dim/2,
// against heads * rot_dim elements that use them), and each thread
// then turns 16 bytes of each side of the pairs at a time. The half layout
// takes the two sides from one head's two halves, the interleaved one has both
// sides in one vector. Ten to sixteen CTAs share an SM (46 to 32
// registers a thread; held to twelve or sixteen, the first size below takes 1 and 4 us more);
// forms that held two or four vectors of the next heads in registers ran at
// half the occupancy and took 76 to 113 us where the form without took 57. Small CTAs
// keep the last wave short: two tokens to 256 threads took 20.1 and 57.4 us for the sizes
// below, one token to 256 threads 20.8 and 61.9, to 64 threads 21.3 and 63.7.
//
// Measured (bf16, 13638 tokens of 32 + 2 * 8 heads of 128 written into pages of
// 64): 53.7 us, 6.25 TB/s, 93% of the measured copy bandwidth; the angles read
// with bank conflicts cost 9 us more. float32, 4099 tokens of 20 heads: 18.3 us, 4.6
// TB/s: they are two to three waves of CTAs, each of which begins with its chain of
// four loads (position, frequencies, angles) before it moves a byte.
#include "hc_common.cuh"
#include "hc_paged_batch.cuh"
#include "hc_paged_internal.h"

namespace hc {
namespace {

constexpr int kThreads = 128;

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
};

struct RotaryArgs {
  // parts of a token's row: heads [0, hq) from q, [hq, hq + hk) from k, the next hk from v
  const void *q, *k, *v;
  void *q_out, *k_cache, *v_cache;
  const void* positions;  // NULL: positions come from the batch
  bool positions32;
  const double* inv_freq;
  int64_t tokens;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs, c_ps, c_ts, c_hs;
  int hq, hk, dim, rot;
  float amplitude, sign;
  BatchView batch;
};

// Pairs that one item turns, and where the (cos, sin) of its i-th pair lies among
// a token's: two pairs to 16 bytes, and items side by side, so that the threads
// of a head read different banks.
template <int V, bool INTER>
struct Angles {
  static constexpr int kPairs = V > 1 && INTER ? V / 2 : V;
  static __device__ __forceinline__ int at(int it, int i, int half) {
    return kPairs == 1 ? it : ((i >> 1) * (half / kPairs) + it) * 2 + (i & 1);
  }
};

// Items of a head's work. V > 1: vectors of V features (interleaved), or pairs
// of vectors from the two halves and then vectors that are copied; V == 1, for
// any alignment: pairs, then single features that are copied.
template <int V, bool INTER>
__host__ __device__ __forceinline__ int items_of(int dim, int rot) {
  if (V > 1 && INTER) return dim / V;
  return rot / 2 / V + (dim - rot) / V;
}

// Item `it` of one head, `src` to `dst` (which may be the same place).
template <typename T, int V, bool INTER>
__device__ __forceinline__ void turn_item(const T* src, T* dst, int it, int rot, const float2* cs) {
  using P = Pack<T, V>;
  if (V > 1 && INTER) {
    P x = *reinterpret_cast<const P*>(src + it * V);
    if (it * V < rot) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 c = cs[Angles<V, INTER>::at(it, i >> 1, rot >> 1)];
        const float a = Ty<T>::to_f(x.e[i]), b = Ty<T>::to_f(x.e[i + 1]);
        x.e[i] = Ty<T>::from_f(a * c.x - b * c.y);
        x.e[i + 1] = Ty<T>::from_f(b * c.x + a * c.y);
      }
    }
    *reinterpret_cast<P*>(dst + it * V) = x;
  } else {
    const int half = rot >> 1, turns = half / V;
    if (it < turns) {
      const int ia = INTER ? 2 * it : it * V, ib = INTER ? 2 * it + 1 : half + it * V;
      P x = *reinterpret_cast<const P*>(src + ia);
      P y = *reinterpret_cast<const P*>(src + ib);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float2 c = cs[Angles<V, INTER>::at(it, i, half)];
        const float a = Ty<T>::to_f(x.e[i]), b = Ty<T>::to_f(y.e[i]);
        x.e[i] = Ty<T>::from_f(a * c.x - b * c.y);
        y.e[i] = Ty<T>::from_f(b * c.x + a * c.y);
      }
      *reinterpret_cast<P*>(dst + ia) = x;
      *reinterpret_cast<P*>(dst + ib) = y;
    } else {
      const int d = rot + (it - turns) * V;
      *reinterpret_cast<P*>(dst + d) = *reinterpret_cast<const P*>(src + d);
    }
  }
}

// V elements per access; a CTA to a token. Dynamic shared memory: rot/2 (cos, sin).
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int64_t s_pos;
  __shared__ int64_t s_slot;  // element offset of the token in the pool, -1: nowhere
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = a.rot >> 1, heads = a.hq + 2 * a.hk;
  float2* cs = reinterpret_cast<float2*>(smem);
  const int64_t t = blockIdx.x;

  // the token's rows are on their way to the L2 while the angles are formed: one prefetch to a head of 128 bytes and more
  {
    const int lines = (a.dim * static_cast<int>(sizeof(T)) + 127) / 128;
    for (int i = tid; i < heads * lines; i += kThreads) {
      const int h = i / lines;
      const T* src = h < a.hq           ? static_cast<const T*>(a.q) + t * a.q_ts + h * a.q_hs
                     : h < a.hq + a.hk  ? static_cast<const T*>(a.k) + t * a.k_ts + (h - a.hq) * a.k_hs
                                        : static_cast<const T*>(a.v) + t * a.v_ts + (h - a.hq - a.hk) * a.v_hs;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(src + (i - h * lines) * (128 / static_cast<int>(sizeof(T)))));
    }
  }
  // frequencies as fractions of a turn, the first of each thread while the position is on its way
  const auto fraction = [&](int i) {
    double f = a.inv_freq[i] * 0.15915494309189535;  // turns per token
    f -= floor(f);
    return __double2ull_rn(f * 18446744073709551616.0);
  };
  const uint64_t first = tid < half ? fraction(tid) : 0;
  if (a.positions != nullptr) {
    if (tid == 0)
      s_pos = a.positions32 ? static_cast<const int32_t*>(a.positions)[t] : static_cast<const int64_t*>(a.positions)[t];
  } else if (warp == kThreads / 32 - 1) {
    const BatchView& b = a.batch;
    const int s = b.cu_q ? warp_last_le(b.seqs, t, [&](int i) { return first_row(b, i); })
                         : static_cast<int>(t);
    if (lane == 0) {
      const int64_t end = first_row(b, s + 1);
      const int64_t pos = kv_len_of(b, s) - (end - t);
      int page = -1;
      // (a row past the last bound, or before the first, is no sequence's and has no place in its table)
      if (pos >= 0 && t >= first_row(b, s) && t < end) page = page_of(b, s, pos / b.page_size);
      s_pos = pos;
      s_slot = page < 0 ? -1 : page * a.c_ps + pos % b.page_size * a.c_ts;
    }
  }
  __syncthreads();
  for (int i = tid; i < half; i += kThreads) {
    const int32_t turn = static_cast<int32_t>((static_cast<uint64_t>(s_pos) * (i == tid ? first : fraction(i))) >> 32);
    float s, c;
    sincospif(static_cast<float>(turn) * 4.656612873077393e-10f, &s, &c);  // half turns: turn * 2^-31
    constexpr int kPairs = Angles<V, INTER>::kPairs;
    cs[Angles<V, INTER>::at(i / kPairs, i % kPairs, half)] = make_float2(a.amplitude * c, a.amplitude * a.sign * s);
  }
  __syncthreads();

  // threads: `items` to a head, as many heads at a time as fit
  const int items = items_of<V, INTER>(a.dim, a.rot);
  const int hpp = items < kThreads ? kThreads / items : 1;
  const int ih = items < kThreads ? tid / items : 0;
  if (ih >= hpp) return;
  for (int it = items < kThreads ? tid - ih * items : tid; it < items; it += kThreads) {
    int h = ih;
    {
      const T* src = static_cast<const T*>(a.q) + t * a.q_ts + h * a.q_hs;
      T* dst = static_cast<T*>(a.q_out) + t * a.o_ts + h * a.o_hs;
      for (; h < a.hq; h += hpp, src += hpp * a.q_hs, dst += hpp * a.o_hs) turn_item<T, V, INTER>(src, dst, it, a.rot, cs);
    }
    if (h >= heads || s_slot < 0) continue;
    {
      const T* src = static_cast<const T*>(a.k) + t * a.k_ts + (h - a.hq) * a.k_hs;
      T* dst = static_cast<T*>(a.k_cache) + s_slot + (h - a.hq) * a.c_hs;
      for (; h < a.hq + a.hk; h += hpp, src += hpp * a.k_hs, dst += hpp * a.c_hs)
        turn_item<T, V, INTER>(src, dst, it, a.rot, cs);
    }
    const int kh = h - a.hq - a.hk;
    const T* src = static_cast<const T*>(a.v) + t * a.v_ts + kh * a.v_hs;
    T* dst = static_cast<T*>(a.v_cache) + s_slot + kh * a.c_hs;
    for (; h < heads; h += hpp, src += hpp * a.v_hs, dst += hpp * a.c_hs)
      for (int c = it; c < a.dim / V; c += items)
        *reinterpret_cast<Pack<T, V>*>(dst + c * V) = *reinterpret_cast<const Pack<T, V>*>(src + c * V);
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch_t(const RotaryArgs& a, cudaStream_t s) {
  rotary_kernel<T, V, INTER><<<static_cast<unsigned>(a.tokens), kThreads, static_cast<size_t>(a.rot / 2) * 8, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool INTER>
cudaError_t launch_v(const RotaryArgs& a, bool vec, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  // 16-byte vectors where every part of a head is whole ones, else element by element
  const bool whole = vec && a.dim % V == 0 && a.rot % (INTER ? V : 2 * V) == 0;
  return whole ? launch_t<T, V, INTER>(a, s) : launch_t<T, 1, INTER>(a, s);
}

cudaError_t launch_any(const RotaryArgs& a, int dtype, bool interleaved, bool vec, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  switch (dtype) {
    case HC_F32:
      return interleaved ? launch_v<float, true>(a, vec, s) : launch_v<float, false>(a, vec, s);
    case HC_F16:
      return interleaved ? launch_v<__half, true>(a, vec, s) : launch_v<__half, false>(a, vec, s);
    default:
      return interleaved ? launch_v<__nv_bfloat16, true>(a, vec, s)
                         : launch_v<__nv_bfloat16, false>(a, vec, s);
  }
}

}  // namespace

cudaError_t launch_rotary(const hc_rotary_t& r, bool vec, cudaStream_t s) {
  RotaryArgs a = {};
  a.q = r.x;
  a.q_out = r.out;
  a.positions = r.positions;
  a.positions32 = r.positions32 != 0;
  a.inv_freq = r.inv_freq;
  a.tokens = r.tokens;
  a.q_ts = r.x_token_stride;
  a.q_hs = r.x_head_stride;
  a.o_ts = r.out_token_stride;
  a.o_hs = r.out_head_stride;
  a.hq = r.heads;
  a.dim = r.head_dim;
  a.rot = r.rot_dim;
  a.amplitude = r.amplitude;
  a.sign = r.inverse ? -1.0f : 1.0f;
  return launch_any(a, r.dtype, r.interleaved != 0, vec, s);
}

cudaError_t launch_rotary_append(const hc_rotary_append_t& r, bool vec, cudaStream_t s) {
  RotaryArgs a = {};
  a.q = r.q;
  a.k = r.k;
  a.v = r.v;
  a.q_out = r.q_out;
  a.k_cache = r.k_cache;
  a.v_cache = r.v_cache;
  a.inv_freq = r.inv_freq;
  a.tokens = r.tokens;
  a.q_ts = r.q_token_stride;
  a.q_hs = r.q_head_stride;
  a.k_ts = r.k_token_stride;
  a.k_hs = r.k_head_stride;
  a.v_ts = r.v_token_stride;
  a.v_hs = r.v_head_stride;
  a.o_ts = r.out_token_stride;
  a.o_hs = r.out_head_stride;
  a.c_ps = r.cache_page_stride;
  a.c_ts = r.cache_token_stride;
  a.c_hs = r.cache_head_stride;
  a.hq = r.heads;
  a.hk = r.kv_heads;
  a.dim = r.head_dim;
  a.rot = r.rot_dim;
  a.amplitude = r.amplitude;
  a.sign = 1.0f;
  a.batch = BatchView{r.page_table, r.kv_lens, r.cu_q, r.table_stride, r.num_pages, r.seqs, r.max_pages, r.page_size, r.tokens};
  return launch_any(a, r.dtype, r.interleaved != 0, vec, s);
}

}  // namespace hc
