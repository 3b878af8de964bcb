/* hc_paged.h -- C ABI of the attention layer that a decoder runs between two
 * hyper-connection blocks when it serves from a paged key/value cache (GB300,
 * sm_103a): rotary positions, the write of new tokens into the cache,
 * attention over the cache, and the upkeep of its pages.
 *
 * The cache of one layer is a pool of pages for the keys and one for the
 * values. A page holds page_size consecutive tokens of one sequence; element
 * (page, token, kv_head, d) of a pool lies at
 *   page * cache_page_stride + token * cache_token_stride + kv_head * cache_head_stride + d
 * (strides in elements, the same for keys and values; d is contiguous). Row s
 * of page_table lists the pages of sequence s in order. kv_lens[s] counts its
 * tokens, the new ones of the call among them; what pages hold past that is
 * never read. With cu_q (seqs + 1 ascending offsets, as a rule from
 * 0 to tokens) the new tokens of sequence s are the rows cu_q[s] ..
 * cu_q[s+1] - 1 of the call; without it (NULL) every sequence has one. The
 * last new token of a sequence has position kv_lens[s] - 1, those before it
 * the positions before. A new token whose position would be negative (an
 * unused slot of a batch has kv_lens[s] = 0) sees nothing and is written
 * nowhere. Rows before cu_q[0] and from cu_q[seqs] on, where a buffer of a
 * fixed size has more rows than the sequences have new tokens, are no
 * sequence's: they see nothing and are written nowhere either (what q_out
 * holds for them is of no use).
 *
 * Memory: all pointers are DEVICE pointers of the caller, except the argument
 * structs, which are read before the call returns. The calls allocate nothing,
 * never synchronise the host and keep no state, so they can be captured in a
 * CUDA graph. All are asynchronous on `stream`. Results are bitwise
 * deterministic for the same inputs, sizes and device.
 *
 * Errors (checked on the host before any launch): HC_ERR_INVALID_ARG for bad
 * sizes, a null pointer, strides below the extents or an output overlapping
 * an input; HC_ERR_UNSUPPORTED for sizes beyond the limits below or a device
 * other than sm_103; HC_ERR_WORKSPACE for a workspace that is missing, short
 * or not 256-byte aligned; HC_ERR_CUDA if a launch fails. hc_last_error() has
 * the message. What lies in device memory cannot be checked on the host:
 * lengths are cut to what the table's row can hold, and a page number outside
 * the pool is never followed (what such a page would hold is unspecified). */
#ifndef HC_PAGED_H
#define HC_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "hc_lowrank_mix.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------- rotary --
 *
 * Pair i (0 <= i < rot_dim / 2) of a head at position p turns by the angle
 * p * inv_freq[i] and is scaled by `amplitude`:
 *
 *   y_a = amplitude * (x_a cos - x_b sin),  y_b = amplitude * (x_b cos + x_a sin)
 *
 * with (a, b) = (i, i + rot_dim/2), or (2i, 2i + 1) with `interleaved`.
 * Features from rot_dim on are copied. `inverse` turns the other way: since a
 * rotation's transpose is its inverse, that is also the gradient with respect
 * to x, given the gradient with respect to y.
 *
 * inv_freq: rot_dim/2 float64 values in radians per token (any scaling for
 * long contexts is a matter of these values and of amplitude). The angle is
 * formed in whole turns, as the position times a 64-bit fraction of a turn
 * modulo one turn, which loses nothing however large the position; sine,
 * cosine and products are fp32, with one rounding to T at the store. */
typedef struct {
  const void* x;         /* (tokens, heads, head_dim) of type dtype */
  const void* positions; /* (tokens) int64, or int32 with positions32 */
  const double* inv_freq;
  void* out; /* like x; may be x itself with the same strides */
  int64_t tokens;
  int64_t x_token_stride, x_head_stride, out_token_stride, out_head_stride; /* elements */
  int32_t heads, head_dim, rot_dim;
  int32_t interleaved, inverse, positions32;
  int32_t dtype; /* hc_dtype_t */
  float amplitude;
} hc_rotary_t;

hc_status_t hc_rotary(const hc_rotary_t* args, struct CUstream_st* stream);

/* The new tokens of a batch: q is rotated into q_out, k is rotated and written
 * into k_cache at its position's place, v is copied into v_cache. k, v and
 * the caches must not overlap. */
typedef struct {
  const void *q, *k, *v; /* (tokens, heads, head_dim), (tokens, kv_heads, head_dim) twice */
  void *q_out, *k_cache, *v_cache;
  const double* inv_freq;
  const int32_t *page_table, *kv_lens, *cu_q;
  int64_t tokens, num_pages, table_stride;
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
  int64_t out_token_stride, out_head_stride;
  int64_t cache_page_stride, cache_token_stride, cache_head_stride;
  int32_t seqs, max_pages, page_size;
  int32_t heads, kv_heads, head_dim, rot_dim;
  int32_t interleaved;
  int32_t dtype;
  float amplitude;
} hc_rotary_append_t;

hc_status_t hc_rotary_append(const hc_rotary_append_t* args, struct CUstream_st* stream);

/* -------------------------------------------------------------- attention --
 *
 * Query head h reads kv head h / (heads / kv_heads). For a new token at
 * position p, over the positions j of its sequence with j <= p and, with a
 * window w > 0, j > p - w:
 *
 *   s_j = scale * <q, k_j>;   with softcap c > 0:  s_j = c * tanh(s_j / c)
 *   out = sum_j exp(s_j - lse) v_j,   lse = log sum_j exp(s_j)
 *
 * A token that sees nothing gets out = 0 and lse = -inf. Scores, softmax and
 * sums are fp32; in the fp16/bf16 kernels the weights of more than eight rows
 * to a key head are rounded to T for the product with the values (the sum of
 * weights is not), out is rounded to T once, lse is fp32. What a token does
 * not see does not touch its result, whatever it holds; an infinity or a NaN
 * among what it sees does, in its own feature.
 *
 * max_q, max_kv: the longest row of new tokens and the longest kv_lens, if the
 * caller knows them (0: unknown). They steer the choice of kernels and how far
 * a sequence is split; results are right whatever they say.
 * Limits: head_dim <= 256, heads * tokens < 2^31. */
typedef struct {
  const void *q, *k_cache, *v_cache;
  const int32_t *page_table, *kv_lens, *cu_q;
  void* out;  /* (tokens, heads, head_dim) */
  float* lse; /* (tokens, heads), or NULL */
  void* workspace;
  size_t workspace_bytes;
  int64_t tokens, num_pages, table_stride;
  int64_t q_token_stride, q_head_stride, out_token_stride, out_head_stride;
  int64_t cache_page_stride, cache_token_stride, cache_head_stride;
  int32_t seqs, max_pages, page_size;
  int32_t heads, kv_heads, head_dim;
  int32_t max_q, max_kv;
  int32_t window; /* 0: none */
  int32_t dtype;
  uint32_t flags; /* HC_FLAG_FORCE_GENERAL or 0 */
  float scale, softcap;
} hc_paged_attention_t;

/* Bytes of workspace for these sizes, strides, hints, scale and flags, which
 * steer the choice of kernels (pointers and lengths are not looked at but for
 * alignment, out and lse not at all); 0 if none is needed. */
size_t hc_paged_attention_workspace_size(const hc_paged_attention_t* args);
hc_status_t hc_paged_attention(const hc_paged_attention_t* args, struct CUstream_st* stream);

/* ------------------------------------------------------------------ pages --
 *
 * A pool of pages across `planes` layers and kinds: page p of plane a is the
 * page_bytes bytes at a * num_pages * page_bytes + p * page_bytes. A page has
 * a reference count in refs (num_pages); the sequences' tables count one each
 * for the first ceil(lens[s] / page_size) entries of a row, others may hold
 * pages too. A page with a count of 0 (or less) is free. Where pages are
 * taken, the free page with the lowest number comes first, and sequences are
 * served in order. The results are new tables, lengths and counts; the inputs
 * stay as they are, and no output overlaps an input. Unused entries of a new
 * table are -1. Page numbers outside the pool are passed over.
 * workspace: hc_pages_workspace_size bytes, 256-byte aligned. */
typedef struct {
  const int32_t *page_table, *lens, *refs;
  int32_t *page_table_out, *lens_out, *refs_out;
  int64_t num_pages, table_stride; /* table_out is (seqs_out, max_pages), contiguous */
  int32_t seqs, max_pages, page_size;
} hc_pages_t;

size_t hc_pages_workspace_size(int64_t num_pages, int32_t seqs);

/* Page dst[i] becomes a copy of page src[i] in every plane, i < count. Entries
 * outside the pool are passed over. The dst are distinct and none is a src. */
hc_status_t hc_page_copy(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                         const int32_t* dst, int64_t count, struct CUstream_st* stream);

/* The `children` new sequences go on from their parents (rows of the table; -1
 * for an empty sequence), and the old ones are given up. Full pages are
 * shared. Of a last page that is not full the first child keeps the original
 * and every other child gets a copy in a page of its own. missing[0]: how many
 * children got no page for want of free ones (their entry is -1). */
hc_status_t hc_page_fork(const hc_pages_t* pages, const int32_t* parents, int32_t children, int32_t* missing, void* cache,
                         int64_t planes, int64_t page_bytes, void* workspace, size_t workspace_bytes,
                         struct CUstream_st* stream);

/* Pages for new_tokens[s] >= 0 more tokens of every sequence. Where pages or
 * the table's width run out, a sequence's new length ends with its pages;
 * missing[0] counts the pages that could not be had. A length ends at 2^31 - 1
 * tokens. */
hc_status_t hc_page_extend(const hc_pages_t* pages, const int32_t* new_tokens, int32_t* missing, void* workspace,
                           size_t workspace_bytes, struct CUstream_st* stream);

/* The sequences with drop[s] != 0 give up their pages (length 0, an empty row). */
hc_status_t hc_page_release(const hc_pages_t* pages, const uint8_t* drop, struct CUstream_st* stream);

/* The n live pages (count above 0) come to lie at 0 .. n-1: the live pages from
 * n on move, in order, into the free ones before n. remap (num_pages): where
 * each live page went, -1 for the others; live[0] = n. lens_out is not used. */
hc_status_t hc_page_compact(const hc_pages_t* pages, int32_t* remap, int32_t* live, void* cache, int64_t planes,
                            int64_t page_bytes, void* workspace, size_t workspace_bytes, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_PAGED_H */
