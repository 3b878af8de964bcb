// C ABI of the paged-cache operators (include/hc_paged.h): every error is found
// on the host, before any launch, and returned as a status.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "hc_args.h"
#include "hc_paged_internal.h"

namespace {

using namespace hc::args;
using hc::dtype_size;

// The largest count of tokens, of which all products below are formed.
hc_status_t check_tokens(int64_t tokens) {
  if (tokens < 0) return fail(HC_ERR_INVALID_ARG, "invalid tokens=%lld", ll(tokens));
  if (tokens >= int64_t{1} << 31) return fail(HC_ERR_UNSUPPORTED, "tokens=%lld beyond 2^31", ll(tokens));
  return HC_OK;
}

hc_status_t check_extent(const char* name, int64_t tokens, int64_t ts, int heads, int64_t hs) {
  if (!sane(ts) || !sane(hs)) return fail(HC_ERR_INVALID_ARG, "invalid strides of %s", name);
  if (!within(tokens, ts) || !within(heads, hs)) return fail(HC_ERR_UNSUPPORTED, "%s beyond 2^46 elements", name);
  return HC_OK;
}

// Rows of heads: (tokens, heads, dim) with element strides, within the extents above. Heads of a token
// must not overlap one another, nor tokens; either may be the outer one.
bool strides_valid(int64_t tokens, int64_t ts, int heads, int64_t hs, int dim) {
  if (tokens <= 0 || heads <= 0) return true;
  if (heads > 1 && hs < dim) return false;
  if (tokens > 1 && ts < dim) return false;
  if (tokens == 1 || heads == 1) return true;
  return ts >= hs * (heads - 1) + dim || hs >= ts * (tokens - 1) + dim;
}
int64_t extent(int64_t tokens, int64_t ts, int heads, int64_t hs, int dim) {
  if (tokens <= 0 || heads <= 0) return 0;
  return (tokens - 1) * ts + (heads - 1) * hs + dim;
}

// Whether two tensors of rows (first element at a and b, `na` and `nb` elements from the first to the last of a row, one step
// from row to row) share an element: b's rows must fit between a's.
bool rows_meet(uintptr_t a, int64_t na, uintptr_t b, int64_t nb, int64_t step, int64_t rows, int64_t es) {
  const Span x = span("", reinterpret_cast<const void*>(a), es * ((rows - 1) * step + na));
  const Span y = span("", reinterpret_cast<const void*>(b), es * ((rows - 1) * step + nb));
  if (!overlaps(x, y)) return false;
  const int64_t at = static_cast<int64_t>(b - a) / es, in = step > 0 ? (at % step + step) % step : 0;
  return rows == 1 || in < na || in + nb > step;
}

hc_status_t check_cache(int64_t pages, int64_t ps, int page, int64_t ts, int kv_heads, int64_t hs, int dim) {
  if (pages < 1 || pages > (int64_t{1} << 31) - 1 || page < 1 || page > (1 << 20))
    return fail(HC_ERR_INVALID_ARG, "invalid pool: num_pages=%lld page_size=%d", ll(pages), page);
  HC_RETURN_IF(check_extent("a page", page, ts, kv_heads, hs));
  if (!sane(ps) || !strides_valid(page, ts, kv_heads, hs, dim) || (pages > 1 && ps < 1))
    return fail(HC_ERR_INVALID_ARG, "cache strides (page %lld, token %lld, head %lld) do not fit heads of %d", ll(ps),
                ll(ts), ll(hs), dim);
  if (pages - 1 > kMaxElems / std::max<int64_t>(ps, 1)) return fail(HC_ERR_UNSUPPORTED, "pool beyond 2^46 elements");
  return HC_OK;
}

hc_status_t check_batch(const int32_t* table, const int32_t* lens, const int32_t* cu, int64_t tokens, int seqs,
                        int max_pages, int64_t table_stride) {
  HC_RETURN_IF(check_tokens(tokens));
  if (seqs < 0 || max_pages < 1 || max_pages > (1 << 20))
    return fail(HC_ERR_INVALID_ARG, "invalid batch: seqs=%d tokens=%lld max_pages=%d", seqs, ll(tokens), max_pages);
  if (table_stride < max_pages && seqs > 1)
    return fail(HC_ERR_INVALID_ARG, "table_stride %lld is below max_pages %d", ll(table_stride), max_pages);
  if (!sane(table_stride)) return fail(HC_ERR_INVALID_ARG, "invalid table_stride");
  if (!within(seqs, table_stride)) return fail(HC_ERR_UNSUPPORTED, "page_table beyond 2^46 entries");
  if (tokens > 0 && (seqs < 1 || table == nullptr || lens == nullptr))
    return fail(HC_ERR_INVALID_ARG, "tokens without sequences, page_table or kv_lens");
  if (cu == nullptr && tokens != seqs)
    return fail(HC_ERR_INVALID_ARG, "without cu_q every sequence has one token: tokens=%lld seqs=%d", ll(tokens), seqs);
  return HC_OK;
}

hc_status_t check_heads(int heads, int dim, int most) {
  if (heads < 1 || dim < 1) return fail(HC_ERR_INVALID_ARG, "invalid heads=%d head_dim=%d", heads, dim);
  if (heads > 65535 || dim > most) return fail(HC_ERR_UNSUPPORTED, "heads=%d head_dim=%d: at most 65535 and %d", heads, dim, most);
  return HC_OK;
}

hc_status_t check_rot(int rot, int dim) {
  if (rot < 0 || rot % 2 != 0 || rot > dim)
    return fail(HC_ERR_INVALID_ARG, "rot_dim %d must be even and at most head_dim %d", rot, dim);
  return HC_OK;
}

}  // namespace

extern "C" {

hc_status_t hc_rotary(const hc_rotary_t* args, cudaStream_t stream) {
  if (args == nullptr) return fail(HC_ERR_INVALID_ARG, "null args");
  const hc_rotary_t& a = *args;
  if (!dtype_valid(a.dtype)) return fail(HC_ERR_INVALID_ARG, "invalid dtype %d", a.dtype);
  HC_RETURN_IF(check_tokens(a.tokens));
  HC_RETURN_IF(check_heads(a.heads, a.head_dim, 1024));
  HC_RETURN_IF(check_rot(a.rot_dim, a.head_dim));
  HC_RETURN_IF(check_extent("x", a.tokens, a.x_token_stride, a.heads, a.x_head_stride));
  HC_RETURN_IF(check_extent("out", a.tokens, a.out_token_stride, a.heads, a.out_head_stride));
  if (!strides_valid(a.tokens, a.out_token_stride, a.heads, a.out_head_stride, a.head_dim))
    return fail(HC_ERR_INVALID_ARG, "invalid strides of out");
  if (a.tokens * a.heads >= (int64_t{1} << 31)) return fail(HC_ERR_UNSUPPORTED, "tokens * heads beyond 2^31");
  if (a.tokens == 0) return HC_OK;
  if (a.x == nullptr || a.out == nullptr || a.positions == nullptr || (a.inv_freq == nullptr && a.rot_dim > 0))
    return fail(HC_ERR_INVALID_ARG, "null pointer");
  const int64_t es = static_cast<int64_t>(dtype_size(static_cast<hc_dtype_t>(a.dtype)));
  if (!on_elements(a.dtype, {a.x, a.out})) return fail(HC_ERR_INVALID_ARG, "misaligned pointer");
  const Span out = span("out", a.out, es * extent(a.tokens, a.out_token_stride, a.heads, a.out_head_stride, a.head_dim));
  const bool in_place = a.out == a.x && a.out_token_stride == a.x_token_stride && a.out_head_stride == a.x_head_stride;
  const Span ins[3] = {
      span("x", in_place ? nullptr : a.x, es * extent(a.tokens, a.x_token_stride, a.heads, a.x_head_stride, a.head_dim)),
      span("positions", a.positions, a.tokens * (a.positions32 ? 4 : 8)), span("inv_freq", a.inv_freq, a.rot_dim * 4)};
  HC_RETURN_IF(check_apart(&out, 1, ins, 3));
  int sms = 0;  // (only to refuse other devices)
  HC_RETURN_IF(hc::current_device_sms(&sms));
  const bool vec = aligned16(a.x) && aligned16(a.out) &&
                   vec_strides(a.dtype, {a.x_token_stride, a.x_head_stride, a.out_token_stride, a.out_head_stride});
  return launched(hc::launch_rotary(a, vec, stream));
}

hc_status_t hc_rotary_append(const hc_rotary_append_t* args, cudaStream_t stream) {
  if (args == nullptr) return fail(HC_ERR_INVALID_ARG, "null args");
  const hc_rotary_append_t& a = *args;
  if (!dtype_valid(a.dtype)) return fail(HC_ERR_INVALID_ARG, "invalid dtype %d", a.dtype);
  HC_RETURN_IF(check_heads(a.heads, a.head_dim, 1024));
  HC_RETURN_IF(check_heads(a.kv_heads, a.head_dim, 1024));
  HC_RETURN_IF(check_rot(a.rot_dim, a.head_dim));
  HC_RETURN_IF(check_batch(a.page_table, a.kv_lens, a.cu_q, a.tokens, a.seqs, a.max_pages, a.table_stride));
  HC_RETURN_IF(check_cache(a.num_pages, a.cache_page_stride, a.page_size, a.cache_token_stride, a.kv_heads,
                           a.cache_head_stride, a.head_dim));
  HC_RETURN_IF(check_extent("q", a.tokens, a.q_token_stride, a.heads, a.q_head_stride));
  HC_RETURN_IF(check_extent("k", a.tokens, a.k_token_stride, a.kv_heads, a.k_head_stride));
  HC_RETURN_IF(check_extent("v", a.tokens, a.v_token_stride, a.kv_heads, a.v_head_stride));
  HC_RETURN_IF(check_extent("q_out", a.tokens, a.out_token_stride, a.heads, a.out_head_stride));
  if (!strides_valid(a.tokens, a.out_token_stride, a.heads, a.out_head_stride, a.head_dim))
    return fail(HC_ERR_INVALID_ARG, "invalid strides of q_out");
  if (a.tokens * (a.heads + 2 * static_cast<int64_t>(a.kv_heads)) >= (int64_t{1} << 31))
    return fail(HC_ERR_UNSUPPORTED, "tokens * heads beyond 2^31");
  if (a.tokens == 0) return HC_OK;
  if (!a.q || !a.k || !a.v || !a.q_out || !a.k_cache || !a.v_cache || (!a.inv_freq && a.rot_dim > 0))
    return fail(HC_ERR_INVALID_ARG, "null pointer");
  const int64_t es = static_cast<int64_t>(dtype_size(static_cast<hc_dtype_t>(a.dtype)));
  const int64_t pool = es * ((a.num_pages - 1) * a.cache_page_stride +
                             extent(a.page_size, a.cache_token_stride, a.kv_heads, a.cache_head_stride, a.head_dim));
  if (!on_elements(a.dtype, {a.q, a.k, a.v, a.q_out, a.k_cache, a.v_cache}))
    return fail(HC_ERR_INVALID_ARG, "misaligned pointer");
  const bool in_place = a.q_out == a.q && a.out_token_stride == a.q_token_stride && a.out_head_stride == a.q_head_stride;
  const Span q = span("q", a.q, es * extent(a.tokens, a.q_token_stride, a.heads, a.q_head_stride, a.head_dim));
  const Span k = span("k", a.k, es * extent(a.tokens, a.k_token_stride, a.kv_heads, a.k_head_stride, a.head_dim));
  const Span v = span("v", a.v, es * extent(a.tokens, a.v_token_stride, a.kv_heads, a.v_head_stride, a.head_dim));
  const Span qo = span("q_out", a.q_out, es * extent(a.tokens, a.out_token_stride, a.heads, a.out_head_stride, a.head_dim));
  const Span kc = span("k_cache", a.k_cache, pool), vc = span("v_cache", a.v_cache, pool);
  const Span small[4] = {span("inv_freq", a.inv_freq, a.rot_dim * 4), span("kv_lens", a.kv_lens, a.seqs * int64_t{4}),
                         span("cu_q", a.cu_q, (a.seqs + int64_t{1}) * 4),
                         span("page_table", a.page_table, ((a.seqs - 1) * a.table_stride + a.max_pages) * 4)};
  const Span outs[3] = {qo, kc, vc};
  for (const Span& o : outs) HC_RETURN_IF(check_apart(&o, 1, small, 4));
  if (!in_place) {
    const Span ins[3] = {q, k, v};
    HC_RETURN_IF(check_apart(&qo, 1, ins, 3));
  } else {
    // q, k and v may be parts of one matrix's rows
    const auto meets = [&](const Span& other, const void* p, int64_t ts, int64_t hs) {
      if (!overlaps(q, other)) return false;
      return ts != a.q_token_stride || rows_meet(q.lo, extent(1, ts, a.heads, a.q_head_stride, a.head_dim),
                                                 reinterpret_cast<uintptr_t>(p), extent(1, ts, a.kv_heads, hs, a.head_dim), ts,
                                                 a.tokens, es);
    };
    if (meets(k, a.k, a.k_token_stride, a.k_head_stride)) return fail(HC_ERR_INVALID_ARG, "q_out overlaps k");
    if (meets(v, a.v, a.v_token_stride, a.v_head_stride)) return fail(HC_ERR_INVALID_ARG, "q_out overlaps v");
  }
  const Span ins[4] = {q, k, v, qo};
  HC_RETURN_IF(check_apart(&kc, 1, ins, 4));
  HC_RETURN_IF(check_apart(&vc, 1, ins, 4));
  // (the caches may be parts of one pool; heads that begin within one another's features are not)
  if (kc.lo < vc.lo + static_cast<uintptr_t>(es * a.head_dim) && vc.lo < kc.lo + static_cast<uintptr_t>(es * a.head_dim))
    return fail(HC_ERR_INVALID_ARG, "k_cache overlaps v_cache");
  int sms = 0;  // (only to refuse other devices)
  HC_RETURN_IF(hc::current_device_sms(&sms));
  const bool vec = aligned16(a.q) && aligned16(a.k) && aligned16(a.v) && aligned16(a.q_out) && aligned16(a.k_cache) &&
                   aligned16(a.v_cache) &&
                   vec_strides(a.dtype, {a.q_token_stride, a.q_head_stride, a.k_token_stride, a.k_head_stride,
                                         a.v_token_stride, a.v_head_stride, a.out_token_stride, a.out_head_stride,
                                         a.cache_page_stride, a.cache_token_stride, a.cache_head_stride});
  return launched(hc::launch_rotary_append(a, vec, stream));
}

namespace {

hc_status_t check_attention(const hc_paged_attention_t& a) {
  if (!dtype_valid(a.dtype)) return fail(HC_ERR_INVALID_ARG, "invalid dtype %d", a.dtype);
  HC_RETURN_IF(check_heads(a.heads, a.head_dim, 256));
  HC_RETURN_IF(check_heads(a.kv_heads, a.head_dim, 256));
  if (a.heads % a.kv_heads != 0)
    return fail(HC_ERR_INVALID_ARG, "heads %d is not a multiple of kv_heads %d", a.heads, a.kv_heads);
  if (a.window < 0 || a.max_q < 0 || a.max_kv < 0 || !(a.softcap >= 0.0f) || !(a.softcap <= 1e30f) ||
      !(a.scale >= -1e30f && a.scale <= 1e30f))
    return fail(HC_ERR_INVALID_ARG, "invalid window, max_q, max_kv, softcap or scale");
  if (a.flags & ~static_cast<uint32_t>(HC_FLAG_FORCE_GENERAL)) return fail(HC_ERR_INVALID_ARG, "unknown flags");
  HC_RETURN_IF(check_batch(a.page_table, a.kv_lens, a.cu_q, a.tokens, a.seqs, a.max_pages, a.table_stride));
  HC_RETURN_IF(check_cache(a.num_pages, a.cache_page_stride, a.page_size, a.cache_token_stride, a.kv_heads,
                           a.cache_head_stride, a.head_dim));
  HC_RETURN_IF(check_extent("q", a.tokens, a.q_token_stride, a.heads, a.q_head_stride));
  HC_RETURN_IF(check_extent("out", a.tokens, a.out_token_stride, a.heads, a.out_head_stride));
  if (!strides_valid(a.tokens, a.out_token_stride, a.heads, a.out_head_stride, a.head_dim))
    return fail(HC_ERR_INVALID_ARG, "invalid strides of out");
  if (a.tokens * a.heads >= (int64_t{1} << 31) || a.seqs > (1 << 24))
    return fail(HC_ERR_UNSUPPORTED, "tokens * heads beyond 2^31 or more than 2^24 sequences");
  return HC_OK;
}

bool attention_aligned(const hc_paged_attention_t& a) {
  return aligned16(a.q) && aligned16(a.k_cache) && aligned16(a.v_cache) &&
         vec_strides(a.dtype, {a.q_token_stride, a.q_head_stride, a.cache_page_stride, a.cache_token_stride,
                               a.cache_head_stride});
}

}  // namespace

size_t hc_paged_attention_workspace_size(const hc_paged_attention_t* args) {
  int sms = 0;
  if (args == nullptr || check_attention(*args) != HC_OK || args->tokens == 0 ||
      hc::current_device_sms(&sms) != HC_OK)
    return 0;
  return hc::attention_workspace(*args, attention_aligned(*args), sms);
}

hc_status_t hc_paged_attention(const hc_paged_attention_t* args, cudaStream_t stream) {
  if (args == nullptr) return fail(HC_ERR_INVALID_ARG, "null args");
  const hc_paged_attention_t& a = *args;
  HC_RETURN_IF(check_attention(a));
  if (a.tokens == 0) return HC_OK;
  if (!a.q || !a.k_cache || !a.v_cache || !a.out) return fail(HC_ERR_INVALID_ARG, "null pointer");
  const int64_t es = static_cast<int64_t>(dtype_size(static_cast<hc_dtype_t>(a.dtype)));
  const int64_t pool = es * ((a.num_pages - 1) * a.cache_page_stride +
                             extent(a.page_size, a.cache_token_stride, a.kv_heads, a.cache_head_stride, a.head_dim));
  if (!on_elements(a.dtype, {a.q, a.k_cache, a.v_cache, a.out})) return fail(HC_ERR_INVALID_ARG, "misaligned pointer");
  const Span ins[6] = {
      span("q", a.q, es * extent(a.tokens, a.q_token_stride, a.heads, a.q_head_stride, a.head_dim)),
      span("k_cache", a.k_cache, pool),
      span("v_cache", a.v_cache, pool),
      span("page_table", a.page_table, ((a.seqs - 1) * a.table_stride + a.max_pages) * 4),
      span("kv_lens", a.kv_lens, a.seqs * int64_t{4}),
      span("cu_q", a.cu_q, (a.seqs + int64_t{1}) * 4)};
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  const bool aligned = attention_aligned(a);
  const size_t need = hc::attention_workspace(a, aligned, sms);
  if (need > 0 && (a.workspace == nullptr || a.workspace_bytes < need ||
                   (reinterpret_cast<uintptr_t>(a.workspace) & 255u) != 0))
    return fail(HC_ERR_WORKSPACE, "workspace needs %zu bytes at a 256-byte boundary, got %zu", need, a.workspace_bytes);
  const Span outs[3] = {
      span("out", a.out, es * extent(a.tokens, a.out_token_stride, a.heads, a.out_head_stride, a.head_dim)),
      span("lse", a.lse, a.tokens * a.heads * 4),
      span("workspace", need ? a.workspace : nullptr, static_cast<int64_t>(need))};
  HC_RETURN_IF(check_apart(outs, 3, ins, 6));
  return launched(hc::launch_attention(a, aligned, sms, stream));
}

// -------------------------------------------------------------------- pages

namespace {

hc_status_t check_pages(const hc_pages_t* p, bool lens_out, int64_t seqs_out) {
  if (p == nullptr) return fail(HC_ERR_INVALID_ARG, "null pages");
  if (p->num_pages < 1 || p->num_pages >= (int64_t{1} << 31) || p->seqs < 0 || p->max_pages < 1 ||
      p->max_pages > (1 << 20) || p->page_size < 1 || (p->seqs > 1 && p->table_stride < p->max_pages) ||
      !sane(p->table_stride))
    return fail(HC_ERR_INVALID_ARG, "invalid sizes: num_pages=%lld seqs=%d max_pages=%d page_size=%d",
                ll(p->num_pages), p->seqs, p->max_pages, p->page_size);
  if (p->seqs > (1 << 24) || seqs_out > (1 << 24)) return fail(HC_ERR_UNSUPPORTED, "more than 2^24 sequences");
  if (!within(p->seqs, p->table_stride)) return fail(HC_ERR_UNSUPPORTED, "page_table beyond 2^46 entries");
  if (p->refs == nullptr || p->refs_out == nullptr || (p->seqs > 0 && (!p->page_table || !p->lens)) ||
      (seqs_out > 0 && (!p->page_table_out || (lens_out && !p->lens_out))))
    return fail(HC_ERR_INVALID_ARG, "null pointer");
  return HC_OK;
}

// The tables and counts, and what a call has beside them: no output may overlap an input or another output. (With `list` an input
// and `more` outputs; a span of no bytes overlaps nothing.)
hc_status_t check_pages_apart(const hc_pages_t& p, bool lens_out, int64_t seqs_out, const Span& list,
                              std::initializer_list<Span> more) {
  const Span ins[4] = {span("page_table", p.page_table, p.seqs > 0 ? ((p.seqs - 1) * p.table_stride + p.max_pages) * 4 : 0),
                       span("lens", p.lens, p.seqs * int64_t{4}), span("refs", p.refs, p.num_pages * 4), list};
  Span outs[8] = {span("page_table_out", p.page_table_out, seqs_out * p.max_pages * 4),
                  span("lens_out", lens_out ? p.lens_out : nullptr, seqs_out * 4),
                  span("refs_out", p.refs_out, p.num_pages * 4)};
  int n = 3;
  for (const Span& o : more) outs[n++] = o;
  return check_apart(outs, n, ins, 4);
}

hc_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(HC_ERR_WORKSPACE, "workspace needs %zu bytes at a 256-byte boundary, got %zu", need, bytes);
  return HC_OK;
}

hc_status_t check_pool(const void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes) {
  if (planes < 0 || num_pages < 1 || num_pages >= (int64_t{1} << 31) || page_bytes < 1 || page_bytes > (int64_t{1} << 36) ||
      planes > (int64_t{1} << 31))
    return fail(HC_ERR_INVALID_ARG, "invalid pool: planes=%lld num_pages=%lld page_bytes=%lld", ll(planes),
                ll(num_pages), ll(page_bytes));
  if (planes > 0 && num_pages > (int64_t{1} << 50) / planes / page_bytes)
    return fail(HC_ERR_UNSUPPORTED, "pool beyond 2^50 bytes");
  if (planes > 0 && cache == nullptr) return fail(HC_ERR_INVALID_ARG, "null cache");
  return HC_OK;
}

}  // namespace

size_t hc_pages_workspace_size(int64_t num_pages, int32_t seqs) {
  if (num_pages < 1 || num_pages >= (int64_t{1} << 31) || seqs < 0) return 0;
  return hc::pages_workspace(num_pages, seqs);
}

hc_status_t hc_page_copy(void* cache, int64_t planes, int64_t num_pages, int64_t page_bytes, const int32_t* src,
                         const int32_t* dst, int64_t count, cudaStream_t stream) {
  HC_RETURN_IF(check_pool(cache, planes, num_pages, page_bytes));
  if (count < 0 || count > num_pages)
    return fail(HC_ERR_INVALID_ARG, "count %lld is not within the pool's %lld pages", ll(count), ll(num_pages));
  if (count == 0 || planes == 0) return HC_OK;
  if (src == nullptr || dst == nullptr) return fail(HC_ERR_INVALID_ARG, "null pointer");
  const Span pool = span("cache", cache, planes * num_pages * page_bytes);
  const Span ins[2] = {span("src", src, count * 4), span("dst", dst, count * 4)};
  HC_RETURN_IF(check_apart(&pool, 1, ins, 2));
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  return launched(hc::launch_page_copy(cache, planes, num_pages, page_bytes, src, dst, count, sms, stream));
}

hc_status_t hc_page_fork(const hc_pages_t* pages, const int32_t* parents, int32_t children, int32_t* missing, void* cache,
                         int64_t planes, int64_t page_bytes, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream) {
  if (children < 0) return fail(HC_ERR_INVALID_ARG, "invalid children=%d", children);
  HC_RETURN_IF(check_pages(pages, true, children));
  HC_RETURN_IF(check_pool(cache, planes, pages->num_pages, page_bytes));
  if ((children > 0 && parents == nullptr) || missing == nullptr) return fail(HC_ERR_INVALID_ARG, "null pointer");
  const size_t need = hc::pages_workspace(pages->num_pages, std::max(pages->seqs, children));
  HC_RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  HC_RETURN_IF(check_pages_apart(*pages, true, children, span("parents", parents, children * int64_t{4}),
                                 {span("missing", missing, 4), span("cache", cache, planes * pages->num_pages * page_bytes),
                                  span("workspace", workspace, static_cast<int64_t>(need))}));
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  return launched(hc::launch_page_fork(*pages, parents, children, missing, cache, planes, page_bytes, workspace, sms, stream));
}

hc_status_t hc_page_extend(const hc_pages_t* pages, const int32_t* new_tokens, int32_t* missing, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  HC_RETURN_IF(check_pages(pages, true, pages ? pages->seqs : 0));
  if ((pages->seqs > 0 && new_tokens == nullptr) || missing == nullptr) return fail(HC_ERR_INVALID_ARG, "null pointer");
  const size_t need = hc::pages_workspace(pages->num_pages, pages->seqs);
  HC_RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  HC_RETURN_IF(check_pages_apart(*pages, true, pages->seqs, span("new_tokens", new_tokens, pages->seqs * int64_t{4}),
                                 {span("missing", missing, 4), span("workspace", workspace, static_cast<int64_t>(need))}));
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  return launched(hc::launch_page_extend(*pages, new_tokens, missing, workspace, sms, stream));
}

hc_status_t hc_page_release(const hc_pages_t* pages, const uint8_t* drop, cudaStream_t stream) {
  HC_RETURN_IF(check_pages(pages, true, pages ? pages->seqs : 0));
  if (pages->seqs > 0 && drop == nullptr) return fail(HC_ERR_INVALID_ARG, "null pointer");
  HC_RETURN_IF(check_pages_apart(*pages, true, pages->seqs, span("drop", drop, pages->seqs), {}));
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  return launched(hc::launch_page_release(*pages, drop, sms, stream));
}

hc_status_t hc_page_compact(const hc_pages_t* pages, int32_t* remap, int32_t* live, void* cache, int64_t planes,
                            int64_t page_bytes, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  HC_RETURN_IF(check_pages(pages, false, pages ? pages->seqs : 0));
  HC_RETURN_IF(check_pool(cache, planes, pages->num_pages, page_bytes));
  if (remap == nullptr || live == nullptr) return fail(HC_ERR_INVALID_ARG, "null pointer");
  const size_t need = hc::pages_workspace(pages->num_pages, pages->seqs);
  HC_RETURN_IF(check_workspace(workspace, workspace_bytes, need));
  HC_RETURN_IF(check_pages_apart(*pages, false, pages->seqs, span("page_table", nullptr, 0),
                                 {span("remap", remap, pages->num_pages * 4), span("live", live, 4),
                                  span("cache", cache, planes * pages->num_pages * page_bytes),
                                  span("workspace", workspace, static_cast<int64_t>(need))}));
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  return launched(hc::launch_page_compact(*pages, remap, live, cache, planes, page_bytes, workspace, sms, stream));
}

}  // extern "C"
