// C ABI of the experts' layer (include/hc_experts.h) and of the choice of tokens
// (include/hc_sample.h): every error is found on the host, before any launch, and
// returned as a status.
#include <cuda_runtime.h>

#include <algorithm>

#include "hc_args.h"
#include "hc_experts_internal.h"

namespace {

using namespace hc::args;
using hc::dtype_size;

// Rows of `width` elements, a step apart. An output's rows must not overlap.
hc_status_t check_rows(const char* name, int64_t rows, int64_t step, int64_t width, bool output) {
  if (!sane(step) || (output && rows > 1 && step < width))
    return fail(HC_ERR_INVALID_ARG, "%s: %lld elements from row to row do not fit rows of %lld", name, ll(step), ll(width));
  if (!within(rows, step)) return fail(HC_ERR_UNSUPPORTED, "%s beyond 2^46 elements", name);
  return HC_OK;
}
int64_t rows_bytes(int64_t rows, int64_t step, int64_t width, int64_t es) {
  return rows < 1 ? 0 : ((rows - 1) * step + width) * es;
}

bool finite(float v) { return v >= -3.4e38f && v <= 3.4e38f; }

// A weight of (experts, inputs, outputs).
hc_status_t check_weight(const char* name, int experts, int inputs, int outputs, int64_t es, int64_t is, int64_t os) {
  const bool by_out = os == 1 && (is >= outputs || inputs == 1), by_in = is == 1 && (os >= inputs || outputs == 1);
  if (!sane(es) || !sane(is) || !sane(os) || !(by_out || by_in))
    return fail(HC_ERR_INVALID_ARG, "%s: strides %lld, %lld, %lld: one of the last two must be 1, the other span its rows", name,
                ll(es), ll(is), ll(os));
  if (!within(experts, es) || !within(inputs, is) || !within(outputs, os))
    return fail(HC_ERR_UNSUPPORTED, "%s beyond 2^46 elements", name);
  return HC_OK;
}
int64_t weight_extent(int experts, int inputs, int outputs, int64_t es, int64_t is, int64_t os) {
  return (experts - 1) * es + (inputs - 1) * is + (outputs - 1) * os + 1;
}

hc_status_t check_mlp(const hc_expert_mlp_t& a) {
  if (!dtype_valid(a.dtype)) return fail(HC_ERR_INVALID_ARG, "invalid dtype %d", a.dtype);
  if (a.flags & ~static_cast<uint32_t>(HC_FLAG_FORCE_GENERAL)) return fail(HC_ERR_INVALID_ARG, "unknown flags");
  if (a.tokens < 0 || a.num_experts < 1 || a.top_k < 1 || a.hidden < 1 || a.inner < 1)
    return fail(HC_ERR_INVALID_ARG, "invalid sizes: tokens=%lld num_experts=%d top_k=%d hidden=%d inner=%d", ll(a.tokens),
                a.num_experts, a.top_k, a.hidden, a.inner);
  if (a.num_experts > 1024 || a.top_k > 32 || a.hidden > 65536 || a.inner > 65536 || a.tokens >= (int64_t{1} << 24) ||
      a.tokens * a.top_k >= (int64_t{1} << 24))
    return fail(HC_ERR_UNSUPPORTED,
                "num_experts=%d top_k=%d hidden=%d inner=%d tokens=%lld: at most 1024, 32, 65536, 65536 and 2^24 - 1 pairs",
                a.num_experts, a.top_k, a.hidden, a.inner, ll(a.tokens));
  HC_RETURN_IF(check_rows("x", a.tokens, a.x_stride, a.hidden, false));
  HC_RETURN_IF(check_rows("out", a.tokens, a.out_stride, a.hidden, true));
  HC_RETURN_IF(check_weight("gate and up", a.num_experts, a.hidden, a.inner, a.up_expert_stride, a.up_in_stride, a.up_out_stride));
  return check_weight("down", a.num_experts, a.inner, a.hidden, a.down_expert_stride, a.down_in_stride, a.down_out_stride);
}

bool mlp_aligned(const hc_expert_mlp_t& a) {
  return aligned16(a.x) && aligned16(a.gate) && aligned16(a.up) && aligned16(a.down) &&
         vec_strides(a.dtype, {a.x_stride, a.up_expert_stride, a.up_in_stride == 1 ? a.up_out_stride : a.up_in_stride,
                               a.down_expert_stride, a.down_in_stride == 1 ? a.down_out_stride : a.down_in_stride});
}

}  // namespace

extern "C" {

hc_status_t hc_expert_route(const hc_expert_route_t* args, cudaStream_t stream) {
  if (args == nullptr) return fail(HC_ERR_INVALID_ARG, "null args");
  const hc_expert_route_t& a = *args;
  if (!dtype_valid(a.dtype)) return fail(HC_ERR_INVALID_ARG, "invalid dtype %d", a.dtype);
  if (a.tokens < 0 || a.experts < 1 || a.groups < 1 || a.experts % std::max(a.groups, 1) != 0 || a.top_groups < 1 ||
      a.top_groups > a.groups || (a.group_best != 1 && a.group_best != 2) || a.top_k < 1 ||
      a.top_k > a.top_groups * static_cast<int64_t>(a.experts / std::max(a.groups, 1)))
    return fail(HC_ERR_INVALID_ARG,
                "invalid sizes: tokens=%lld experts=%d groups=%d top_groups=%d group_best=%d top_k=%d", ll(a.tokens), a.experts,
                a.groups, a.top_groups, a.group_best, a.top_k);
  if (!finite(a.scale)) return fail(HC_ERR_INVALID_ARG, "invalid scale");
  if (a.experts > 1024 || a.groups > 32 || a.top_k > 32 || a.tokens >= (int64_t{1} << 31))
    return fail(HC_ERR_UNSUPPORTED, "experts=%d groups=%d top_k=%d tokens=%lld: at most 1024, 32, 32 and 2^31 - 1", a.experts,
                a.groups, a.top_k, ll(a.tokens));
  HC_RETURN_IF(check_rows("logits", a.tokens, a.logits_stride, a.experts, false));
  if (a.tokens == 0) return HC_OK;
  if (!a.logits || !a.experts_out || !a.weights_out) return fail(HC_ERR_INVALID_ARG, "null pointer");
  if (!on_elements(a.dtype, {a.logits}) || !on_words({a.bias, a.live, a.experts_out, a.weights_out}))
    return fail(HC_ERR_INVALID_ARG, "misaligned pointer");
  const int64_t es = static_cast<int64_t>(dtype_size(static_cast<hc_dtype_t>(a.dtype)));
  const Span ins[3] = {span("logits", a.logits, rows_bytes(a.tokens, a.logits_stride, a.experts, es)),
                       span("bias", a.bias, a.experts * int64_t{4}), span("live", a.live, 4)};
  const Span outs[2] = {span("experts_out", a.experts_out, a.tokens * a.top_k * 4),
                        span("weights_out", a.weights_out, a.tokens * a.top_k * 4)};
  HC_RETURN_IF(check_apart(outs, 2, ins, 3));
  int sms = 0;  // (only to refuse other devices)
  HC_RETURN_IF(hc::current_device_sms(&sms));
  return launched(hc::launch_expert_route(a, stream));
}

size_t hc_expert_mlp_workspace_size(const hc_expert_mlp_t* args) {
  int sms = 0;
  if (args == nullptr || check_mlp(*args) != HC_OK || args->tokens == 0 || hc::current_device_sms(&sms) != HC_OK) return 0;
  return hc::expert_mlp_workspace(*args, mlp_aligned(*args), sms);
}

hc_status_t hc_expert_mlp(const hc_expert_mlp_t* args, cudaStream_t stream) {
  if (args == nullptr) return fail(HC_ERR_INVALID_ARG, "null args");
  const hc_expert_mlp_t& a = *args;
  HC_RETURN_IF(check_mlp(a));
  if (a.tokens == 0) return HC_OK;
  if (!a.x || !a.gate || !a.up || !a.down || !a.experts || !a.weights || !a.out)
    return fail(HC_ERR_INVALID_ARG, "null pointer");
  if (!on_elements(a.dtype, {a.x, a.gate, a.up, a.down, a.out}) || !on_words({a.experts, a.weights}))
    return fail(HC_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  const bool aligned = mlp_aligned(a);
  const size_t need = hc::expert_mlp_workspace(a, aligned, sms);
  if (need > 0 && (a.workspace == nullptr || a.workspace_bytes < need ||
                   (reinterpret_cast<uintptr_t>(a.workspace) & 255u) != 0))
    return fail(HC_ERR_WORKSPACE, "workspace needs %zu bytes at a 256-byte boundary, got %zu", need, a.workspace_bytes);
  const int64_t es = static_cast<int64_t>(dtype_size(static_cast<hc_dtype_t>(a.dtype)));
  const int64_t up = es * weight_extent(a.num_experts, a.hidden, a.inner, a.up_expert_stride, a.up_in_stride, a.up_out_stride);
  const Span ins[6] = {
      span("x", a.x, rows_bytes(a.tokens, a.x_stride, a.hidden, es)),
      span("gate", a.gate, up),
      span("up", a.up, up),
      span("down", a.down, es * weight_extent(a.num_experts, a.inner, a.hidden, a.down_expert_stride, a.down_in_stride,
                                              a.down_out_stride)),
      span("experts", a.experts, a.tokens * a.top_k * 4),
      span("weights", a.weights, a.tokens * a.top_k * 4)};
  const Span outs[2] = {span("out", a.out, rows_bytes(a.tokens, a.out_stride, a.hidden, es)),
                        span("workspace", need ? a.workspace : nullptr, static_cast<int64_t>(need))};
  HC_RETURN_IF(check_apart(outs, 2, ins, 6));
  return launched(hc::launch_expert_mlp(a, aligned, sms, stream));
}

hc_status_t hc_token_sample(const hc_token_sample_t* args, cudaStream_t stream) {
  if (args == nullptr) return fail(HC_ERR_INVALID_ARG, "null args");
  const hc_token_sample_t& a = *args;
  if (!dtype_valid(a.dtype)) return fail(HC_ERR_INVALID_ARG, "invalid dtype %d", a.dtype);
  if (a.rows < 0 || a.vocab < 1) return fail(HC_ERR_INVALID_ARG, "invalid sizes: rows=%lld vocab=%d", ll(a.rows), a.vocab);
  if (a.vocab > hc::kSampleMaxVocab || a.rows >= (int64_t{1} << 24))
    return fail(HC_ERR_UNSUPPORTED, "rows=%lld vocab=%d: at most 2^24 - 1 and %d", ll(a.rows), a.vocab, hc::kSampleMaxVocab);
  HC_RETURN_IF(check_rows("logits", a.rows, a.logits_stride, a.vocab, false));
  if (a.rows == 0) return HC_OK;
  if (!a.logits || !a.uniform || !a.tokens_out) return fail(HC_ERR_INVALID_ARG, "null pointer");
  if (!on_elements(a.dtype, {a.logits}) ||
      !on_words({a.uniform, a.temperatures, a.top_ps, a.min_ps, a.top_ks, a.tokens_out, a.logprobs_out}))
    return fail(HC_ERR_INVALID_ARG, "misaligned pointer");
  const int64_t es = static_cast<int64_t>(dtype_size(static_cast<hc_dtype_t>(a.dtype))), n = a.rows * 4;
  const Span ins[6] = {span("logits", a.logits, rows_bytes(a.rows, a.logits_stride, a.vocab, es)),
                       span("uniform", a.uniform, n),
                       span("temperatures", a.temperatures, n),
                       span("top_ps", a.top_ps, n),
                       span("min_ps", a.min_ps, n),
                       span("top_ks", a.top_ks, n)};
  const Span outs[2] = {span("tokens_out", a.tokens_out, n), span("logprobs_out", a.logprobs_out, n)};
  HC_RETURN_IF(check_apart(outs, 2, ins, 6));
  int sms = 0;
  HC_RETURN_IF(hc::current_device_sms(&sms));
  return launched(hc::launch_token_sample(a, sms, stream));
}

}  // extern "C"
