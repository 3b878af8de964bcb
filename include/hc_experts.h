/* hc_experts.h -- C ABI of the feed-forward layer whose weights belong to
 * experts, the other layer that a decoder runs between two hyper-connection
 * blocks when it serves (GB300, sm_103a): routing of tokens to experts, and
 * the products of the chosen experts.
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
 * the message. */
#ifndef HC_EXPERTS_H
#define HC_EXPERTS_H

#include <stddef.h>
#include <stdint.h>

#include "hc_lowrank_mix.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- routing --
 *
 * With the logits x_e of a token, its scores are s = softmax(x) over all
 * experts, or s_e = 1 / (1 + exp(-x_e)) with `sigmoid`. What is compared is
 * c_e = s_e + bias_e. The experts are `groups` runs of equal length; a group
 * counts as the sum of its group_best (1 or 2) largest c_e, and the top_groups
 * best groups stay. Of their experts the top_k with the largest c_e are chosen,
 * in that order. Wherever two values are equal, the lower index comes first;
 * values are compared as the real numbers that the inputs define (rounding of
 * intermediate results does not change the order, down to differences of about
 * 1e-15 of the values). The weights are the scores of the chosen (without the
 * bias), with `renormalise` divided by their sum, times `scale`.
 *
 * A NaN among the logits counts as minus infinity, a NaN among the biases as
 * a bias of minus infinity. An expert whose logit is minus infinity has the
 * score 0; a token without any other logit has scores of 0, and weights of 0.
 * Logits of plus infinity share a softmax among them, and all others have the
 * score 0. Where a bias is given or two values of a group count, scores below
 * 1e-300 are 0. live: the rows from
 * live[0] on are no token's: they get experts of -1 and weights of 0 (NULL: all
 * rows are tokens'). Limits: experts <= 1024, groups <= 32, top_k <= 32. */
typedef struct {
  const void* logits;  /* (tokens, experts) of type dtype */
  const float* bias;   /* (experts), or NULL */
  const int32_t* live; /* (1), or NULL */
  int32_t* experts_out; /* (tokens, top_k) */
  float* weights_out;   /* (tokens, top_k) */
  int64_t tokens, logits_stride; /* elements from row to row */
  int32_t experts, top_k, groups, top_groups, group_best;
  int32_t sigmoid, renormalise;
  int32_t dtype; /* hc_dtype_t */
  float scale;
} hc_expert_route_t;

hc_status_t hc_expert_route(const hc_expert_route_t* args, struct CUstream_st* stream);

/* --------------------------------------------------------------- products --
 *
 *   out_t = sum_j weights[t, j] * (silu(x_t gate_e) * (x_t up_e)) down_e,  e = experts[t, j]
 *
 * with silu(a) = a / (1 + exp(-a)), element by element. Entries of `experts`
 * outside 0 .. num_experts - 1 take no part (-1 for rows that are no token's);
 * a row without any other gets zeros. An expert may be listed twice for a token.
 *
 * Element (e, i, o) of a weight lies at e * expert_stride + i * in_stride +
 * o * out_stride, where one of the last two is 1: weights with contiguous
 * outputs, or with contiguous inputs as checkpoints keep them. gate and up have
 * the same strides.
 *
 * Numerics: products are summed in fp32. In the fp16/bf16 kernels the inner
 * values silu(.) * (.) are rounded to T for the product with down (the tensor
 * core's operands are 16 bits; a value below 2^-251 of its x up is 0). Each chosen expert's result is fp32, and so is
 * the sum over them, rounded to T once. Finite inner values beyond
 * fp16's largest one count in full: what that leaves of them is multiplied with
 * down in fp32, a row of down for each. Limits: top_k <= 32, num_experts <= 1024,
 * hidden and inner <= 65536, tokens * top_k < 2^24. */
typedef struct {
  const void* x; /* (tokens, hidden) of type dtype */
  const void *gate, *up, *down; /* (num_experts, hidden, inner) twice, (num_experts, inner, hidden) */
  const int32_t* experts; /* (tokens, top_k) */
  const float* weights;   /* (tokens, top_k) */
  void* out; /* (tokens, hidden) */
  void* workspace;
  size_t workspace_bytes;
  int64_t tokens, x_stride, out_stride; /* elements from row to row */
  int64_t up_expert_stride, up_in_stride, up_out_stride;       /* of gate and up */
  int64_t down_expert_stride, down_in_stride, down_out_stride; /* of down */
  int32_t num_experts, top_k, hidden, inner;
  int32_t dtype; /* hc_dtype_t */
  uint32_t flags; /* HC_FLAG_FORCE_GENERAL or 0 */
} hc_expert_mlp_t;

/* Bytes of workspace for these sizes, strides and flags (pointers are not
 * looked at but for alignment, out and workspace not at all). */
size_t hc_expert_mlp_workspace_size(const hc_expert_mlp_t* args);
hc_status_t hc_expert_mlp(const hc_expert_mlp_t* args, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_EXPERTS_H */
