/* hc_sample.h -- C ABI of the end of a serving step (GB300, sm_103a): the next
 * tokens, drawn from the logits with random numbers that the caller gives.
 *
 * Memory, streams, determinism and errors are as in hc_paged.h. */
#ifndef HC_SAMPLE_H
#define HC_SAMPLE_H

#include <stddef.h>
#include <stdint.h>

#include "hc_lowrank_mix.h"

#ifdef __cplusplus
extern "C" {
#endif

/* With the logits x_i of a row and m their largest:
 *
 *   w_i = exp((x_i - m) / temperature)
 *   top_k > 0: only the top_k tokens with the largest x_i stay
 *   top_p < 1: of those, in the order of falling x_i, a token stays while the
 *              w before it come to less than top_p times the sum of all that
 *              top_k left (the first one always stays)
 *   min_p > 0: of those, the tokens with w_i >= min_p stay (the largest w is 1)
 *
 * where equal x_i are ordered by their index. The token is the first one, in
 * the order of the index, for which the w_i that stay, added up to it and with
 * it, come to more than uniform * (their sum); its log-probability is
 * log(w_i / sum). A temperature of 0 (or less, or NaN) takes the largest logit,
 * the first of equal ones, with a log-probability of 0.
 *
 * Weights are formed and added as integers, so that sums are exact whatever
 * their order. In units of 2^-43 of the largest, each is within about 2^-38 of
 * its own size; in calls that filter nothing and have 2^21 logits or more,
 * within 2^-30 of it, in units of 2^-43 or less of the largest of each 512
 * logits. A result differs from the definition above only where a sum comes
 * within about that much of what it is compared with. A token whose weight is
 * below 2^-44 is not drawn.
 *
 * Per-row parameters are arrays, or with a NULL pointer one value for all rows.
 * top_k <= 0, top_p >= 1 (or NaN) and min_p <= 0 (or NaN) leave everything;
 * top_p <= 0 leaves the first token; min_p > 1 is 1. uniform is cut to 0 .. 1 (NaN: 0).
 * A NaN among the logits counts as minus infinity. Logits of plus infinity
 * share a row among them. A row without any logit above minus infinity gets
 * the token -1 and a log-probability of minus infinity. Limit: vocab <= 409600. */
typedef struct {
  const void* logits;   /* (rows, vocab) of type dtype */
  const float* uniform; /* (rows) */
  const float *temperatures, *top_ps, *min_ps; /* (rows), or NULL */
  const int32_t* top_ks;                       /* (rows), or NULL */
  int32_t* tokens_out;  /* (rows) */
  float* logprobs_out;  /* (rows), or NULL */
  int64_t rows, logits_stride; /* elements from row to row */
  int32_t vocab;
  int32_t top_k;
  float temperature, top_p, min_p;
  int32_t dtype; /* hc_dtype_t */
} hc_token_sample_t;

hc_status_t hc_token_sample(const hc_token_sample_t* args, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* HC_SAMPLE_H */
