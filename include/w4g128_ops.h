/*
 * w4g128_ops -- the operators that stand around the weight stream in a decode
 * or verify step: the mixture-of-experts layer on packed int4-g128 experts,
 * attention of a few new tokens over a paged cache, and token sampling.
 * (Token Rush README: the step is captured whole, with attention "over the
 * live length", sampling and the token fed back on the device; progress table
 * steps 4 and 13-14.)  Same conventions as w4g128.h: device pointers owned by
 * the caller, nothing allocated, calls asynchronous on `stream`, argument
 * errors returned before anything is launched, results bitwise deterministic.
 * A workspace must not be used by two calls that can run at the same time,
 * on two streams or in two captured graphs.
 */
#ifndef W4G128_OPS_H
#define W4G128_OPS_H

#include "w4g128.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Status-word code of w4g128_attend: a length, a row offset or a page id in
 * device memory lies outside what the arguments allow. */
#define W4G128_ERR_CACHE 9

/* ------------------------------------------------------------------------
 * SAMPLING
 *
 * One token per row from bf16 logits (the output of an lm_head product) and a
 * given random number u.  Tokens are ordered by falling logit, the lower
 * index first among equals (-0 equals +0), and weighted
 *   w_i = exp((logit_i - largest logit) / temperature).
 * Three filters each keep a prefix of that order, and at least its first
 * token: the first top_k tokens; of those, the tokens whose predecessors' sum
 * is below top_p times the sum of the top_k; the tokens with w_i >= min_p.
 * The token is the first one kept whose sum of weights, itself included,
 * exceeds u times the kept sum; its log-probability among the kept tokens is
 * log(w_i / kept sum).  Logits of -inf and NaN are never chosen.  A row
 * without any other gets token -1 and log-probability -inf.  If the largest
 * logit is +inf, the +inf tokens weigh 1 and all others 0.
 *
 * The weights are carried as 62-bit fractions of the largest and summed
 * exactly, so the token is the one that the formulas give in about 1e-13
 * relative precision, whatever the order of the sums. */
typedef struct {
  const w4g128_bf16* logits; /* row r at logits + r * row_stride; 2-byte aligned */
  long long row_stride;      /* elements, >= vocab */
  const float* temperature;  /* [rows], or NULL: 1.  Not above 0 (or NaN): the largest logit is taken (top_k = 1) */
  const int* top_k;          /* [rows], or NULL: no limit.  Not above 0: no limit */
  const float* top_p;        /* [rows], or NULL: 1.  1 and above (or NaN): no limit */
  const float* min_p;        /* [rows], or NULL: 0.  0 and below (or NaN): no limit */
  const float* u;            /* [rows], in [0, 1); taken as 0 below it (or NaN), as the last fraction below 1 above it */
  int* tokens;               /* [rows] */
  float* logprobs;           /* [rows], or NULL */
  int rows;                  /* 1 .. W4G128_MAX_SAMPLE_ROWS */
  int vocab;                 /* 1 .. W4G128_MAX_VOCAB */
} w4g128_sample_args;

#define W4G128_MAX_SAMPLE_ROWS 4096
#define W4G128_MAX_VOCAB 524160

/* Samples every row.  Needs no workspace.  The arrays named by `args` are
 * device memory and are read and written when the call runs; `args` itself is
 * host memory and is read during the call.  Returns W4G128_ERR_INVALID_ARG
 * (null logits, u or tokens; rows out of range), W4G128_ERR_SHAPE (vocab out
 * of range, row_stride below vocab), W4G128_ERR_ALIGN (logits 2 bytes, the
 * other arrays 4). */
W4G128_API int w4g128_sample(const w4g128_sample_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4G128_OPS_H */
