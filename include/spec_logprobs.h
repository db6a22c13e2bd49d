/*
 * spec_logprobs.h -- log probabilities of given tokens, with the entropy of their rows
 * and the likeliest alternatives.
 *
 * A serving loop reports these for the tokens a verify round committed: the logit rows
 * are the round's, the tokens its out_tokens.  The conventions of spec_verify.h hold:
 * device pointers unless stated otherwise, caller-owned buffers, calls enqueue on
 * `stream` and return at once.
 */
#ifndef SPEC_LOGPROBS_H
#define SPEC_LOGPROBS_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most alternatives a row can report. */
#define SPEC_LOGPROBS_MAX_TOP 20

typedef struct {
  const void* logits;          /* [rows][ld] of dtype                                        */
  spec_dtype dtype;
  int64_t ld;                  /* row stride in elements, >= V                               */
  int32_t V;                   /* vocabulary size, > 0                                       */
  int32_t rows;                /* >= 0                                                       */
  const int32_t* tokens;       /* [rows]; a negative token asks for nothing: its row is not
                                  read, its numbers are 0 and its ids -1                      */
  const float* temperatures;   /* [rows], may be NULL; T > 0 scales the row by 1 / T, T <= 0
                                  (a greedy row) leaves it as it is                           */
  float* logprobs;             /* out [rows]: log p(token), p = softmax(x / T)                */
  float* entropy;              /* out [rows], may be NULL: -sum p log p (nats)                */
  int32_t top;                 /* 0..SPEC_LOGPROBS_MAX_TOP alternatives a row                 */
  int32_t* top_ids;            /* out [rows][top]: the row's likeliest tokens, likeliest
                                  first, ties by lowest id; -1 past the vocabulary's end       */
  float* top_logprobs;         /* out [rows][top]: their log p (-inf with id -1)              */
  int32_t* row_status;         /* out [rows], may be NULL: SPEC_OK; SPEC_ERR_TOKEN_RANGE for a
                                  token >= V; SPEC_ERR_NONFINITE for a row that holds NaN or
                                  +inf, or -inf only; SPEC_ERR_TIMEOUT if a bounded wait gave
                                  up.  Such a row's numbers are NaN, its ids -1               */
} spec_logprobs_args;

/*
 * spec_token_logprobs -- one pass over the logit rows.
 *
 * -inf logits have probability 0; -0 counts as +0.  Errors: SPEC_ERR_INVALID_ARG for
 * NULL required pointers (logits, tokens, logprobs; top_ids and top_logprobs with
 * top > 0), V <= 0, rows < 0, ld < V, top out of range or an unknown dtype;
 * SPEC_ERR_CUDA if the launch fails.  rows = 0 is a no-op.
 *
 * Rows whose address is 16-byte aligned (base and ld * element size) are fastest; others are
 * streamed from the aligned 16 bytes that their start lies in (what is before it is not used)
 * and taken apart element by element, with the same results.
 * SPEC_LOGPROBS_TEST_WITHHOLD_COPY=1 in the environment, tests of the failure path only:
 * the first row's first copy is never issued, so that its wait gives up after 2 s; with 2
 * the first copy of its second look, at the blocks that hold the alternatives.
 */
int spec_token_logprobs(const spec_logprobs_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGPROBS_H */
