/*
 * spec_linear.h -- linear attention with a decay for each head, around the verify
 * round of a target whose layers keep a recurrent state.
 *
 * Head h of lane b keeps a state S [dk][dv] in fp32.  Token t of the lane brings a
 * query and a key (head h / (v_heads / k_heads) of k_heads), a value, and a
 * log decay g_t; the recurrence is
 *
 *   S_t = exp(g_t) S_(t-1) + k_t v_t^T          o_t = scale * S_t^T q_t
 *
 *   spec_linear_prefill  whole prompts: outputs of every token and the state after
 *                        the last one
 *   spec_linear_verify   one to a few columns a lane (an anchor and its drafts):
 *                        the live state is read, the state after every column goes
 *                        to the snapshots that spec_commit_state rolls from
 *                        (FreeToken issue #828, "Design": per-request state; ignis
 *                        docs, "One round, step by step", step 5).  One column is
 *                        single-token decoding.
 *
 * The conventions of spec_verify.h hold: device pointers unless stated otherwise,
 * caller-owned buffers, calls enqueue on `stream` and return at once.
 */
#ifndef SPEC_LINEAR_H
#define SPEC_LINEAR_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head size (dk and dv) the calls take. */
#define SPEC_LINEAR_MAX_DIM 256

typedef struct {
  /* Activations of `dtype`, tokens packed lane after lane: q and k are
   * [rows][k_heads][dk], v and out [rows][v_heads][dv], the last dimension
   * contiguous, the other strides in elements as given (>= 0 for inputs). */
  const void* q;
  const void* k;
  const void* v;
  void* out;
  int64_t q_row_stride, q_head_stride;
  int64_t k_row_stride, k_head_stride;
  int64_t v_row_stride, v_head_stride;
  int64_t out_row_stride, out_head_stride;
  /* Log decays g, fp32 [rows][v_heads]; strides in elements, 0 allowed (a decay
   * for each head that is the same for all tokens has row stride 0).  -inf resets
   * the state before the token; NaN and +inf fail the lane, and so may growth (g > 0)
   * whose factor, exp of a sum of g over tokens in a row, is infinite in fp32. */
  const float* log_decay;
  int64_t decay_row_stride, decay_head_stride;
  /* Lane b owns rows row_offsets[b] .. row_offsets[b + 1] - 1 (none: an empty lane,
   * whose state passes through unchanged).  [lanes + 1], ascending, within 0..rows. */
  const int32_t* row_offsets;
  /* States, fp32 [lanes][v_heads][dk][dv], the last two dimensions contiguous;
   * base 16-byte aligned, lane and head strides (elements) multiples of 4.
   * state_in may be NULL: zeros. */
  const float* state_in;
  int64_t state_in_lane_stride, state_in_head_stride;
  /* Prefill: the state after the lane's last token (may be state_in itself; NULL: not
   * wanted).  Verify: snapshot of column c of lane b at state_out + b * lane_stride +
   * c * col_stride; slots past the lane's columns are not written; with cols = 1 it
   * may be state_in itself. */
  float* state_out;
  int64_t state_out_lane_stride, state_out_col_stride, state_out_head_stride;
  /* Read and updated in place, may be NULL: a lane whose status is not SPEC_OK on
   * entry is left out.  SPEC_ERR_LAYOUT: row_offsets descend, leave 0..rows or give
   * the lane more than max_len rows (nothing written).  SPEC_ERR_NONFINITE: the
   * lane's state came to hold an infinity or NaN (its outputs and state are
   * unspecified).  SPEC_ERR_TIMEOUT: a bounded wait gave up (likewise). */
  int32_t* lane_status;
  spec_dtype dtype;
  int32_t lanes, rows, max_len; /* max_len: most rows of one lane; verify: snapshots of a lane */
  int32_t k_heads, v_heads;     /* v_heads a multiple of k_heads                               */
  int32_t dk, dv;               /* 1..SPEC_LINEAR_MAX_DIM, dv a multiple of 4                   */
  float scale;
  /* Prefill only: scratch memory, 16-byte aligned, not shared with a call that may run at
   * the same time; spec_linear_workspace() says how much is of use.  With less of it, or
   * none (NULL), long prompts of few lanes are cut in fewer segments and take longer. */
  void* workspace;
  uint64_t workspace_bytes;
} spec_linear_args;

/*
 * spec_linear_workspace -- the most scratch memory, in bytes, that spec_linear_prefill can
 * use with up to this many lanes and up to max_len tokens a lane on the current device
 * (host-only; 0 if none, also for sizes that the prefill refuses): a buffer for the
 * largest call serves all smaller ones.  It is bounded by one 128 x 128 state for each SM.
 */
uint64_t spec_linear_workspace(int32_t lanes, int32_t v_heads, int32_t dk, int32_t dv, int32_t max_len);

/*
 * spec_linear_prefill -- every token's output and the final states of whole prompts.
 *
 * Errors: SPEC_ERR_INVALID_ARG for NULL required pointers (q, k, v, out, log_decay,
 * row_offsets with lanes and rows > 0), sizes or dtype outside the ranges above,
 * misaligned states or a misaligned workspace; SPEC_ERR_CUDA if a launch fails.
 *
 * Prompts in bf16 with dk and dv up to 128 (max_len >= 8; q, k, v and out 16-byte aligned in
 * base and strides) run in chunks of 128 tokens on the tensor cores; everything else
 * runs token after token, with the same results up to rounding but slower on long
 * prompts.  out must not overlap q, k or v.
 *
 * SPEC_LINEAR_TEST_WITHHOLD_COPY=1 in the environment, tests of the failure path only: the
 * chunked kernel's first CTA never issues its first copy, so that its waits give up
 * after some seconds and its lanes report SPEC_ERR_TIMEOUT.
 */
int spec_linear_prefill(const spec_linear_args* args, void* stream);

/*
 * spec_linear_verify -- the recurrence over each lane's columns, the state after every
 * column staged.  state_in is not written (unless state_out is the same memory).
 *
 * A column's output and snapshot do not depend on the columns after it or on the
 * number of columns: they are bit for bit those of decoding the tokens one call at a
 * time from the previous snapshot.
 *
 * Errors: as spec_linear_prefill, and state_out is required.
 */
int spec_linear_verify(const spec_linear_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LINEAR_H */
