/*
 * spec_cache.h -- a paged key/value cache and the attention that reads it, around the
 * verify round of a target with attention layers.
 *
 * A lane's tokens lie in pages of page_size slots: position p of lane b is slot
 * p % page_size of page block_tables[b][p / page_size].  A call's columns (one for decoding, an anchor and its
 * drafts for a verify round, a prompt's part for prefill) follow the cached_lens[b] tokens that the lane's
 * cache holds before the call: column i is at position cached_lens[b] + i.
 *
 *   spec_cache_write      the columns' keys and values go into their slots, rounded to
 *                         the cache's type
 *   spec_cache_read       slots come back as the values they stand for
 *   spec_paged_attention  the columns attend over the slots up to their own
 *
 * A round writes its columns, attends, verifies, and adds each lane's committed count to
 * cached_lens (FreeToken issue #828, "Design": rejected drafts leave nothing behind; ignis docs, "One round,
 * step by step", step 5): the slots of rejected drafts are written over by the next round.
 *
 * Types of the cache.  SPEC_CACHE_BF16 holds numbers as they are.  The 8-bit types hold, for
 * each token and head, numbers y and a power of two 2^e as the byte e + 127; they stand
 * for y 2^e.  e is the least integer of SPEC_CACHE_LEAST_EXP or more with
 * top * 2^e >= max |x|, and y is x / 2^e rounded to nearest, ties to even: to an e4m3
 * number (top 448) or to an integer (top 127).  A head that holds NaN, an infinity or a number beyond
 * top * 2^SPEC_CACHE_MOST_EXP gets the byte 255 and reads back as NaN.  (Attention
 * takes these bytes; what others give is unspecified.)  With a power of two every step but
 * the rounding is exact: what is stored is a function of the numbers alone, and it reads back exactly,
 * in bf16 too.
 *
 * The conventions of spec_verify.h hold: device pointers unless stated otherwise,
 * caller-owned buffers, calls enqueue on `stream` and return at once.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head size the calls take, and the exponents of the 8-bit types. */
#define SPEC_CACHE_MAX_DIM 256
#define SPEC_CACHE_LEAST_EXP (-48)
#define SPEC_CACHE_MOST_EXP 48

typedef enum { SPEC_CACHE_BF16 = 1, SPEC_CACHE_E4M3 = 2, SPEC_CACHE_INT8 = 3 } spec_cache_type;

/* The cache and the lanes' places in it. */
typedef struct {
  /* Keys and values of `type`, [pages][page_size][kv_heads][dim] in whatever order the
   * strides (in elements, the same for both, >= 0) say, the last dimension contiguous;
   * bases 16-byte aligned, strides multiples of 16 bytes.  With u the largest power of two
   * up to 64 KB that divides the three strides in bytes, the last head lies less than 2^32 u bytes
   * behind the first (64 GB at least). */
  void* k_pages;
  void* v_pages;
  int64_t page_stride, slot_stride, head_stride;
  /* 8-bit types: the exponents' bytes, [pages][page_size][kv_heads], strides as given
   * (>= 0).  NULL for SPEC_CACHE_BF16. */
  uint8_t* k_exps;
  uint8_t* v_exps;
  int64_t exp_page_stride, exp_slot_stride, exp_head_stride;
  /* [lanes][table_width], rows table_stride apart (>= table_width). */
  const int32_t* block_tables;
  int64_t table_stride;
  const int32_t* cached_lens;  /* [lanes] */
  /* Lane b owns rows row_offsets[b] .. row_offsets[b + 1] - 1 (none: nothing to do).
   * [lanes + 1], ascending, within 0..rows.  (Where they are not, each lane goes by its own two; what a row
   * of two lanes is given, is one of theirs.) */
  const int32_t* row_offsets;
  /* Read and updated in place (to be read when the call's work is done), may be NULL: a lane whose
   * status, one of spec_verify.h's, is not SPEC_OK on entry is left out, and its status stays.  Otherwise a
   * lane's first error is reported.  SPEC_ERR_LAYOUT: row_offsets descend, leave 0..rows or give the lane more
   * than max_len rows; cached_lens is negative or the lane's last position lies beyond
   * its table; a page that the lane needs is outside 0..pages - 1 (never read or
   * written).  SPEC_ERR_NONFINITE, SPEC_ERR_TIMEOUT: see the calls.  A failed lane's
   * outputs, and its columns' slots, are unspecified; other lanes' are not touched by it. */
  int32_t* lane_status;
  spec_cache_type type;
  int32_t pages, page_size;     /* > 0 */
  int32_t table_width;          /* pages of a lane, >= 0 */
  int32_t lanes, rows, max_len; /* max_len: most rows of one lane */
  int32_t kv_heads;             /* > 0 */
  int32_t dim;                  /* head size, a multiple of 16, 16..SPEC_CACHE_MAX_DIM */
} spec_paged_cache;

typedef struct {
  spec_paged_cache cache;
  /* The columns' keys and values, [rows][kv_heads][dim] of `dtype`, lanes packed one after the
   * other, the last dimension contiguous, the other strides in elements as given (>= 0 when
   * they are read, > 0 when written); bases 16-byte aligned, strides multiples of 16 bytes. */
  void* k;
  void* v;
  int64_t k_row_stride, k_head_stride;
  int64_t v_row_stride, v_head_stride;
  spec_dtype dtype;
} spec_cache_rows_args;

/*
 * spec_cache_write -- the columns' keys and values into their slots (k and v are read).
 *
 * SPEC_ERR_NONFINITE for a lane with a key or value that the cache cannot hold (8-bit types:
 * above; bf16: NaN, an infinity, or an fp32 number that rounds to one).
 * Two lanes must not write one slot.  Errors: SPEC_ERR_INVALID_ARG for NULL
 * required pointers, sizes, types, strides or alignments outside the ranges above;
 * SPEC_ERR_CUDA if a launch fails.  lanes = 0 is a no-op.
 */
int spec_cache_write(const spec_cache_rows_args* args, void* stream);

/*
 * spec_cache_read -- slots back into packed rows (k and v are written): row i of lane b is the
 * token at position cached_lens[b] + i, so that cached_lens of 0 and as many rows as the lane
 * has tokens give all of them.  Values come back exactly, in bf16 as in fp32.
 * Errors: as spec_cache_write.  Values that are not finite are no error.
 */
int spec_cache_read(const spec_cache_rows_args* args, void* stream);

typedef struct {
  spec_paged_cache cache;
  /* Queries and outputs, bf16 [rows][q_heads][dim], the last dimension contiguous, the other
   * strides in elements, multiples of 8 (>= 0 for q, > 0 for out); bases 16-byte aligned.  Query head h reads
   * head h / (q_heads / kv_heads) of the cache. */
  const void* q;
  void* out;
  int64_t q_row_stride, q_head_stride;
  int64_t out_row_stride, out_head_stride;
  /* May be NULL: the natural logarithm of each row's sum of exp(scores), fp32
   * [rows][q_heads], rows lse_row_stride apart (parts of a context that were attended
   * to apart are merged by it). */
  float* lse;
  int64_t lse_row_stride;
  int32_t q_heads;     /* a multiple of kv_heads */
  int32_t window;      /* > 0: a column sees itself and the window - 1 positions before it; 0: all */
  int32_t max_context; /* most positions of one lane, its columns among them (a lane with more
                          fails with SPEC_ERR_LAYOUT); 0: as many as its table holds */
  float scale;         /* scores = scale * q . k */
  /* Scratch memory, 16-byte aligned, not shared with a call that may run at the same time; may be
   * NULL.  spec_paged_attention_workspace() says how much is of use.  With less, no lane's context
   * is split over thread blocks, and few lanes with long contexts take longer. */
  void* workspace;
  uint64_t workspace_bytes;
} spec_paged_attention_args;

/*
 * spec_paged_attention_workspace -- the most scratch memory, in bytes, that
 * spec_paged_attention can use with these heads and up to max_len columns a lane on the
 * current device (host-only; 0 for sizes that it refuses).  It does not depend on lanes or contexts,
 * and a buffer for more columns serves fewer.
 */
uint64_t spec_paged_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t max_len);

/*
 * spec_paged_attention -- softmax attention of each lane's columns over its cache.
 *
 * Column i of a lane sees positions 0 .. cached_lens + i (the last window of them):
 * its own and what is before it, which spec_cache_write has put there.  Every column
 * sees one position at least.  Slots that no column of the lane sees may hold anything, NaN
 * included, and rows behind the last lane's are left as they are.  out must not overlap q.
 *
 * Scores, sums and the output's sum are fp32; the weights enter the second product
 * rounded to bf16 (8-bit caches: with the value's 2^e to fp16, off by 2^-11 of their own or, with many
 * columns, 2^-25 of the row's largest, 2^-32 with few), the output is rounded once more.
 * SPEC_ERR_NONFINITE for a lane with an output that is not finite, as when a query, or a value that one of its
 * columns sees, is not, or a key that makes a score NaN or +inf.  (A score of -inf is no error: its position
 * weighs nothing.)  SPEC_ERR_TIMEOUT: a bounded wait gave up.
 *
 * Errors: SPEC_ERR_INVALID_ARG as above, for q_heads that are no multiple of kv_heads, a
 * negative window or max_context or a misaligned workspace; SPEC_ERR_CUDA if a launch fails.
 * lanes = 0 is a no-op.
 *
 * SPEC_PAGED_TEST_WITHHOLD_COPY=1 in the environment, tests of the failure path only: the thread block with
 * the first position never gets one of its first copies (with many columns: hands on its first tile), so that
 * its waits give up after some seconds and its lanes report SPEC_ERR_TIMEOUT.
 */
int spec_paged_attention(const spec_paged_attention_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
