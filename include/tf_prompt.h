/*
 * The prompt path around the paged latent cache of tf_paged_mla.h: rotary positions, the write of a
 * projection's rows into their pages, the rows back from the pages, and attention of whole prompts whose
 * heads have keys and values of their own.
 *
 * What a model layer does with a batch of prompts (or prompt chunks):
 *   tf_paged_append_rope   the new rows: RMS norm of the latent, rotary key, into the pages
 *   tf_paged_read          the streams' rows, kept prefixes among them, as contiguous bf16 (the caller's
 *                          projections make each head's keys and values of them)
 *   tf_rope_apply          the queries' rotary part
 *   tf_prompt_attend       attention over those keys and values
 * A decode step writes its rows with tf_paged_append_rope, rotates its queries with tf_rope_apply and goes on
 * with tf_paged_mla_attend.  Rows go into a cache through its page table and come back the same way (issue
 * #1142, piece 2); a prompt chunk attends its prefix and itself (the chunked-prefill note, section 1).
 *
 * Packed rows: a call over S streams takes h_n[s] rows of each, those of stream s after those of
 * stream s - 1.  A stream may have none.
 *
 * Conventions as in tf_paged_mla.h: device pointers are prefixed d_, host pointers h_; TF_OK or a negative
 * TF_E_* code; arguments are checked on the host before anything is launched; launches are asynchronous on
 * cuda_stream, on the device that is current and holds the tensors; the host arrays may change as soon as a call
 * returns; the library allocates no device memory.  Calls can be captured into a CUDA graph (those that
 * take a pool once it has had a launch); the graph keeps the host arrays' values.
 */
#ifndef TF_PROMPT_H
#define TF_PROMPT_H

#include <stddef.h>
#include <stdint.h>

#include "tf_paged_mla.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions ----
 * A head's values x[0 .. dim) are dim / 2 pairs; at position p pair i is turned by the angle p f_i:
 *   (a, b) -> A (a cos - b sin, b cos + a sin)
 * Pairs: TF_ROPE_INTERLEAVED (x[2i], x[2i + 1]); TF_ROPE_HALF (x[i], x[i + dim / 2]).
 * Frequencies, in radians a position, with g_i = base^(-2 i / dim):
 *   TF_ROPE_PLAIN    f_i = g_i, A = 1
 *   TF_ROPE_LINEAR   f_i = g_i / factor, A = 1 (position interpolation)
 *   TF_ROPE_YARN     f_i = g_i (1 - r_i) + g_i / factor r_i, A = 0.1 ln(factor) + 1, as YaRN (Peng et al.,
 *                    2023) scales a model that was trained on `original` positions: r_i = clamp((i - lo) /
 *                    max(hi - lo, 0.001), 0, 1), lo = max(0, floor(d(beta_fast))), hi = min(dim - 1, ceil(d(beta_slow))),
 *                    d(b) = dim ln(original / (2 pi b)) / (2 ln base), the pair that turns b times over `original`
 * amplitude > 0 takes the place of A.
 * Angles: a pair's turn per position is kept as a 64-bit fraction of a full turn and multiplied by the
 * position modulo one turn, so an angle at position 2^31 is as good as one at 1 (2^-21 turns, the double's
 * own rounding of f); sines and cosines are fp32, and the turned values are rounded once to bf16. */
#define TF_ROPE_INTERLEAVED 0
#define TF_ROPE_HALF 1
#define TF_ROPE_PLAIN 0
#define TF_ROPE_LINEAR 1
#define TF_ROPE_YARN 2
#define TF_ROPE_MAX_DIM 256

typedef struct {
    int32_t dim;       /* rotated values of a head: a multiple of 16, at most TF_ROPE_MAX_DIM */
    int32_t layout;    /* TF_ROPE_INTERLEAVED or TF_ROPE_HALF */
    int32_t scaling;   /* TF_ROPE_PLAIN, TF_ROPE_LINEAR or TF_ROPE_YARN */
    int32_t reserved;  /* 0 */
    double base;       /* > 1, finite */
    double factor;     /* >= 1, finite; not read for TF_ROPE_PLAIN */
    double original;   /* TF_ROPE_YARN: positions the model was trained on, >= 1 */
    double beta_fast, beta_slow;   /* TF_ROPE_YARN: turns, beta_fast > beta_slow > 0 (32 and 1 are usual) */
    double amplitude;  /* 0: as above */
} tf_rope_desc;

/* Host memory of the caller's, filled in once by tf_rope_make and then only read. */
typedef struct {
    int32_t dim, layout;
    float amplitude;
    uint32_t made;     /* set by tf_rope_make; other calls refuse a table without it */
    uint64_t turn[TF_ROPE_MAX_DIM / 2];   /* of each pair: turns a position, in units of 2^-64 */
} tf_rope;

/* Host arithmetic only.  TF_E_ARG for a null pointer or a value outside what is said above. */
int tf_rope_make(const tf_rope_desc *desc, tf_rope *out);

/* Turns `dim` values of each of H heads in packed rows: row i of stream s to position h_pos[s] + i.
 * Row j's head h starts at d_x + j * x_row + h * x_head (bf16 values; strides in values) and goes to
 * d_y + j * y_row + h * y_head; other values of y are left alone, so a part of a head is turned by pointers to
 * that part.  y may be x with the same strides (in place); it must not overlap x otherwise.  Strides may have
 * any sign and order as long as y's heads do not overlap each other (TF_E_ARG).
 * Errors: TF_E_ARG for a null pointer, a table not made by tf_rope_make, S outside [1, TF_MAX_STREAMS], H
 * outside [1, TF_MAX_HEADS], a negative h_n, or a pointer or stride that is not a multiple of 8 values;
 * TF_E_RANGE for a negative position or one past INT32_MAX; TF_E_UNSUPPORTED for more than 2^31 - 1 rows.  No rows:
 * nothing is launched, and d_x and d_y may be NULL. */
int tf_rope_apply(const tf_rope *rope, const int64_t *h_pos, const int64_t *h_n, int32_t S, int32_t H, const void *d_x,
                  int64_t x_row, int64_t x_head, void *d_y, int64_t y_row, int64_t y_head, void *cuda_stream);

/* ---- append of a projection's rows ----
 * tf_paged_append of packed rows, with what a layer does to them first.  Row j is d_rows + j * row_stride:
 * 512 latent values x and 64 rope values, bf16.  Row i of stream s goes to the stream's row h_pos[s] + i:
 *   latent   x_k rsqrt(mean(x^2) + eps) gain_k   (fp32; d_gain: bf16 [512]; NULL: x as it is)
 *   rope     turned to its position by `rope`, a table of dim 64 (NULL: as it is)
 * each rounded once to bf16.  On FP8 pools the fp32 latent is quantized as in tf_paged_append (scale = amax / 448,
 * codes rounded to nearest even), without a rounding to bf16 before.
 * The norm is fp32 throughout: a square sum past fp32's largest value (values from some 2^59 on) is infinite, and a
 * finite row comes out as zeros; squares below fp32's smallest count as 0 beside eps.
 * Rows that are not finite: a NaN of the fp32 latent (with a gain one in the row makes every value NaN, and an
 * infinity becomes NaN and the row's finite values 0) is NaN when it is read, on pages of either format; on FP8 pages
 * its code is NaN, amax is that of the other values, which keep theirs, and an infinity without a gain makes the
 * scale infinite, so that every value of its row is read as NaN.
 * The same row of a stream must not be written twice in a call (streams that share a page).  A table entry outside
 * the pool is recorded as TF_E_DEVICE and its rows are skipped.
 * Errors: TF_E_ARG for a null pool or host array, S outside [1, TF_MAX_STREAMS], max_pages < 1, a negative
 * h_n, a page table that is not 4-byte aligned, null or unaligned rows (16 bytes; row_stride a multiple of 8 and at least 576) or gain (16 bytes), a table not
 * made by tf_rope_make or of another dim, with a gain an eps that is not a finite number > 0; TF_E_RANGE for a cache outside the pool, a
 * position outside the table or past INT32_MAX, or a NULL table wider than the pool; TF_E_UNSUPPORTED for more than 2^31 - 1 rows.
 * No rows: nothing is launched. */
int tf_paged_append_rope(tf_kvpool *pool, int32_t cache, const int32_t *d_pt, int32_t max_pages, const int64_t *h_pos,
                         const int64_t *h_n, int32_t S, const void *d_rows, int64_t row_stride, const void *d_gain,
                         float eps, const tf_rope *rope, void *cuda_stream);

/* ---- rows back from the pages ----
 * Rows h_from[s] .. h_from[s] + h_n[s] - 1 of every stream, packed: row j's 512 latent values go to
 * d_latent + j * lat_stride and its 64 rope values to d_rope + j * rope_stride (bf16; strides in values).
 * Either pointer may be NULL (that part is not read).  BF16 pages: the stored bits.  FP8 pages: bf16(code * scale),
 * as attention takes them.  Values between the rows are left alone; the two outputs must not overlap each other.  A table entry outside the pool is recorded
 * as TF_E_DEVICE and its rows are left alone.
 * Errors: TF_E_ARG for a null pool or host array, both outputs NULL, S outside [1, TF_MAX_STREAMS], max_pages < 1, a negative
 * h_n, a page table that is not 4-byte aligned, an output that is not 16-byte aligned or a stride that is not a multiple of 8 and at least 512 (64); TF_E_RANGE for a cache outside the
 * pool, rows outside the table or past INT32_MAX, or a NULL table wider than the pool; TF_E_UNSUPPORTED for more than 2^31 - 1 rows.
 * No rows: nothing is launched. */
int tf_paged_read(tf_kvpool *pool, int32_t cache, const int32_t *d_pt, int32_t max_pages, const int64_t *h_from,
                  const int64_t *h_n, int32_t S, void *d_latent, int64_t lat_stride, void *d_rope, int64_t rope_stride,
                  void *cuda_stream);

/* ---- attention of prompts ----
 * Stream s has h_nq[s] query rows, packed, and h_nk[s] keys, packed on their own.  H query heads share Hkv key
 * heads: head h reads key head h / (H / Hkv).  For query row i of a stream:
 *   s_j = scale q_i . k_j,   j < n = nk - nq + i + 1 (causal: the queries are the stream's last rows), else n = nk
 *   out_i = sum_j softmax(s)_j v_j  (bf16);   lse_i = log sum_j exp(s_j)  (fp32, [rows][H], may be NULL)
 * A row that sees no key (no keys at all, or more queries than keys) gives out 0 and lse -inf.
 * dqk and dv: (64, 64), (128, 128) or (192, 128).  The heads' values lie by strides (tf_heads), so the keys and
 * values of one joint projection are passed as they are.  With d_kr the last 64 of a key's dqk values are those of
 * d_kr + row * kr_row, the same for every head (a rotary key), and k holds the dqk - 64 others.
 * Scores are bf16 products summed in fp32, the softmax is fp32, its weights are rounded to bf16 for the second
 * product (relative 2^-8 each, as in tf_paged_mla_attend).  Work is dealt out by the batch's sizes, so a row's bits
 * may differ (within rounding) between batches, and are the same on every call of one batch.  Keys are summed in parts
 * of 131,072 at most (the tensor cores' sums are cut, not rounded, and lose up to 2^-10 over one) that fp32 joins: longer
 * streams need a workspace.  On a TF_POOL_BATCH_INVARIANT pool keys are split there alone, so that a stream has the same
 * bits whatever else is in the batch (a few rows over a long context are slower: one SM a key head); the workspace is as
 * on other pools or smaller, and tf_prompt_plan_info tells of the others.
 * What other streams hold, NaN included, never reaches a stream's outputs, and a NaN or infinity among its own keys or
 * values reaches no row that does not see it: bits stay, but for the column of a value that is not finite in rows of the
 * same 128-row query tile, which are made again and may be rounded in another way (slowly: a microsecond for some three
 * keys of a row).  A row that sees a value that is not finite has NaN in its column, or that infinity.
 * out's rows and heads may lie in any order but must not overlap each other (TF_E_ARG), nor anything that the call reads.
 * d_ws: tf_prompt_workspace_bytes(...) bytes, 256-byte aligned (NULL if that is 0): partial sums of streams whose
 * keys are split.  Not to be shared by calls that may run at the same time.
 * pool: its device error word takes what a kernel records (a wait that ran out); its pages are not read.
 * Errors: TF_E_ARG for a null pointer (k, v and kr may be NULL without keys; q and out without rows), S outside [1, TF_MAX_STREAMS],
 * H outside [1, TF_MAX_HEADS], Hkv that does not divide H, negative counts, a scale that is not a number > 0
 * (below 2^127), a causal other than 0 or 1, a pointer that is not 16-byte aligned (d_lse: 4) or a stride that is not a multiple of 8 values, below 1 or
 * above 2^36 (out's strides may be any multiple of 8; so may the head stride of a single head), an unaligned or missing workspace; TF_E_NOMEM for
 * one that is too small; TF_E_UNSUPPORTED for other dqk and dv, with d_kr a dqk of 64, or more than 2^31 - 1 rows, keys or tiles of work. */
typedef struct {
    void *d_p;          /* bf16; value c of head h of row j at d_p + j * row + h * head + c */
    int64_t row, head;  /* strides in values */
} tf_heads;

size_t tf_prompt_workspace_bytes(const int64_t *h_nq, const int64_t *h_nk, int32_t S, int32_t H, int32_t Hkv, int32_t dqk,
                                 int32_t dv, int32_t causal);

int tf_prompt_attend(tf_kvpool *pool, const int64_t *h_nq, const int64_t *h_nk, int32_t S, int32_t H, int32_t Hkv,
                     int32_t dqk, int32_t dv, const tf_heads *q, const tf_heads *k, const void *d_kr, int64_t kr_row,
                     const tf_heads *v, float scale, int32_t causal, const tf_heads *out, float *d_lse, void *d_ws,
                     size_t ws_bytes, void *cuda_stream);

/* The work plan of that call, for inspection (host arithmetic only).  sms <= 0: the current device's.
 *   info->items   work items: (stream, key head, block of query rows, split of the keys)
 *   info->rows    query rows (tokens times heads of a key head) that an item's accumulators hold, at most 256
 *   info->splits  most splits of one stream's keys (1: no second launch)
 *   info->slots   128-row slots of fp32 partials in the workspace
 * Errors: TF_E_ARG for a null info, and what the workspace's size refuses. */
typedef struct {
    int64_t items, slots;
    int32_t rows, splits;
} tf_prompt_plan;

int tf_prompt_plan_info(const int64_t *h_nq, const int64_t *h_nk, int32_t S, int32_t H, int32_t Hkv, int32_t dqk,
                        int32_t dv, int32_t causal, int32_t sms, tf_prompt_plan *info);

#ifdef __cplusplus
}
#endif

#endif /* TF_PROMPT_H */
