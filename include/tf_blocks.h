/*
 * Sparse attention over blocks that a cheap score selects for each query row, and attention of
 * streams that share a prefix, over the paged latent cache of tf_paged_mla.h.
 *
 * A block is TF_BLOCK_ROWS rows of a stream that follow one another: block b of a stream is its rows
 * 64 b .. 64 b + 63, as many of them as the stream holds, and a page is eight blocks.  A step of
 * sparse attention is four calls:
 *   tf_block_keys_update        after the append: the mean row of the blocks that got rows
 *   tf_block_scores             a score of every visible block for each query row
 *   tf_topk_blocked             the k best of each score row (its d_idx are block numbers)
 *   tf_paged_mla_attend_blocks  each query row over its own k blocks
 *
 * Pooled index keys, and scores that add the rectified products of all heads, are the TensorFold
 * pages' way to choose rows (issue #1142, "What happens now" and piece 2); streams hold prefix pages by
 * reference (PR #1732, "What this changes").
 *
 * Conventions as in tf_paged_mla.h: device pointers are prefixed d_, host pointers h_; TF_OK or a
 * negative TF_E_* code; arguments are checked on the host before anything is launched; launches are
 * asynchronous on cuda_stream, on the device that is current and holds the pool, and the host arrays
 * may change as soon as a call returns; the library allocates no device memory.  Calls can be
 * captured into a CUDA graph once the pool has had a launch; the graph keeps the host arrays' values.
 */
#ifndef TF_BLOCKS_H
#define TF_BLOCKS_H

#include <stddef.h>
#include <stdint.h>

#include "tf_paged_mla.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TF_BLOCK_ROWS 64

/* ---- block keys ----
 * The key of a block is the mean of its rows: 512 latent and 64 rope values, each added up in fp32,
 * divided by the number of rows the stream holds of the block and rounded once to bf16.  On FP8
 * pages a latent value is bf16(code * scale), as attention takes it.  Keys lie by pool page, so
 * streams that share a page share its keys: bf16 [num_pages][8][576], 9,216 bytes a page, one such
 * array for each cache, owned by the caller.  A page that one stream has filled only in part must not
 * be another stream's too (as for tf_paged_append).
 *
 * tf_block_keys_update averages, for every stream s < S, each block that holds a row of
 * [h_from[s], h_len[s]), from all its rows up to h_len[s].  After an append of n rows at pos that is
 * h_from = pos, h_len = pos + n.  h_from[s] == h_len[s] leaves the stream's keys alone.  Keys of no
 * other block are read or written.
 * Keys do not move with rows: pages that tf_state_copy_rows filled, and pages of a pool that came with its
 * rows, hold whatever keys their last owner left until an update from h_from = 0 (or a copy of the source
 * pages' keys, for whole pages).
 * d_pt / max_pages as in tf_paged_append.  d_bkeys: 16-byte aligned.  A table entry outside the pool is
 * recorded as TF_E_DEVICE and its blocks are skipped.
 * Errors: TF_E_ARG for a null pointer, S outside [1, TF_MAX_STREAMS], max_pages < 1 or an unaligned
 * d_bkeys; TF_E_RANGE for a cache outside the pool, h_from outside [0, h_len], h_len past the table, or a
 * NULL table wider than the pool; TF_E_UNSUPPORTED for h_len above INT32_MAX or 2^31 blocks in a call. */
size_t tf_block_keys_bytes(const tf_kvpool *pool);   /* of one cache; 0 for NULL */

int tf_block_keys_update(tf_kvpool *pool, int32_t cache, const int32_t *d_pt, int32_t max_pages,
                         const int64_t *h_from, const int64_t *h_len, int32_t S, void *d_bkeys, void *cuda_stream);

/* ---- block scores ----
 * Query row r of stream s is at position pos = h_len[s] - R + r; its own block is own = pos / 64.  For
 * each block b of 0 .. own:
 *   score[s,r,b] = sum_h w[s,r,h] max(0, scale q[s,r,h] . k_b)        bf16 products, fp32 sums
 * but +inf for b < sink and for b > own - local: the first `sink` blocks and the last `local` ones, the
 * row's own among them, are always chosen first.  local is at least 1, so no score depends on a row
 * behind the query: every other block is full and lies before the row's own.  A NaN in a query, a key or a
 * weight makes the scores NaN that it enters (tf_topk_blocked ranks those below all others).
 * d_q: bf16 [S][R][H][576], the queries of the attention; d_w: fp32 [S][R][H], or NULL for ones.
 * d_scores: fp32 [S * R][ld], ld a multiple of 4 and at least cols, the blocks of the longest stream.
 *   Columns 0 .. cols - 1 of every row are written (-inf behind the row's own block), the others left.
 * d_nblk: int32 [S * R], each row's visible blocks own + 1 (d_len of tf_topk_blocked), or NULL.
 * d_bkeys, d_q and d_scores: 16-byte aligned.  A table entry outside the pool is recorded as
 * TF_E_DEVICE and the scores of its blocks are undefined.
 * Errors: TF_E_ARG for a null pointer other than d_pt, d_w and d_nblk, S, R, H, max_pages, sink < 0, local < 1,
 * ld, scale or alignment outside what is said here and in tf_paged_mla_attend; TF_E_RANGE for a length
 * below R or past the table, or a NULL table wider than the pool; TF_E_UNSUPPORTED for a length above INT32_MAX
 * or S * R * H above 2^30. */
int tf_block_scores(tf_kvpool *pool, const void *d_bkeys, const int32_t *d_pt, int32_t max_pages,
                    const int64_t *h_len, int32_t S, int32_t R, int32_t H, const void *d_q, const float *d_w, float scale,
                    int32_t sink, int32_t local, float *d_scores, int64_t ld, int32_t *d_nblk, void *cuda_stream);

/* ---- attention over listed blocks ----
 * Query row r of stream s, at position pos = h_len[s] - R + r, attends the keys of its listed blocks that it
 * can see: rows j <= pos of the blocks d_blk[s][r][0 .. n), n = min(max_blk, pos / 64 + 1); the list's
 * other entries are not read.
 *   s_j = scale * (q[s][r][h][0:512] . C_j + q[s][r][h][512:576] . Kr_j)
 *   out[s][r][h][:] = sum_j softmax(s)_j * C_j;  lse[s][r][h] = log sum_j exp(s_j).
 * An entry of -1 is no block, and a block behind pos has no key to see; what rows behind pos hold, NaN
 * included, does not reach the outputs; a row left without keys gives out 0 and lse -inf.  A block listed twice counts twice.  The order of a list decides only the order of
 * the sums.  An entry below -1 or at and past the stream's last block is recorded as TF_E_DEVICE, and so is
 * a table entry outside the pool that a listed block needs; the call's output is then undefined.  Entries of
 * pages that no list names are not used.
 * d_blk: int32 [S][R][max_blk]; everything else as in tf_paged_mla_attend, BF16 and FP8 pages alike.  The
 * blocks are dealt out by the default plan whatever the pool's flags: a row's bits may differ (within
 * rounding) between batches and are the same on every call of one batch.  The rows of an FP8 pool that many
 * query rows read are first expanded to BF16 pages in the workspace, whose size then includes them.
 * Errors: as for tf_paged_mla_attend, and TF_E_ARG for max_blk < 1 or a null d_blk. */
size_t tf_paged_mla_blocks_workspace_bytes(const tf_kvpool *pool, int32_t S, int32_t R, int32_t H, const int64_t *h_len,
                                           int32_t max_blk);   /* pool may be NULL: a BF16 pool */

int tf_paged_mla_attend_blocks(tf_kvpool *pool, int32_t cache, const int32_t *d_pt, int32_t max_pages,
                               const int64_t *h_len, const int32_t *d_blk, int32_t max_blk, int32_t S, int32_t R,
                               int32_t H, const void *d_q, float scale, void *d_out, float *d_lse, void *d_ws,
                               size_t ws_bytes, void *cuda_stream);

/* ---- attention of streams that share a prefix ----
 * What tf_paged_mla_attend computes, for a batch in which streams with the same first rows follow one
 * another: group g is the next h_gsize[g] streams (the sizes add up to S), whose rows 0 .. h_prefix[g] - 1
 * are the same.  The shared rows, in whole 64-row tiles, are read through the first stream's table, the rest
 * of each stream through its own.  Where R * H is not a multiple of 64 the columns (stream, row, head) of a
 * group are packed, and a shared tile is loaded and multiplied once for 64 of them, whatever stream they
 * belong to (16 heads: a quarter of the work).  Where it is, a stream's columns fill their products by
 * themselves: the work is tf_paged_mla_attend's, and the tiles that the streams share meet in L2.  That the
 * rows are the same is the caller's word: pages held by reference, or copies of the same bytes.  A group of
 * one stream, or a prefix of 0, shares nothing.  Table entries of pages of which a stream reads no row of its
 * own are not used, but for the group's first stream.
 * 0 <= h_prefix[g] <= h_len[s] - R + 1 for every stream s of the group: each query row sees all of it.
 * Both arrays have G entries, 1 <= G <= S.  All else as in tf_paged_mla_attend, BF16 and FP8 pages alike (a
 * NaN among a stream's last R rows reaches all R outputs: their columns share the products);
 * the keys are dealt out by a plan of their own whatever the pool's flags, so bits may differ (within
 * rounding) from tf_paged_mla_attend and between batches, and are the same on every call of one batch.
 * The workspace can be larger than that call's (and holds a BF16 copy of the rows of an FP8 pool that
 * many columns read).
 * Errors: as for tf_paged_mla_attend; TF_E_ARG for a null array, a size below 1 or sizes that do not add up;
 * TF_E_RANGE for a prefix outside its bounds; TF_E_UNSUPPORTED if R * H is not a multiple of 64 and S plus
 * the groups that share passes TF_MAX_STREAMS. */
size_t tf_paged_mla_shared_workspace_bytes(const tf_kvpool *pool, int32_t S, int32_t R, int32_t H, const int64_t *h_len,
                                           const int32_t *h_gsize, int32_t G, const int64_t *h_prefix);   /* pool may be NULL: a BF16 pool */

int tf_paged_mla_attend_shared(tf_kvpool *pool, int32_t cache, const int32_t *d_pt, int32_t max_pages,
                               const int64_t *h_len, const int32_t *h_gsize, int32_t G, const int64_t *h_prefix, int32_t S,
                               int32_t R, int32_t H, const void *d_q, float scale, void *d_out, float *d_lse, void *d_ws,
                               size_t ws_bytes, void *cuda_stream);

/* ---- the work plans of the two attention calls, for inspection ----
 * Host arithmetic only, nothing launched.  sms > 0: for a device of that many SMs (at most
 * TF_PLAN_MAX_RANGES) that runs sms / k clusters of k CTAs at a time; sms <= 0: the current device, as the
 * calls do (without one: TF_PLAN_MAX_RANGES SMs and no clusters).
 * A unit is a group of at most 64 columns over its key tiles: of blocks, unit (s * R + r) * ceil(H / 64) + g is
 * head group g of query row r of stream s, a tile a block; of shared prefixes they are numbered entry by
 * entry (the streams' own rows, then the groups' shared rows where R * H is not a multiple of 64), an entry
 * without tiles having none.
 *   info->ctas   CTAs; CTA i takes the unit tiles from range_bounds[i] up to range_bounds[i + 1], each a unit in
 *                the upper 32 bits and a tile of it in the lower ones
 *   info->merge  CTAs of a unit that a cluster merges (0: ranges; what they cut is merged by a second launch)
 *   info->cut    1 if some bound lies inside a unit
 *   info->units  units
 *   info->slots  64-column slots of fp32 partials that the workspace holds
 * range_bounds: int64 [TF_PLAN_MAX_RANGES + 1], or NULL.
 * Errors: TF_E_ARG for a null info, and what the calls' workspace sizes refuse. */
typedef struct {
    int32_t ctas, merge, cut, pad;
    int64_t units, slots;
} tf_unit_plan;

int tf_paged_mla_blocks_plan_info(int32_t S, int32_t R, int32_t H, const int64_t *h_len, int32_t max_blk, int32_t sms,
                                  tf_unit_plan *info, int64_t *range_bounds);

int tf_paged_mla_shared_plan_info(int32_t S, int32_t R, int32_t H, const int64_t *h_len, const int32_t *h_gsize, int32_t G,
                                  const int64_t *h_prefix, int32_t sms, tf_unit_plan *info, int64_t *range_bounds);

#ifdef __cplusplus
}
#endif

#endif /* TF_BLOCKS_H */
