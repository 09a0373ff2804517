/* Attention over a few pages of a long context, beside lora_kv_attn of lora_kv.h: every page keeps bounds of its
 * keys, a cheap score over the bounds lists the pages that matter to a token, and attention reads only those.
 * Three calls, each of them graph-capturable:
 *
 *   lora_kv_bounds_update  after an append: the bounds of the pages that grew
 *   lora_kv_block_select   each token's list of pages, for each KV head
 *   lora_kv_attn_blocks    attention over the listed pages
 *
 * Same status codes and conventions as lora_sgmv.h.                         */
#ifndef LORA_BLOCKS_H
#define LORA_BLOCKS_H

#include "lora_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bounds of the keys of each page and KV head, in whole numbers of steps 2^f.  With hi_d and lo_d the largest and least
 * finite value of dimension d over the page's positions (0 where there is none) and m the largest of their magnitudes,
 *     f = the least f with m <= 127 2^f, within -50 .. 50 (-50 for m = 0),
 *     H_d = hi_d / 2^f rounded up, L_d = lo_d / 2^f rounded down, both within -127 .. 127.
 * The row of page g and head h, at rows + g * page_stride + h * head_stride, holds H [head_dim] and L [head_dim]
 * in bytes, padding up to a multiple of 64 that is 0, then f in an int32 and 12 bytes that are not used. */
typedef struct {
  void *rows;           /* device, 16-byte aligned */
  int64_t page_stride, head_stride; /* bytes, multiples of 16, >= 0 */
} lora_kv_bounds;
/* Bytes of a row: 64 ceil(2 head_dim / 64) + 16.  Host only.  Errors: LORA_EUNSUPPORTED (head_dim), LORA_EINVAL. */
lora_status lora_kv_bounds_row_bytes(int32_t head_dim, int64_t *bytes);
/* The bounds that a lora_kv made with LORA_KV_BOUNDS keeps in its pages.  Errors: LORA_EINVAL (made without). */
lora_status lora_kv_get_bounds(const lora_kv *kv, lora_kv_bounds *bounds);

/* Writes the bounds of every page that holds one of the positions [begin[r], end[r]) of sequence seq[r], r < n,
 * from the page's positions below end[r].
 *   seq, begin, end  device int32 [n]; a negative seq is skipped (padding), one >= num_seqs too, as is a range
 *                    that is empty or not within the sequence's pages (debug build: LORA_DEBUG_BAD_TOKEN)
 *   max_tokens       host bound of end[r] - begin[r]; pages of a longer range past that many
 *                    positions are not written (LORA_DEBUG_BAD_TOKEN)
 * Absent pages are skipped (LORA_DEBUG_BAD_PAGE).  No two ranges may touch the same page.
 * The launch has as many workgroups for every range as max_tokens positions have pages: long ranges beside short ones are
 * better cut at page borders.
 * Errors: LORA_EINVAL, LORA_EUNSUPPORTED (view, 2^24 workgroups and more), LORA_EHIP.                          */
lora_status lora_kv_bounds_update(const lora_kv_view *kv, const lora_kv_bounds *bounds, const int32_t *seq,
                                  const int32_t *begin, const int32_t *end, int32_t n, int32_t max_tokens,
                                  hipStream_t stream);

#define LORA_BLOCKS_MAX_PAGES 32768  /* max_pages of the view, for lora_kv_block_select */
#define LORA_BLOCKS_MAX_COUNT 4096

/* Lists pages for token t at position p = token_pos[t] of sequence token_seq[t], n = p / page_tokens + 1 pages, and each KV
 * head: all n of them if n <= count; else the first `sink`, the last `recent` and, of the others,
 * those of the highest scores, ties to the lower page.  blocks[t][head] holds their numbers (0 .. n - 1)
 * in ascending order, then -1.
 *     score = max over the query heads g of the KV head of  2^(f + s_g) sum_d max(Q_gd H_d, Q_gd L_d),
 * Q_g the query row in whole numbers of steps 2^s_g: s_g from the row as f from a page's bounds, Q rounded to nearest even,
 * within -127 .. 127, elements that are not finite counting as 0.  The sum bounds <Q, K> of the rounded query; the
 * whole numbers stay below 2^24, so scores are exact in fp32 and lists are the same on every machine.  An absent page
 * scores -inf.  One step serves all dimensions of a page: where a few hold keys many times larger than the others', bounds of
 * the others are coarse and lists differ more from those of unrounded bounds (64 of 512 random pages of 64 keys of 128,
 * 8 query heads: 88 to 92 % the same pages; with two dimensions 10 times larger 30 to 64 %, 80 times 32 to 40 %, and up
 * to a seventh less of the softmax's weight on them).
 *   token_seq, token_pos  device int32 [num_tokens]; a token whose seq is negative (padding) or outside
 *                         [0, num_seqs), or whose position is not within the sequence's pages, lists -1 only (debug build:
 *                         LORA_DEBUG_BAD_TOKEN unless padding)
 *   q        as for lora_kv_attn, num_tokens rows of q_heads
 *   count, sink, recent  1 <= count <= LORA_BLOCKS_MAX_COUNT; sink, recent >= 0, recent >= 1, sink + recent <= count
 *   blocks   device int32 [num_tokens][kv_heads][count]
 *   workspace  optional device memory (NULL, 0: none), 16-byte aligned.  Where it holds what
 *              lora_kv_block_select_workspace says, few lists that may be long are scored by a launch of their own; lists
 *              are the same either way.  Contents on entry do not matter.  Calls that share it must not overlap, in graphs too.
 * Errors: LORA_EINVAL, LORA_EUNSUPPORTED (view, more than LORA_BLOCKS_MAX_PAGES pages in a sequence,
 * count, 2^24 tokens of all KV heads and more, 2^22 where sequences may have more than 2048 pages), LORA_EHIP. */
lora_status lora_kv_block_select(const lora_kv_view *kv, const lora_kv_bounds *bounds, const int32_t *token_seq,
                                 const int32_t *token_pos, int32_t num_tokens, const void *q, int64_t q_token_stride,
                                 int64_t q_head_stride, int32_t q_heads, int32_t count, int32_t sink, int32_t recent,
                                 int32_t *blocks, void *workspace, int64_t workspace_bytes, hipStream_t stream);
/* Workspace bytes for num_tokens tokens (0: it would not be used).  Host only.  Errors: LORA_EINVAL, LORA_EUNSUPPORTED (the view
 * and the number of tokens that lora_kv_block_select refuses).                                              */
lora_status lora_kv_block_select_workspace(const lora_kv_view *kv, int32_t num_tokens, int64_t *bytes);

/* lora_kv_attn over listed pages: token t and KV head h keep the positions j <= token_pos[t] on the pages
 * blocks[t][h][0 .. count) of its sequence.  Any lists are taken, in any order (a page that is listed twice counts
 * twice); an entry outside [0, max_pages) names nothing.  A token that keeps nothing gets out = 0, lse = -inf.
 *   plan  of lora_kv_attn_plan with flags LORA_ATTN_BLOCKS (no causal flag, no window): one
 *         request of one token for each token, its sequence, and as kv_len the positions of its list's
 *         pages, min(count, its pages) * page_tokens at least (count * page_tokens serves every step)
 * Everything else, errors included, as lora_kv_attn; a count below 1 or above LORA_BLOCKS_MAX_COUNT: LORA_EUNSUPPORTED. */
lora_status lora_kv_attn_blocks(const lora_kv_view *kv, const lora_attn_plan *plan, const lora_attn_item *items,
                                const int32_t *blocks, int32_t count, const int32_t *token_pos, const void *q,
                                int64_t q_token_stride, int64_t q_head_stride, void *out, int64_t out_token_stride,
                                int64_t out_head_stride, float *lse, float scale, void *workspace,
                                int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_BLOCKS_H */
