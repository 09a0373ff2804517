/* The KV half of the unified page pool: keys and values of sequences in pages of
 * the pool that also holds adapter rows ("Multi-LoRA serving: the single
 * translator with a thousand glossaries" TL;DR and section "Operational
 * pitfalls": adapter weights live in the same memory pool as the KV cache, both
 * pageable; the glossary entry "Multi-LoRA Serving", skillsintelligence.tools,
 * intro paragraph).  Four parts, from the device up:
 *
 *   pages      lora_pages_copy, lora_page_table_remap: pages moved in one launch
 *   append     lora_kv_append: new tokens' K and V rows written through the page table, in 8 bits where
 *              the cache holds those; lora_kv_read: rows read back
 *   attention  lora_kv_attn_plan, lora_kv_attn: new tokens (a prompt's chunk, or single decode
 *              tokens) attend to everything cached of their sequence
 *   sequences  lora_kv_*: host bookkeeping of which pages a sequence holds -- extend, fork
 *              (shared pages, copied when written), truncate, free, compact
 *
 * Same status codes and conventions as lora_sgmv.h.                         */
#ifndef LORA_KV_H
#define LORA_KV_H

#include "lora_sgmv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* A paged KV cache as the kernels read it.  Position p of sequence s and KV head h
 * is the row of head_dim elements at
 *     k + page * page_stride + h * head_stride + (p % page_tokens) * token_stride,
 *     page = page_table[s * max_pages + p / page_tokens],
 * and likewise in v.  A page id outside [0, num_pages) makes the positions it
 * would hold absent: attention does not see them and append does not write
 * them (the debug build records LORA_DEBUG_BAD_PAGE).  Any order of page,
 * head and token is described by the strides; rows must not overlap.        */
typedef struct {
  int32_t dtype;        /* LORA_BF16, or LORA_FP8_E4M3 (lora_kv8_view below) */
  int32_t head_dim;     /* a multiple of 8, 8..256 */
  int32_t kv_heads;     /* >= 1 */
  int32_t page_tokens;  /* positions per page, >= 1 */
  int32_t num_pages;    /* pages behind k and v (bounds for page ids) */
  int32_t num_seqs;     /* rows of page_table */
  int32_t max_pages;    /* row length of page_table */
  int32_t reserved;     /* 0 */
  void *k, *v;          /* device, 16-byte aligned: position 0, head 0 of page 0 (NULL without pages) */
  int64_t page_stride, head_stride, token_stride; /* elements, multiples of 8, >= 0 */
  const int32_t *page_table; /* device [num_seqs][max_pages] (NULL only where that is empty) */
} lora_kv_view;

/* A cache of 8-bit rows: half the bytes of a cache for twice the positions ("Multi-LoRA Inference Serving", the paragraphs
 * on quantization, for the adapters' rows).  Every call that takes a lora_kv_view takes the
 * first member of this one too: dtype LORA_FP8_E4M3 says that the rest follows it.
 * A row x of head_dim elements, of one position, head and of K or V, is stored as codes c and an exponent e:
 *     e = max(-117, the least e with max |x_i| <= 448 2^e),   c_i = x_i 2^-e rounded to nearest even in E4M3,
 * and stands for c_i 2^e.  The maximum is over finite elements (e = -117 where it is 0); one that is not
 * finite is stored as E4M3's NaN; magnitudes above 1.875 2^127 count as that, since 2^128 would not be finite.  A power
 * of two costs no precision over any other factor but where codes are subnormal (below 2^-13
 * of the row's largest), makes both directions exact, and every c 2^e a normal bf16 number or 0.
 * In the view: head_dim a multiple of 16; k and v hold bytes, their strides (in elements, which are
 * bytes) multiples of 16.  e + 127 of position p, head h is the byte at
 *     k_scales + page * scale_page_stride + h * scale_head_stride + (p % page_tokens) * scale_token_stride
 * and likewise in v_scales.                                                 */
#define LORA_FP8_E4M3 2
typedef struct {
  lora_kv_view kv;      /* dtype LORA_FP8_E4M3 */
  uint8_t *k_scales, *v_scales; /* device (NULL without pages) */
  int64_t scale_page_stride, scale_head_stride, scale_token_stride; /* bytes, >= 0 */
} lora_kv8_view;

/* ------------------------------------------------------------------------ */
/* Copies page src[i] to page dst[i] of one storage, i < n, in one launch: the move
 * list of a compaction, the copy of a forked sequence's last page.
 *   storage    device, num_pages pages of page_bytes bytes (a positive multiple of 16)
 *   src, dst   device int32 [n]; a pair with an id outside [0, num_pages) is
 *              skipped (debug build: LORA_DEBUG_BAD_PAGE).  No page may be written
 *              twice or both read and written, except src[i] == dst[i], which changes nothing.
 * Errors: LORA_EINVAL, LORA_EUNSUPPORTED (64 GiB and more to copy), LORA_EHIP. */
lora_status lora_pages_copy(void *storage, int64_t page_bytes, int32_t num_pages, const int32_t *src,
                            const int32_t *dst, int32_t n, hipStream_t stream);
/* table_out[i] = remap[table_in[i]] for entries in [0, num_pages); other entries
 * (such as -1) are copied as they are.  remap device int32 [num_pages]; table_in and
 * table_out device int32 [count], the same array or not overlapping.
 * Errors: LORA_EINVAL, LORA_EUNSUPPORTED (2^32 entries and more), LORA_EHIP. */
lora_status lora_page_table_remap(const int32_t *remap, int32_t num_pages, const int32_t *table_in,
                                  int32_t *table_out, int64_t count, hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Writes the K and V rows of num_tokens new tokens.
 *   k_new, v_new  device; token t, head h at t * new_token_stride + h * new_head_stride
 *                 elements (multiples of 8, >= 0), head_dim contiguous elements
 *   token_seq     device int32 [num_tokens]: row of the page table; a negative
 *                 one (padding) is skipped, one >= num_seqs too (debug build:
 *                 LORA_DEBUG_BAD_TOKEN)
 *   token_pos     device int32 [num_tokens]: position in the sequence; outside
 *                 [0, max_pages * page_tokens) it is skipped (LORA_DEBUG_BAD_TOKEN)
 * No two tokens may name the same place (a page held by two sequences is
 * written by neither: extend copies it first).  Errors: LORA_EINVAL,
 * LORA_EUNSUPPORTED (view; 64 GiB and more of new K rows), LORA_EHIP.       */
lora_status lora_kv_append(const lora_kv_view *kv, const void *k_new, const void *v_new, int64_t new_token_stride,
                           int64_t new_head_stride, const int32_t *token_seq, const int32_t *token_pos,
                           int32_t num_tokens, hipStream_t stream);
/* The other way: rows of listed positions copied out of the cache in bf16 (those of an 8-bit cache are exact),
 * to hand a sequence over or to keep it elsewhere.  Arguments as for lora_kv_append, k_out and v_out
 * written where it reads k_new and v_new (their rows must not overlap); a position may be listed twice.
 * Where append would skip a token, and on an absent page, the rows of k_out and v_out are left as they are. */
lora_status lora_kv_read(const lora_kv_view *kv, void *k_out, void *v_out, int64_t out_token_stride,
                         int64_t out_head_stride, const int32_t *token_seq, const int32_t *token_pos, int32_t num_tokens,
                         hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Attention of new tokens over the cache.  Request r of a batch has q_len[r] new
 * tokens, the last ones of its sequence's kv_len[r] positions (their K and V
 * rows are in the cache: append first); new token i stands at position
 * p = kv_len[r] - q_len[r] + i.  Query head h reads KV head h / (q_heads / kv_heads).
 * Token i keeps the positions j with
 *     0 <= j < kv_len[r],   j <= p if causal,   j > p - window if window > 0,
 * on pages that exist, and
 *     s_j = scale <q, K_j>,  lse = ln sum_j exp(s_j),  out = sum_j exp(s_j - lse) V_j.
 * A token that keeps nothing (kv_len 0, or a chunk longer than its sequence)
 * gets out = 0 and lse = -inf.  What stands in positions that a token does
 * not keep never reaches it, NaN and infinities included.
 *
 * Plan (host).  Rows of a request are its (token, query head of one KV head) pairs, row
 * i * group + g with group = q_heads / kv_heads, so that the query heads that share a KV
 * head share its rows of K and V.  An item is up to LORA_ATTN_ROWS (few rows: decode) or
 * LORA_ATTN_TILE_ROWS rows of one request over one range of positions; every
 * KV head runs every item.  Where the items are too few to fill the device the
 * positions are cut into ranges whose partial results (fp32) go to a workspace, and
 * a second launch joins them in order.  A plan serves every layer of a step; it is
 * uploaded once and launched many times.  Items heaviest first.             */
typedef struct {
  int32_t q_begin;   /* the request's first token in q and out */
  int32_t row0;      /* first row (token * group + head in group) of the request */
  int32_t rows;      /* 1.. LORA_ATTN_ROWS or LORA_ATTN_TILE_ROWS */
  int32_t seq;       /* row of the page table */
  int32_t pos0;      /* position of the request's token 0 (negative: rows that keep nothing) */
  int32_t kv_begin;  /* positions [kv_begin, kv_end) */
  int32_t kv_end;
  int32_t part;      /* -1: the item's results are final; else its first row of partial
                        results.  Join items: the number of parts, each `rows` rows of
                        partial results, the first at row kv_begin; kv_end as in the last part */
} lora_attn_item;

#define LORA_ATTN_ROWS 16
#define LORA_ATTN_TILE_ROWS 128
#define LORA_ATTN_MAX_PARTS 64
#define LORA_ATTN_CAUSAL 1
#define LORA_ATTN_TREE 8     /* the plan is for lora_kv_attn_tree (lora_tree.h) */
#define LORA_ATTN_BLOCKS 16  /* the plan is for lora_kv_attn_blocks (lora_blocks.h) */

typedef struct {
  int32_t q_heads, kv_heads, head_dim;
  int32_t flags;        /* of LORA_ATTN_*; lora_kv_attn takes LORA_ATTN_CAUSAL or 0 */
  int32_t window;       /* 0: none */
  int32_t num_tokens;   /* new tokens of the batch (the last of q_starts) */
  int32_t num_row_items, num_tile_items, num_joins; /* items: row items, tile items, joins, in this order */
  int32_t num_part_rows; /* rows of partial results (of one KV head) */
  int64_t workspace_bytes;
} lora_attn_plan;

/* q_starts [num_reqs + 1] (from 0, not decreasing), seq and kv_len [num_reqs]: host
 * arrays; several requests may name the same sequence.
 *   max_parts  ranges a request's positions may be cut into (1: never cut,
 *              0: the library's choice, at most LORA_ATTN_MAX_PARTS)
 *   items, capacity  host array, or NULL to learn the counts (plan is filled
 *              in either way)
 * Errors: LORA_EINVAL (sizes, q_starts, heads not a multiple, window < 0,
 * max_parts), LORA_ERANGE (a sequence outside [0, num_seqs), a kv_len above
 * max_kv), LORA_EUNSUPPORTED (head_dim), LORA_ENOMEM (capacity; plan still
 * filled in).
 *   num_seqs, max_kv  the view's num_seqs and max_pages * page_tokens (bounds) */
lora_status lora_kv_attn_plan(const int32_t *q_starts, const int32_t *seq, const int32_t *kv_len, int32_t num_reqs,
                              int32_t num_seqs, int64_t max_kv, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                              int32_t flags, int32_t window, int32_t max_parts, lora_attn_plan *plan,
                              lora_attn_item *items, int32_t capacity);

/* Runs a plan.
 *   items      device, the plan's items
 *   q, out     device bf16 [num_tokens][q_heads] rows of head_dim elements; token and head
 *              strides in elements, multiples of 8, >= 0 (out: rows must not overlap)
 *   lse        device fp32 [num_tokens][q_heads], or NULL
 *   scale      factor of the products, finite (the usual one is head_dim^-1/2); a row whose scores pass
 *              2^127 in magnitude has unspecified results
 *   V          rows whose largest magnitude is 0 or within 2^-92 .. 2^100, for up to 2^19 positions: weights run up to 2^8 on the
 *              way, so that sums of larger rows may pass 2^128, and a weight of an 8-bit row, which is rounded with the row's
 *              factor, loses bits below 2^-126
 *   workspace  device, 16-byte aligned, at least plan->workspace_bytes (NULL with 0);
 *              contents on entry do not matter.  Calls that share it must not
 *              overlap, in graphs too.
 * Products of bf16 in fp32 (an 8-bit cache's rows enter them exactly); maximum and sum of the softmax in fp32; its weights
 * are rounded to bf16 for their product with V (out is bf16), the sum is not;
 * out rounded once.  Bit-identical from run to run.  Device-side items are
 * checked against the plan and the view: a bad one is skipped (debug build:
 * LORA_DEBUG_BAD_ITEM), and the join of ranges that reach past the view with them, so
 * that a plan made for a larger view leaves those rows of out and lse as they are.
 * Rows of out and lse beyond num_tokens are left as they are.
 * Errors: LORA_EINVAL, LORA_EUNSUPPORTED (dtype, head_dim, strides of 2^35 elements, of scales 2^32,
 * 2^24 items of all KV heads and more), LORA_EHIP.                          */
lora_status lora_kv_attn(const lora_kv_view *kv, const lora_attn_plan *plan, const lora_attn_item *items, const void *q,
                         int64_t q_token_stride, int64_t q_head_stride, void *out, int64_t out_token_stride,
                         int64_t out_head_stride, float *lse, float scale, void *workspace, int64_t workspace_bytes,
                         hipStream_t stream);

/* ------------------------------------------------------------------------ */
/* Sequences over a pool's pages (host bookkeeping).  The pool's pages of page_rows x
 * row_width elements hold page_tokens = page_rows * row_width / (2 kv_heads head_dim)
 * positions each: first K [kv_heads][page_tokens][head_dim], then V (the flags below change both).  The pool may hold adapters
 * too (lora_cache): each page belongs to whoever took it.  A page that an eviction of a lora_cache
 * gave back may still be read on that cache's compute stream, and extend and compact take it
 * without asking: a pool's lora_cache and lora_kv use one stream, the cache's compute stream.
 * Pages freed by hand (lora_pool_free) are those that no queued work reads any more.
 *
 * A lora_kv owns the contents of the caller's device page table [max_seqs][max_pages] (-1
 * where there is no page).  Every device step goes on the `stream` of the call; use one
 * stream per lora_kv, the one its kernels run on, and not while it is being captured into
 * a graph (LORA_EINVAL).  A page that a call drops may still be read by work queued on
 * that stream, so it is kept as a spare: the same lora_kv takes it again at once (the
 * stream orders the two uses), and lora_kv_trim gives spares back to the
 * pool once that work is done.  A lora_kv and its pool are not thread-safe.
 *
 *   create    fills the page table with -1, done on return, ordered behind no stream: nothing queued
 *             may still use that memory, and no stream of the device may be in capture.
 *             LORA_KV_HOST_ONLY: bookkeeping only, no device work (tests).  Errors: LORA_EINVAL,
 *             LORA_EUNSUPPORTED (a pool that is not plain bf16, head_dim, a page that
 *             holds no position, whose V is not 16-byte aligned or that exceeds 32 GiB)
 *   extend    sequence seqs[i] grows by new_tokens[i] >= 0 positions (a sequence not in use
 *             starts at 0): pages are taken, and a shared page that the growth
 *             writes into is replaced by a copy.  All or nothing.  Errors: LORA_ERANGE (a sequence id),
 *             LORA_EINVAL (an id twice, a negative count, more than max_pages pages), LORA_ENOMEM
 *   fork      dst[i] (not in use) becomes a copy of src that shares all its pages.  A src of
 *             length 0 gives sequences of length 0.
 *   truncate  drops the positions at and behind new_len (0 <= new_len <= length)
 *   free      drops sequences entirely; an id that is not in use is an error (LORA_EINVAL)
 *   compact   moves pages that sequences hold to lower ids that are free in the pool or spare, highest
 *             page to lowest id, until none is lower; copies their contents and rewrites the
 *             page table; *moved = pages copied.  The pages left are spares
 *   trim      gives back spares whose work is done; wait != 0 waits for all of it.  *left =
 *             spares still held
 * On an error nothing is changed, except that LORA_EHIP leaves the device
 * contents unspecified.                                                     */
#define LORA_KV_HOST_ONLY 1
#define LORA_KV_FP8 4     /* flag: 8-bit rows.  A page holds K codes [kv_heads][page_tokens][head_dim], V codes, then the
                             scale bytes of K [kv_heads][page_tokens] and of V; head_dim a multiple of 16 */
#define LORA_KV_BOUNDS 8  /* flag: each page ends in the bounds of its keys (lora_blocks.h), which copies and moves of
                             the page take along */
typedef struct lora_kv lora_kv;
typedef struct {
  int32_t seqs;        /* sequences in use */
  int32_t pages;       /* pages held by sequences, shared ones counted once */
  int32_t shared;      /* of those, held by two or more */
  int32_t spare;       /* dropped, not given back yet */
  int32_t highest;     /* highest page id held or spare, -1 for none */
  int32_t page_tokens;
} lora_kv_stats;
lora_status lora_kv_create(lora_pool *pool, int32_t kv_heads, int32_t head_dim, int32_t max_seqs, int32_t max_pages,
                           int32_t *device_page_table, int32_t flags, lora_kv **out);
lora_status lora_kv_extend(lora_kv *kv, const int32_t *seqs, const int32_t *new_tokens, int32_t n, hipStream_t stream);
lora_status lora_kv_fork(lora_kv *kv, int32_t src, const int32_t *dst, int32_t n, hipStream_t stream);
lora_status lora_kv_truncate(lora_kv *kv, int32_t seq, int32_t new_len, hipStream_t stream);
lora_status lora_kv_free(lora_kv *kv, const int32_t *seqs, int32_t n, hipStream_t stream);
lora_status lora_kv_compact(lora_kv *kv, int32_t *moved, hipStream_t stream);
lora_status lora_kv_trim(lora_kv *kv, int32_t wait, int32_t *left);
/* *length = -1 for a sequence not in use; page_ids: capacity max_pages, or NULL. */
lora_status lora_kv_seq(const lora_kv *kv, int32_t seq, int32_t *length, int32_t *page_ids, int32_t *num_pages);
lora_status lora_kv_get_stats(const lora_kv *kv, lora_kv_stats *stats);
/* The descriptor that append and attention take (a cache made with LORA_KV_FP8: lora_kv_get_view8, else LORA_EINVAL). */
lora_status lora_kv_get_view(const lora_kv *kv, lora_kv_view *view);
lora_status lora_kv_get_view8(const lora_kv *kv, lora_kv8_view *view);
/* Waits for the work that its stream (that of its last call, which must still
 * exist) holds by now, gives every page back to the pool (which must still exist too) and
 * frees the object.  Pages whose work cannot be waited for (the stream is in capture, an
 * error) stay taken for good.  The pool's device is current, as for every call here. */
void lora_kv_destroy(lora_kv *kv);

/* ------------------------------------------------------------------------ */
/* lora_debug_flags of lora_sgmv.h for the kernels declared here, which keep words of their
 * own: LORA_DEBUG_BAD_PAGE, _BAD_TOKEN and _BAD_ITEM as named above. */
lora_status lora_kv_debug_flags(uint32_t *flags, int32_t clear);

#ifdef __cplusplus
}
#endif

#endif /* LORA_KV_H */
