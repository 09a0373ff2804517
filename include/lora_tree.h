/* Trees of drafted tokens over a paged KV cache, beside lora_kv_attn of lora_kv.h: a server that drafts
 * several continuations of a sequence checks all of them in one step, and goes on with the path that the model accepts.
 *
 * A request's new tokens are the nodes of a tree (or of several, hanging below the context): node i of request r is
 * token q_starts[r] + i of q, its K and V rows stand at position kv_len[r] - q_len[r] + i of the sequence
 * (append first), and parent[q_starts[r] + i] < i is its parent's number, or -1 for the context.
 * Same status codes and conventions as lora_sgmv.h.                         */
#ifndef LORA_TREE_H
#define LORA_TREE_H

#include "lora_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_TREE_MAX_NODES 4096  /* of one request */

/* What a tree's attention reads: for each token of the batch, which nodes of its request it keeps (bit a % 64 of word
 * a / 64 for node a) and how many ancestors it has. */
typedef struct {
  uint64_t *mask;  /* device [num_tokens][words] */
  int32_t *depth;  /* device [num_tokens] */
  int32_t words;   /* 1 .. LORA_TREE_MAX_NODES / 64 */
  int32_t num_tokens;
} lora_tree;

/* Fills mask and depth: a node keeps itself and its ancestors, with window > 0 those fewer than `window` above it.
 *   q_starts  device int32 [num_reqs + 1], those of the attention's plan
 *   parent    device int32 [tree->num_tokens]
 * A parent outside [-1, i) counts as -1 (debug build: LORA_DEBUG_BAD_TOKEN).  A request with more than
 * 64 words nodes, or whose tokens are not within [0, num_tokens), is skipped (LORA_DEBUG_BAD_TOKEN): its rows stay as
 * they are.  Errors: LORA_EINVAL, LORA_EUNSUPPORTED (words, 2^24 requests and more), LORA_EHIP. */
lora_status lora_tree_mask(const int32_t *q_starts, int32_t num_reqs, const int32_t *parent, int32_t window,
                           const lora_tree *tree, hipStream_t stream);

/* lora_kv_attn for trees.  With base = kv_len - q_len, node i keeps
 *     the context:  0 <= j < base, and j > base + depth[i] - window if window > 0 (depth[i] taken within [0, i]),
 *     drafted ones: j = base + a for each a with its bit set (and a <= i if the plan is causal),
 * so that a window counts positions along the path.  The mask need not come from lora_tree_mask: any bits are taken
 * as they are, those of nodes that the request does not have are ignored, nodes past 64 words are kept by none, and a
 * node that keeps nothing gets out = 0 and lse = -inf.
 *   plan  of lora_kv_attn_plan with LORA_ATTN_TREE in its flags (and LORA_ATTN_CAUSAL, which spares
 *         the positions behind a node: parents come first)
 * Everything else, errors included, as lora_kv_attn; a tree of fewer tokens than the plan's: LORA_EINVAL.   */
lora_status lora_kv_attn_tree(const lora_kv_view *kv, const lora_attn_plan *plan, const lora_attn_item *items,
                              const lora_tree *tree, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                              void *out, int64_t out_token_stride, int64_t out_head_stride, float *lse, float scale,
                              void *workspace, int64_t workspace_bytes, hipStream_t stream);

/* Moves the rows of an accepted path to where the sequence goes on: for r < num_reqs and i = 0, 1, ..., the K and V rows
 * (and scale bytes) of position base[r] + path[r][i] of sequence seq[r] are copied to position base[r] + i, in
 * effect one after the other.  The sequence is then base[r] + (length of the path) positions long (lora_kv_truncate).
 *   seq, base  device int32 [num_reqs]
 *   path       device int32 [num_reqs][max_path]: nodes in ascending order (parents come first); a negative entry ends
 *              the path, and so does one that is not above the entry before it (debug build: LORA_DEBUG_BAD_TOKEN)
 * A request whose seq is negative is skipped (padding), one >= num_seqs or with a negative base too
 * (LORA_DEBUG_BAD_TOKEN); a position outside the sequence's pages (LORA_DEBUG_BAD_TOKEN) or on an absent page
 * (LORA_DEBUG_BAD_PAGE) skips its copy.  No two requests may write the same page, nor one read what another
 * writes.  Errors: LORA_EINVAL, LORA_EUNSUPPORTED (view, 2^24 workgroups and more, rows of a position in 2^31 pieces of 16
 * bytes and more), LORA_EHIP.     */
lora_status lora_kv_keep_path(const lora_kv_view *kv, const int32_t *seq, const int32_t *base, const int32_t *path,
                              int32_t num_reqs, int32_t max_path, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_TREE_H */
