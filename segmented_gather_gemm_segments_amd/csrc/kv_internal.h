// Declarations shared by the files of the paged KV cache (kv_host.cpp,
// kv_pages.hip, kv_tree.hip, kv_blocks.hip, kv_attn*.hip).  Not part of the public ABI.
#pragma once

#include <memory>
#include <utility>
#include <vector>

#include "lora_internal.h"
#include "lora_blocks.h"
#include "lora_kv.h"
#include "lora_tree.h"

namespace lora {

// Whether a launch of this many workgroups goes past the 2^32 - 1 threads that one may have.
inline bool too_many(int64_t workgroups, int64_t threads) { return workgroups > (int64_t)UINT32_MAX / threads; }

// A page that one launch can copy.
constexpr int64_t kKvMaxPageBytes = (int64_t)1 << 35;

// Checks a descriptor's geometry and pointers (LORA_OK, or an error with its message).
lora_status check_view(const lora_kv_view *kv);

// Device steps of the sequence bookkeeping (kv_pages.hip).  Lists travel as kernel
// arguments, so no staging buffer can change under a pending launch.
lora_status kv_move_pages(void *storage, int64_t page_bytes, const std::vector<std::pair<int32_t, int32_t>> &moves,
                          hipStream_t stream);  // (from, to)
lora_status kv_write_table(int32_t *table, const std::vector<std::pair<int64_t, int32_t>> &entries,
                           hipStream_t stream);  // (index, page)
lora_status kv_clear_table(int32_t *table, int64_t count);  // -1 everywhere, done on return
// A mark on the stream: done once the work queued so far is.
lora_status kv_mark(hipStream_t stream, std::shared_ptr<void> *mark);
bool kv_mark_done(const std::shared_ptr<void> &mark, bool wait);
lora_status kv_not_capturing(hipStream_t stream);

// Checks a tree's sizes and pointers.
lora_status check_tree(const lora_tree *tree);

// The debug words of the other files (lora_kv_debug_flags adds that of kv_pages.hip; 0 in release builds).
lora_status kv_attn_debug(uint32_t *flags, int32_t clear);
lora_status kv_attn_tree_debug(uint32_t *flags, int32_t clear);
lora_status kv_attn_blocks_debug(uint32_t *flags, int32_t clear);
lora_status kv_attn8_debug(uint32_t *flags, int32_t clear);
lora_status kv_attn8_tree_debug(uint32_t *flags, int32_t clear);
lora_status kv_attn8_blocks_debug(uint32_t *flags, int32_t clear);
lora_status kv_tree_debug(uint32_t *flags, int32_t clear);
lora_status kv_blocks_debug(uint32_t *flags, int32_t clear);

}  // namespace lora
