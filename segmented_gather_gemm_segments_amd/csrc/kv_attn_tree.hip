// Attention's kernels for a tree's mask over bf16 rows (kv_attn.h).
#include "kv_attn.h"

void lora::attn_items_tree(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream) {
  launch_items<false, Mask::kTree>(a, plan, stream);
}
lora_status lora::kv_attn_tree_debug(uint32_t *flags, int32_t clear) { return kv_debug_word(flags, clear); }
