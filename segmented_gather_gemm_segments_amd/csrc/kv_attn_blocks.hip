// Attention's kernels for listed pages of bf16 rows (kv_attn.h).
#include "kv_attn.h"

void lora::attn_items_blocks(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream) {
  launch_items<false, Mask::kBlocks>(a, plan, stream);
}
lora_status lora::kv_attn_blocks_debug(uint32_t *flags, int32_t clear) { return kv_debug_word(flags, clear); }
