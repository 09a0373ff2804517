// Attention's kernels for a causal mask over 8-bit rows (kv_attn.h).
#include "kv_attn.h"

void lora::attn8_items(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream) {
  launch_items<true, Mask::kCausal>(a, plan, stream);
}
lora_status lora::kv_attn8_debug(uint32_t *flags, int32_t clear) { return kv_debug_word(flags, clear); }
