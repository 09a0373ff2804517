// Where rows of a paged KV cache stand.  After kv_debug.h.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "kv_debug.h"
#include "lora_kv.h"

namespace {

// The place of a listed token's row in the cache: its page and slot, or page -1 where the token is skipped.
struct Place {
  int page, slot;
};
__device__ __forceinline__ Place place_of(const lora_kv_view &kv, int s, int p) {
  const bool in = s < kv.num_seqs && p >= 0 && p < kv.max_pages * kv.page_tokens;
  KV_CHECK(in || s < 0, LORA_DEBUG_BAD_TOKEN);
  if (s < 0 || !in) return {-1, 0};
  const int page = kv.page_table[(int64_t)s * kv.max_pages + p / kv.page_tokens];
  KV_CHECK((unsigned)page < (unsigned)kv.num_pages, LORA_DEBUG_BAD_PAGE);
  return {(unsigned)page < (unsigned)kv.num_pages ? page : -1, p % kv.page_tokens};
}
__device__ __forceinline__ int64_t row_at(const lora_kv_view &kv, Place x, int h) {
  return x.page * kv.page_stride + h * kv.head_stride + x.slot * kv.token_stride;
}
__device__ __forceinline__ int64_t scale_at(const lora_kv8_view &v, Place x, int h) {
  return x.page * v.scale_page_stride + h * v.scale_head_stride + x.slot * v.scale_token_stride;
}

// The view with what 8-bit rows add to it (nothing for bf16 rows): what kernels for either kind of row take.
inline lora_kv8_view view8(const lora_kv_view *kv) {
  lora_kv8_view v{};
  if (kv->dtype == LORA_FP8_E4M3) v = *reinterpret_cast<const lora_kv8_view *>(kv);
  else v.kv = *kv;
  return v;
}

}  // namespace
