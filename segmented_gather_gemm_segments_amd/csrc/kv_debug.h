// The debug build's error word of one source file (see LORA_DEBUG in
// lora_sgmv.h): its kernels record the bad device-side values that every build skips.
// Include once per .hip file of the KV cache, inside no namespace.
#pragma once

#include <hip/hip_runtime.h>

#ifndef LORA_DEBUG
#define LORA_DEBUG 0
#endif

namespace {
#if LORA_DEBUG
__device__ uint32_t g_kv_debug_word;
#define KV_CHECK(cond, bit)                                                                                   \
  do {                                                                                                        \
    if (!(cond)) __hip_atomic_fetch_or(&g_kv_debug_word, bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);      \
  } while (0)
#else
#define KV_CHECK(cond, bit) \
  do {                      \
  } while (0)
#endif

// Adds the word's bits to *flags and, with clear, resets it.
inline lora_status kv_debug_word(uint32_t *flags, int32_t clear) {
#if LORA_DEBUG
  uint32_t word = 0;
  hipError_t e = hipMemcpyFromSymbol(&word, HIP_SYMBOL(g_kv_debug_word), sizeof word, 0, hipMemcpyDeviceToHost);
  if (e != hipSuccess) return lora::hip_fail(e, "reading the debug word");
  *flags |= word;
  if (clear) {
    const uint32_t zero = 0;
    e = hipMemcpyToSymbol(HIP_SYMBOL(g_kv_debug_word), &zero, sizeof zero, 0, hipMemcpyHostToDevice);
    if (e != hipSuccess) return lora::hip_fail(e, "clearing the debug word");
  }
#endif
  return LORA_OK;
}
}  // namespace
