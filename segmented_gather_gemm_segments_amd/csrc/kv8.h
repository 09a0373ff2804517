// Rows of an 8-bit KV cache: E4M3 codes and the exponent of a power of two (lora_kv8_view in lora_kv.h).
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;

// 8 codes of E4M3 times a power of two, exactly (gfx950 converts two at a time).
__device__ __forceinline__ bf16x8_t widen8(uint32_t lo, uint32_t hi, float scale) {
  auto two = [&](uint32_t w, auto high) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, decltype(high)::value));
  };
  const std::false_type l{};
  const std::true_type h{};
  return __builtin_bit_cast(bf16x8_t, make_uint4(two(lo, l), two(lo, h), two(hi, l), two(hi, h)));
}
__device__ __forceinline__ float exponent(uint32_t byte) { return __uint_as_float(byte << 23); }
// 0x80 in each byte of four codes that is E4M3's NaN.
__device__ __forceinline__ uint32_t nan8(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

constexpr int kLeastExp = -117;                // of a row: 2^-9, E4M3's least, is then 2^-126
constexpr float kLargest = 0x1.ep127f;         // 1.875 2^127: 240 2^120, the largest that a code stands for

// The exponent of a row whose largest finite magnitude is top: the least e with top <= 448 2^e = 1.75 2^(e + 8).
__device__ __forceinline__ int row_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  return max((int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u), kLeastExp);
}
// Codes of 8 elements (a pair of bf16 in each word) over 2^e, inv = 2^-e.  Products with a power of two are exact, so the
// conversion's rounding (to nearest even) is the only one.
__device__ __forceinline__ uint2 narrow8(uint4 u, float inv) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t out[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = __uint_as_float(e & 1 ? w[2 * i + e / 2] & 0xffff0000u : w[2 * i + e / 2] << 16);
      y[e] = std::isfinite(x) ? fminf(fmaxf(x, -kLargest), kLargest) * inv : NAN;
    }
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    out[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], c, true);
  }
  return make_uint2(out[0], out[1]);
}
// The largest finite magnitude of 8 bf16 elements.
__device__ __forceinline__ float top8(uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t m = (e ? w[i] >> 16 : w[i]) & 0x7fffu;  // magnitudes of bf16 order as their bits
      top = max(top, m < 0x7f80u ? m : 0u);
    }
  return __uint_as_float(top << 16);
}

}  // namespace
