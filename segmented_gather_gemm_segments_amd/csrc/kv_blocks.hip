// Pages selected by bounds of their keys (lora_blocks.h): the bounds and the selection.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kv_internal.h"
#include "kv8.h"
#include "kv_debug.h"
#include "kv_rows.h"

using namespace lora;

namespace {

typedef __attribute__((ext_vector_type(4))) int i32x4_t;

// The exponent of whole-number steps: the least f with m <= 127 2^f = (127 / 64) 2^(f + 6), within its limits.
__device__ __forceinline__ int step_exponent(float m) {
  const uint32_t u = __float_as_uint(m);
  return min(max((int)(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > 0x7e0000u), -50), 50);
}
__device__ __forceinline__ float bf16_at(uint4 u, int e) {  // e a constant
  const uint32_t w = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
  return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ uint32_t byte4(const int *c) {
  return (uint32_t)(c[0] & 255) | (uint32_t)(c[1] & 255) << 8 | (uint32_t)(c[2] & 255) << 16 | (uint32_t)c[3] << 24;
}

// ----------------------------------------------------------------- bounds
// A workgroup per page of a range and KV head: threads take 8 dimensions of every R-th key, then thread d joins dimension d's R
// values through LDS.  Reads the page's keys once.
constexpr int kThreads = 256;

template <bool F8>
__global__ __launch_bounds__(kThreads) void bounds_kernel(lora_kv8_view v, lora_kv_bounds bounds,
                                                          const int32_t *__restrict__ seq, const int32_t *__restrict__ begins,
                                                          const int32_t *__restrict__ ends, int max_tokens, int pages) {
  __shared__ __attribute__((aligned(16))) float top[2][kThreads * 8];
  __shared__ float wave_top[kThreads / 64];
  __shared__ __attribute__((aligned(16))) int8_t codes[512];
  const lora_kv_view &kv = v.kv;
  const int h = blockIdx.x % kv.kv_heads, j = blockIdx.x / kv.kv_heads % pages, r = blockIdx.x / kv.kv_heads / pages;
  const int s = seq[r], begin = begins[r], end = ends[r];
  const bool good = s < kv.num_seqs && begin >= 0 && end > begin && end <= kv.max_pages * kv.page_tokens;
  KV_CHECK(s < 0 || (good && (int64_t)end - begin <= max_tokens) || threadIdx.x != 0, LORA_DEBUG_BAD_TOKEN);
  if (s < 0 || !good) return;
  const int64_t at = begin / kv.page_tokens + (int64_t)j;  // the page's number in the sequence
  if (at * kv.page_tokens >= min((int64_t)end, (int64_t)begin + max_tokens)) return;
  const int page = kv.page_table[(int64_t)s * kv.max_pages + at];
  KV_CHECK((unsigned)page < (unsigned)kv.num_pages || threadIdx.x != 0, LORA_DEBUG_BAD_PAGE);
  if ((unsigned)page >= (unsigned)kv.num_pages) return;
  const int D = kv.head_dim, chunks = D >> 3, R = kThreads / chunks;
  const int filled = (int)min((int64_t)kv.page_tokens, end - at * kv.page_tokens);
  const int c = (int)threadIdx.x % chunks, r0 = (int)threadIdx.x / chunks;
  float hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) hi[e] = -INFINITY, lo[e] = INFINITY;
  if (r0 < R) {
#pragma unroll 4
    for (int slot = r0; slot < filled; slot += R) {
      const Place place = {page, slot};
      uint4 u;
      if constexpr (F8) {
        const uint2 k = *reinterpret_cast<const uint2 *>((const uint8_t *)kv.k + row_at(kv, place, h) + c * 8);
        u = __builtin_bit_cast(uint4, widen8(k.x, k.y, exponent(v.k_scales[scale_at(v, place, h)])));
      } else {
        u = *reinterpret_cast<const uint4 *>((const uint16_t *)kv.k + row_at(kv, place, h) + c * 8);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = bf16_at(u, e);
        const bool ok = std::isfinite(x);
        hi[e] = ok ? fmaxf(hi[e], x) : hi[e];
        lo[e] = ok ? fminf(lo[e], x) : lo[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      top[0][threadIdx.x * 8 + e] = hi[e];
      top[1][threadIdx.x * 8 + e] = lo[e];
    }
  }
  __syncthreads();
  const int d = (int)threadIdx.x;
  float a = 0.f, b = 0.f;
  if (d < D) {
    a = -INFINITY;
    b = INFINITY;
    for (int i = 0; i < R; ++i) {
      a = fmaxf(a, top[0][i * D + d]);
      b = fminf(b, top[1][i * D + d]);
    }
    if (a < b) a = b = 0.f;  // no finite value
  }
  float m = fmaxf(fabsf(a), fabsf(b));
  for (int x = 1; x < 64; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
  if (threadIdx.x % 64 == 0) wave_top[threadIdx.x / 64] = m;
  __syncthreads();
  for (int w = 0; w < kThreads / 64; ++w) m = fmaxf(m, wave_top[w]);
  const int f = step_exponent(m);
  const float unit = exponent((uint32_t)(127 - f));  // 2^-f
  const int padded = (2 * D + 63) / 64 * 64;
  if (d < D) {
    codes[d] = (int8_t)fminf(fmaxf(ceilf(a * unit), -127.f), 127.f);
    codes[D + d] = (int8_t)fminf(fmaxf(floorf(b * unit), -127.f), 127.f);
  }
  for (int i = 2 * D + d; i < padded; i += kThreads) codes[i] = 0;
  __syncthreads();
  char *row = (char *)bounds.rows + page * bounds.page_stride + h * bounds.head_stride;
  if (d < padded / 16) reinterpret_cast<uint4 *>(row)[d] = reinterpret_cast<const uint4 *>(codes)[d];
  if (d == 0) *reinterpret_cast<int32_t *>(row + padded) = f;
}

// ----------------------------------------------------------------- selection
// A workgroup per token and KV head.  max(q hi, q lo) is the positive part of q times hi plus its negative part times lo, so a
// page's sums for 16 query heads are a product of int8 rows twice as long, on the matrix cores: operand A the heads, B 16
// pages a wave reads from memory in the order of the operand.  Scores become keys that order as they do, in
// LDS; the count-th largest is found 8 bits at a time from histograms, and the list is written in the order of pages.
//
// Bounds cross the device once for the heads that share them, 2 head_dim + 16 bytes a page.
constexpr int kSelect = 512;
constexpr int kSelectWaves = kSelect / 64;

__device__ const uint4 g_zeros = {0, 0, 0, 0};

// Orders as the score does.
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t u = __float_as_uint(score);
  return u >> 31 ? ~u : u | 0x80000000u;
}

template <int KEYS>
__global__ __launch_bounds__(kSelect) void select_kernel(lora_kv_view kv, lora_kv_bounds bounds,
                                                         const int32_t *__restrict__ token_seq,
                                                         const int32_t *__restrict__ token_pos, const uint16_t *__restrict__ q,
                                                         int64_t q_ts, int64_t q_hs, int group, int count, int sink, int recent,
                                                         int32_t *__restrict__ blocks) {
  __shared__ uint32_t keys[KEYS];
  __shared__ __attribute__((aligned(16))) char qc[16][512];
  __shared__ float unit[16];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];
  __shared__ uint32_t part[2][kSelectWaves][2];
  const int h = blockIdx.x % kv.kv_heads, t = blockIdx.x / kv.kv_heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  int32_t *out = blocks + (int64_t)blockIdx.x * count;
  const int s = token_seq[t], pos = token_pos[t];
  const bool good = s >= 0 && s < kv.num_seqs && pos >= 0 && pos < kv.max_pages * kv.page_tokens;
  KV_CHECK(good || s < 0 || tid != 0, LORA_DEBUG_BAD_TOKEN);
  const int n = good ? pos / kv.page_tokens + 1 : 0;
  if (n <= count) {
    for (int i = tid; i < count; i += kSelect) out[i] = i < n ? i : -1;
    return;
  }
  const int32_t *table = kv.page_table + (int64_t)s * kv.max_pages;
  const int D = kv.head_dim, steps = (2 * D + 63) / 64;
  for (int g0 = 0; g0 < group; g0 += 16) {
    // the query rows in whole numbers: 32 threads a head, 8 elements each
    __syncthreads();
    {
      const int g = tid >> 5, c = tid & 31;
      const bool mine = g0 + g < group && c * 8 < D;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (mine) u = *reinterpret_cast<const uint4 *>(q + t * q_ts + (h * group + g0 + g) * q_hs + c * 8);
      float m = top8(u);
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor(m, x));
      const int e = step_exponent(m);
      const float inv = exponent((uint32_t)(127 - e));
      int up[8], down[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = bf16_at(u, i);
        const int w = std::isfinite(x) ? (int)fminf(fmaxf(rintf(x * inv), -127.f), 127.f) : 0;
        up[i] = max(w, 0);
        down[i] = min(w, 0);
      }
      if (c * 8 < D) {
        *reinterpret_cast<uint2 *>(&qc[g][c * 8]) = make_uint2(byte4(up), byte4(up + 4));
        *reinterpret_cast<uint2 *>(&qc[g][D + c * 8]) = make_uint2(byte4(down), byte4(down + 4));
      }
      if (2 * D + c * 8 < 64 * steps) *reinterpret_cast<uint2 *>(&qc[g][2 * D + c * 8]) = make_uint2(0, 0);
      if (c == 0) unit[g] = exponent((uint32_t)(127 + e));
    }
    __syncthreads();
    for (int p0 = 16 * wave; p0 < n; p0 += 16 * kSelectWaves) {
      const int p = p0 + fr, page = p < n ? table[p] : -1;
      const bool there = (unsigned)page < (unsigned)kv.num_pages;
      KV_CHECK(there || p >= n || fg != 0, LORA_DEBUG_BAD_PAGE);
      const char *row = there ? (const char *)bounds.rows + page * bounds.page_stride + h * bounds.head_stride : nullptr;
      const int f = there ? *reinterpret_cast<const int32_t *>(row + 64 * steps) : 0;
      i32x4_t sum = {0, 0, 0, 0};
      for (int k = 0; k < steps; ++k) {
        const uint4 b = *reinterpret_cast<const uint4 *>(there ? row + 64 * k + 16 * fg : (const char *)&g_zeros);
        const uint4 a = *reinterpret_cast<const uint4 *>(&qc[fr][64 * k + 16 * fg]);
        sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), sum, 0, 0, 0);
      }
      // column fr: this lane's page; rows 4 fg ..: heads
      float best = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (g0 + 4 * fg + e < group) best = fmaxf(best, (float)sum[e] * unit[4 * fg + e]);
      best = fmaxf(best, __shfl_xor(best, 16));
      best = fmaxf(best, __shfl_xor(best, 32));
      best = there ? best * exponent((uint32_t)(127 + min(max(f, -50), 50))) : -INFINITY;
      if (fg == 0 && p < n) {
        const uint32_t key = p < sink || p >= n - recent ? ~0u : key_of(best);
        keys[p] = g0 == 0 ? key : max(keys[p], key);
      }
    }
  }
  // the count-th largest key, from its highest 8 bits to its lowest
  uint32_t prefix = 0, fixed = 0, need = (uint32_t)count;
  for (int shift = 24; shift >= 0; shift -= 8) {
    __syncthreads();
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelect)
      if ((keys[i] & fixed) == prefix) atomicAdd(&hist[keys[i] >> shift & 255], 1u);
    __syncthreads();
    if (wave == 0) {
      // keys of higher digits than this lane's 4
      uint32_t bin[4], all = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) all += bin[x] = hist[4 * lane + x];
      uint32_t above = all;
      for (int x = 1; x < 64; x <<= 1) {
        const uint32_t y = __shfl_down(above, x);
        above += lane + x < 64 ? y : 0;
      }
      above -= all;
#pragma unroll
      for (int x = 3; x >= 0; --x) {
        if (above < need && above + bin[x] >= need) {
          found[0] = 4 * lane + x;
          found[1] = need - above;
        }
        above += bin[x];
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    fixed |= 255u << shift;
    need = found[1];
  }
  // all keys above it and the first `need` that equal it, in the order of pages
  uint32_t more = 0, same = 0;  // in the pages before
  for (int p0 = 0, turn = 0; p0 < n; p0 += kSelect, turn ^= 1) {
    const int p = p0 + tid;
    const uint32_t key = p < n ? keys[p] : 0;
    const uint64_t gt = __ballot(p < n && key > prefix), eq = __ballot(p < n && key == prefix);
    if (lane == 0) {
      part[turn][wave][0] = __popcll(gt);
      part[turn][wave][1] = __popcll(eq);
    }
    __syncthreads();
    const uint64_t below = (1ull << lane) - 1;
    uint32_t g = more + __popcll(gt & below), e = same + __popcll(eq & below);
#pragma unroll
    for (int w = 0; w < kSelectWaves; ++w) {
      g += w < wave ? part[turn][w][0] : 0;
      e += w < wave ? part[turn][w][1] : 0;
      more += part[turn][w][0];
      same += part[turn][w][1];
    }
    if (p < n && (key > prefix || (key == prefix && e < need))) out[g + min(e, need)] = p;
  }
}

lora_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, what);
}

lora_status check_bounds(const lora_kv_bounds *b) {
  if (!b) return fail(LORA_EINVAL, "null bounds");
  if (((uintptr_t)b->rows & 15) || b->page_stride < 0 || b->head_stride < 0 || b->page_stride % 16 || b->head_stride % 16)
    return fail(LORA_EINVAL, "bounds must be 16-byte aligned, their strides multiples of 16, not negative");
  return LORA_OK;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3) == 0; }

}  // namespace

lora_status lora::kv_blocks_debug(uint32_t *flags, int32_t clear) { return kv_debug_word(flags, clear); }

extern "C" lora_status lora_kv_bounds_update(const lora_kv_view *kv, const lora_kv_bounds *bounds, const int32_t *seq,
                                             const int32_t *begin, const int32_t *end, int32_t n, int32_t max_tokens,
                                             hipStream_t stream) {
  lora_status st = check_view(kv);
  if (st == LORA_OK) st = check_bounds(bounds);
  if (st != LORA_OK) return st;
  if (n < 0 || max_tokens < 0) return fail(LORA_EINVAL, "%d ranges of %d positions", n, max_tokens);
  if (n == 0 || max_tokens == 0 || kv->num_pages == 0 || kv->num_seqs == 0 || kv->max_pages == 0) return ok();
  if (!bounds->rows || !seq || !begin || !end) return fail(LORA_EINVAL, "null pointer");
  if (!aligned4(seq) || !aligned4(begin) || !aligned4(end)) return fail(LORA_EINVAL, "seq, begin and end must be 4-byte aligned");
  // pages that max_tokens positions may lie on
  int64_t pages = ((int64_t)max_tokens + kv->page_tokens - 2) / kv->page_tokens + 1;
  if (pages > kv->max_pages) pages = kv->max_pages;
  if (pages * kv->kv_heads >= 1 << 24 || pages * kv->kv_heads * n >= 1 << 24)
    return fail(LORA_EUNSUPPORTED, "bounds of too many pages for one launch");
  const auto kernel = kv->dtype == LORA_FP8_E4M3 ? bounds_kernel<true> : bounds_kernel<false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(pages * kv->kv_heads * n)), dim3(kThreads), 0, stream, view8(kv), *bounds, seq,
                     begin, end, max_tokens, (int)pages);
  return launched("bounds launch");
}

extern "C" lora_status lora_kv_block_select(const lora_kv_view *kv, const lora_kv_bounds *bounds,
                                            const int32_t *token_seq, const int32_t *token_pos, int32_t num_tokens,
                                            const void *q, int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads,
                                            int32_t count, int32_t sink, int32_t recent, int32_t *blocks,
                                            hipStream_t stream) {
  lora_status st = check_view(kv);
  if (st == LORA_OK) st = check_bounds(bounds);
  if (st != LORA_OK) return st;
  if (num_tokens < 0 || q_heads < 1 || q_heads % kv->kv_heads)
    return fail(LORA_EINVAL, "%d tokens of %d query heads over %d KV heads", num_tokens, q_heads, kv->kv_heads);
  if (count < 1 || sink < 0 || recent < 1 || (int64_t)sink + recent > count)
    return fail(LORA_EINVAL, "lists of %d pages, the first %d and the last %d among them", count, sink, recent);
  if (count > LORA_BLOCKS_MAX_COUNT) return fail(LORA_EUNSUPPORTED, "lists of %d pages, not 1..%d", count, LORA_BLOCKS_MAX_COUNT);
  if (kv->max_pages > LORA_BLOCKS_MAX_PAGES)
    return fail(LORA_EUNSUPPORTED, "sequences of up to %d pages, not %d", kv->max_pages, LORA_BLOCKS_MAX_PAGES);
  if (q_token_stride < 0 || q_head_stride < 0 || q_token_stride % 8 || q_head_stride % 8)
    return fail(LORA_EINVAL, "strides of q must be multiples of 8 elements, not negative");
  if ((int64_t)num_tokens * kv->kv_heads >= 1 << 24) return fail(LORA_EUNSUPPORTED, "too many tokens for one launch");
  if (num_tokens == 0) return ok();
  const bool some = kv->num_pages > 0 && kv->num_seqs > 0 && kv->max_pages > 0;
  if (!token_seq || !token_pos || !q || !blocks || (some && !bounds->rows)) return fail(LORA_EINVAL, "null pointer");
  if (((uintptr_t)q & 15) || !aligned4(token_seq) || !aligned4(token_pos) || !aligned4(blocks))
    return fail(LORA_EINVAL, "q must be 16-byte aligned, the other arrays 4-byte");
  // the keys' LDS leaves a compute unit several workgroups where sequences are short
  const auto kernel = kv->max_pages <= 2048 ? select_kernel<2048> : kv->max_pages <= 8192 ? select_kernel<8192>
                                                                                          : select_kernel<LORA_BLOCKS_MAX_PAGES>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(num_tokens * kv->kv_heads)), dim3(kSelect), 0, stream, *kv, *bounds, token_seq,
                     token_pos, (const uint16_t *)q, q_token_stride, q_head_stride, q_heads / kv->kv_heads, count, sink, recent,
                     blocks);
  return launched("page selection launch");
}
