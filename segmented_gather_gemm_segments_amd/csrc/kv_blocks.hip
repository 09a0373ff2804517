// Pages selected by bounds of their keys (lora_blocks.h): the bounds and the selection.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

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
// values through LDS.  Reads the page's keys once: 32 pages of 64 keys, 8 KV heads of 128, 7 us from memory, 4.9 from the last
// cache, most of it the launch and a chain of range, page and keys; a workgroup for each page keeps that chain one page long.
// The 33 pages of a prompt's chunk of 2048 take as long.  The grid has the longest range's pages for every range: that chunk beside
// 255 single tokens, 51 us as it comes and 13.4 with its range cut into pieces of two pages.
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
// Bounds cross the device once for the heads that share them, 2 head_dim + 16 bytes a page.  A wave keeps 4 groups of 16
// pages in flight where its workgroup has a compute unit to itself; 2 where several share one and registers decide how many
// (1024 lists of up to 125 pages: 11.6 us, with 4 groups 18.3), or head_dim is above 128.  32 tokens, 8 KV heads of 128,
// up to 512 pages, 23 MB of rows: 11.8 us back to back, where the last cache holds them, 14.2 from memory (a decoder reads its
// K and V in between).  Times below are of the first kind.  One compute unit reads no more than about 40 GB/s of such rows, so where lists are few and may
// be long a launch of its own scores their pages, 256 a workgroup, into a workspace (8 lists of 8125 pages: 21.5 us, in one
// launch 95).
__device__ const uint4 g_zeros = {0, 0, 0, 0};

// Orders as the score does.
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t u = __float_as_uint(score);
  return u >> 31 ? ~u : u | 0x80000000u;
}

struct Select {
  lora_kv_view kv;
  lora_kv_bounds bounds;
  const int32_t *token_seq, *token_pos;
  const uint16_t *q;
  int64_t q_ts, q_hs;
  int32_t group, count, sink, recent;
  int32_t *blocks;
  uint32_t *keys;  // [lists][max_pages], or null: scored by the workgroup that selects
};

// A list's token: its page table, its number of pages (0: none), from which its row of queries does not depend.
struct Token {
  const int32_t *table;
  int n;
};
__device__ __forceinline__ Token token_of(const Select &a, int t) {
  const int s = a.token_seq[t], pos = a.token_pos[t];
  const bool good = s >= 0 && s < a.kv.num_seqs && pos >= 0 && pos < a.kv.max_pages * a.kv.page_tokens;
  KV_CHECK(good || s < 0 || threadIdx.x != 0, LORA_DEBUG_BAD_TOKEN);
  return {a.kv.page_table + (int64_t)(good ? s : 0) * a.kv.max_pages, good ? pos / a.kv.page_tokens + 1 : 0};
}

// Keys of pages [begin, end) of token t's sequence and KV head h, each given to store(page, key, whether it is the first for
// its page) as often as there are 16 query heads; returns the page's key so far.  S: products of 64 numbers that a row of
// bounds takes at most; waves [0, WAVES) of the workgroup, with U groups of 16 pages in flight each.
template <int WAVES, int U, int S, typename Store>
__device__ __forceinline__ void score(const Select &a, const Token &token, int t, int h, int begin, int end, char (*qc)[512],
                                      float *unit, Store store) {
  const lora_kv_view &kv = a.kv;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int D = kv.head_dim, steps = (2 * D + 63) / 64;
  // the next turn's pages are looked up a load sooner, where registers are left for it (320 lists of up to 1000 pages: 28 us,
  // else 31; heads of 256, 694 lists of up to 469: 23 and 21.4).  Lists of few turns lose a little by it: 784 of up to 250 pages
  // 15.2 us, else 14.2.
  constexpr bool kAhead = S <= 4;
  constexpr int kTurn = 16 * U * WAVES;
  const int first = begin + 16 * wave;
  int page[U], next[U], f[U];
  i32x4_t b[U][S];
  auto look_up = [&](int p0) {
#pragma unroll
    for (int i = 0; i < U; ++i) next[i] = token.table[min(p0 + 16 * WAVES * i + fr, end - 1)];
  };
  auto load = [&](int p0) {
    if (!kAhead) look_up(p0);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      page[i] = next[i];
      KV_CHECK((unsigned)page[i] < (unsigned)kv.num_pages || fg != 0, LORA_DEBUG_BAD_PAGE);
      // an absent page's row is not read
      const bool there = (unsigned)page[i] < (unsigned)kv.num_pages;
      const char *row = (const char *)a.bounds.rows + page[i] * a.bounds.page_stride + h * a.bounds.head_stride;
      f[i] = *(there ? reinterpret_cast<const int32_t *>(row + 64 * steps) : reinterpret_cast<const int32_t *>(&g_zeros));
#pragma unroll
      for (int k = 0; k < S; ++k)
        b[i][k] = *reinterpret_cast<const i32x4_t *>(there && k < steps ? row + 64 * k + 16 * fg : (const char *)&g_zeros);
    }
    if (kAhead) look_up(p0 + kTurn < end ? p0 + kTurn : first);
  };
  if (kAhead) look_up(first);
  for (int g0 = 0; g0 < a.group; g0 += 16) {
    if (first < end) load(first);  // on its way while the queries are rounded
    if (g0) __syncthreads();       // the rows before have been read
    // the query rows in whole numbers: 32 threads a head, 8 elements each
    for (int g = tid >> 5; g < min(a.group - g0, 16); g += 2 * WAVES) {
      const int c = tid & 31;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (c * 8 < D) u = *reinterpret_cast<const uint4 *>(a.q + t * a.q_ts + (h * a.group + g0 + g) * a.q_hs + c * 8);
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
    for (int p0 = first; p0 < end; p0 += kTurn) {
      if (p0 != first) load(p0);
      i32x4_t sum[U];
#pragma unroll
      for (int i = 0; i < U; ++i) sum[i] = i32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < S; ++k) {
        if (k >= steps) break;
        const i32x4_t x = *reinterpret_cast<const i32x4_t *>(&qc[fr][64 * k + 16 * fg]);
#pragma unroll
        for (int i = 0; i < U; ++i) sum[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x, b[i][k], sum[i], 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        // column fr: this lane's page; rows 4 fg ..: heads
        const int p = p0 + 16 * WAVES * i + fr;
        float best = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g0 + 4 * fg + e < a.group) best = fmaxf(best, (float)sum[i][e] * unit[4 * fg + e]);
        best = fmaxf(best, __shfl_xor(best, 16));
        best = fmaxf(best, __shfl_xor(best, 32));
        best = (unsigned)page[i] < (unsigned)kv.num_pages ? best * exponent((uint32_t)(127 + min(max(f[i], -50), 50))) : -INFINITY;
        if (fg == 0 && p < end) store(p, key_of(best), g0 == 0);
      }
    }
  }
}

constexpr int kScorePages = 256;  // of a workgroup that only scores: two turns of its 4 waves

template <int S>
__global__ __launch_bounds__(256) void score_kernel(Select a, int parts) {
  __shared__ __attribute__((aligned(16))) char qc[16][512];
  __shared__ float unit[16];
  const int part = blockIdx.x % parts, list = blockIdx.x / parts, h = list % a.kv.kv_heads, t = list / a.kv.kv_heads;
  const Token token = token_of(a, t);
  const int begin = part * kScorePages, end = min(token.n, begin + kScorePages);
  if (token.n <= a.count || begin >= end) return;
  uint32_t *keys = a.keys + (int64_t)list * a.kv.max_pages;
  score<4, 2, S>(a, token, t, h, begin, end, qc, unit, [&](int p, uint32_t key, bool first) { keys[p] = first ? key : max(keys[p], key); });
}

template <int KEYS, int THREADS, int S>
__global__ __launch_bounds__(THREADS) void select_kernel(Select a) {
  constexpr int kWaves = THREADS / 64;
  __shared__ uint32_t keys[KEYS];
  __shared__ __attribute__((aligned(16))) char qc[16][512];
  __shared__ float unit[16];
  __shared__ uint32_t hist[256], found[3], range[kWaves][2], part[kWaves][2];
  const int h = blockIdx.x % a.kv.kv_heads, t = blockIdx.x / a.kv.kv_heads;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Token token = token_of(a, t);
  const int n = token.n, count = a.count, sink = a.sink, recent = a.recent;
  int32_t *out = a.blocks + (int64_t)blockIdx.x * count;
  if (n <= count) {
    for (int i = tid; i < count; i += THREADS) out[i] = i < n ? i : -1;
    return;
  }
  if (a.keys) {
    const uint32_t *from = a.keys + (int64_t)blockIdx.x * a.kv.max_pages;
    for (int i = tid; i < n; i += THREADS) keys[i] = from[i];
  } else {
    score<kWaves, (S <= 4 && THREADS > 256) ? 4 : 2, S>(a, token, t, h, 0, n, qc, unit, [&](int p, uint32_t key, bool first) { keys[p] = first ? key : max(keys[p], key); });
  }
  // Of the keys between the first and the last pages, which are listed anyway, the need-th largest: 8 bits at a time from the
  // highest in which they differ.  Counted from the least of them, so that their first digits spread over the bins (a
  // bin's additions come one after the other).
  uint32_t need = (uint32_t)(count - sink - recent);
  uint32_t least = ~0u, most = 0;
  for (int i = tid; i < 256; i += THREADS) hist[i] = 0;
  __syncthreads();
  for (int i = sink + tid; i < n - recent; i += THREADS) {
    least = min(least, keys[i]);
    most = max(most, keys[i]);
  }
  for (int x = 1; x < 64; x <<= 1) {
    least = min(least, (uint32_t)__shfl_xor(least, x));
    most = max(most, (uint32_t)__shfl_xor(most, x));
  }
  if (lane == 0) {
    range[wave][0] = least;
    range[wave][1] = most;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    least = min(least, range[w][0]);
    most = max(most, range[w][1]);
  }
  int left = need ? 32 - __clz(most - least) : 0;  // bits not looked at yet
  uint32_t prefix = 0;                              // the others, of the key that is looked for
  bool whole = need == 0;                           // all keys from the prefix on are listed
  if (whole) prefix = most - least + 1;
  while (left > 0 && !whole) {
    const int bits = min(left, 8), shift = left - bits;
    for (int i = sink + tid; i < n - recent; i += THREADS) {
      const uint32_t key = keys[i] - least;
      if (left == 32 || key >> left == prefix) atomicAdd(&hist[key >> shift & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    if (wave == 0) {
      // keys of higher digits than this lane's 4
      uint32_t bin[4], all = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        all += bin[x] = hist[4 * lane + x];
        hist[4 * lane + x] = 0;  // for the next digit
      }
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
          found[2] = above + bin[x] == need;
        }
        above += bin[x];
      }
    }
    __syncthreads();
    prefix = prefix << bits | found[0];
    need = found[1];
    whole = found[2];
    left = shift;
  }
  // Where a digit's keys are all listed the lower ones do not matter; else the prefix is the whole key, and of those that
  // equal it the first `need` are listed.  In the order of pages: each wave counts its share, then writes it.
  const int share = ((n + kWaves - 1) / kWaves + 63) / 64 * 64, begin = wave * share, end = min(n, begin + share);
  auto which = [&](int p, bool &over, bool &level) {
    const uint32_t key = p < end ? keys[p] - least : 0, high = left == 32 ? 0 : key >> left;
    const bool anyway = p < end && (p < sink || p >= n - recent), on = p < end && !anyway;
    over = anyway || (on && (high > prefix || (whole && high == prefix)));
    level = on && !whole && high == prefix;
  };
  uint32_t more = 0, same = 0;
  for (int p0 = begin; p0 < end; p0 += 64) {
    bool over, level;
    which(p0 + lane, over, level);
    more += __popcll(__ballot(over));
    same += __popcll(__ballot(level));
  }
  if (lane == 0) {
    part[wave][0] = more;
    part[wave][1] = same;
  }
  __syncthreads();
  more = same = 0;  // in the pages before
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    more += w < wave ? part[w][0] : 0;
    same += w < wave ? part[w][1] : 0;
  }
  for (int p0 = begin; p0 < end; p0 += 64) {
    bool over, level;
    which(p0 + lane, over, level);
    const uint64_t gt = __ballot(over), eq = __ballot(level), below = (1ull << lane) - 1;
    const uint32_t g = more + __popcll(gt & below), e = same + __popcll(eq & below);
    if (over || (level && e < need)) out[g + min(e, need)] = p0 + lane;
    more += __popcll(gt);
    same += __popcll(eq);
  }
}

constexpr int kMostKeys = 2048;  // of a workgroup of 512 threads or fewer

// Whether a call's pages are scored by a launch of their own: few lists that may be long.
bool splits(const lora_kv_view *kv, int64_t lists) { return lists > 0 && lists <= 64 && kv->max_pages > 512; }

lora_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, what);
}

// Checks that one launch can list the pages of so many tokens.
lora_status check_lists(const lora_kv_view *kv, int32_t num_tokens) {
  if (kv->max_pages > LORA_BLOCKS_MAX_PAGES)
    return fail(LORA_EUNSUPPORTED, "sequences of up to %d pages, not %d", kv->max_pages, LORA_BLOCKS_MAX_PAGES);
  const int64_t lists = (int64_t)num_tokens * kv->kv_heads;
  if (lists >= 1 << 24 || too_many(lists, kv->max_pages > kMostKeys ? 1024 : 256))
    return fail(LORA_EUNSUPPORTED, "too many tokens for one launch");
  return LORA_OK;
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

extern "C" lora_status lora_kv_block_select_workspace(const lora_kv_view *kv, int32_t num_tokens, int64_t *bytes) {
  lora_status st = check_view(kv);
  if (st != LORA_OK) return st;
  if (!bytes || num_tokens < 0) return fail(LORA_EINVAL, "%d tokens, or null bytes", num_tokens);
  if ((st = check_lists(kv, num_tokens)) != LORA_OK) return st;
  const int64_t lists = (int64_t)num_tokens * kv->kv_heads;
  *bytes = splits(kv, lists) ? lists * kv->max_pages * (int64_t)sizeof(uint32_t) : 0;
  return ok();
}

extern "C" lora_status lora_kv_block_select(const lora_kv_view *kv, const lora_kv_bounds *bounds,
                                            const int32_t *token_seq, const int32_t *token_pos, int32_t num_tokens,
                                            const void *q, int64_t q_token_stride, int64_t q_head_stride, int32_t q_heads,
                                            int32_t count, int32_t sink, int32_t recent, int32_t *blocks, void *workspace,
                                            int64_t workspace_bytes, hipStream_t stream) {
  lora_status st = check_view(kv);
  if (st == LORA_OK) st = check_bounds(bounds);
  if (st != LORA_OK) return st;
  if (num_tokens < 0 || q_heads < 1 || q_heads % kv->kv_heads)
    return fail(LORA_EINVAL, "%d tokens of %d query heads over %d KV heads", num_tokens, q_heads, kv->kv_heads);
  if (count < 1 || sink < 0 || recent < 1 || (int64_t)sink + recent > count)
    return fail(LORA_EINVAL, "lists of %d pages, the first %d and the last %d among them", count, sink, recent);
  if (count > LORA_BLOCKS_MAX_COUNT) return fail(LORA_EUNSUPPORTED, "lists of %d pages, not 1..%d", count, LORA_BLOCKS_MAX_COUNT);
  if (q_token_stride < 0 || q_head_stride < 0 || q_token_stride % 8 || q_head_stride % 8)
    return fail(LORA_EINVAL, "strides of q must be multiples of 8 elements, not negative");
  if ((st = check_lists(kv, num_tokens)) != LORA_OK) return st;
  const int64_t lists = (int64_t)num_tokens * kv->kv_heads;
  if (num_tokens == 0) return ok();
  const bool some = kv->num_pages > 0 && kv->num_seqs > 0 && kv->max_pages > 0;
  if (!token_seq || !token_pos || !q || !blocks || (some && !bounds->rows)) return fail(LORA_EINVAL, "null pointer");
  if (workspace_bytes < 0 || ((uintptr_t)workspace & 15)) return fail(LORA_EINVAL, "workspace of %lld bytes must be 16-byte aligned", (long long)workspace_bytes);
  if (((uintptr_t)q & 15) || !aligned4(token_seq) || !aligned4(token_pos) || !aligned4(blocks))
    return fail(LORA_EINVAL, "q must be 16-byte aligned, the other arrays 4-byte");
  const int64_t need = lists * kv->max_pages * (int64_t)sizeof(uint32_t);
  const int steps = (2 * kv->head_dim + 63) / 64, size = steps <= 2 ? 2 : steps <= 4 ? 4 : 8;
  Select a{*kv, *bounds, token_seq, token_pos, (const uint16_t *)q, q_token_stride, q_head_stride, q_heads / kv->kv_heads, count,
           sink, recent, blocks, nullptr};
  if (splits(kv, lists) && workspace && workspace_bytes >= need) {
    a.keys = (uint32_t *)workspace;
    const int parts = (kv->max_pages + kScorePages - 1) / kScorePages;
    const auto kernel = size == 2 ? score_kernel<2> : size == 4 ? score_kernel<4> : score_kernel<8>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(lists * parts)), dim3(256), 0, stream, a, parts);
  }
  // Threads of a workgroup: 512 where every compute unit has one of them at most, for a shorter way over the pages (256 lists of
  // up to 512 pages: 11.8 us, with 256 threads 15.2); 256 up to five a compute unit (1024 lists of up to 125 pages: 11.6 us,
  // with 128 threads 12.6); then 128, for fewer waves that wait for one wave's part (1812 lists of up to 209 pages: 12.5 us,
  // with 256 threads 16.1); 1024 for long sequences, whose keys leave a compute unit few workgroups.  Lengths are on the device,
  // so the table's width stands for them, and short sequences in a wide table pay for it: lists of up to 100 pages in a table of
  // up to 2048 and of more, 8 lists 8.0 and 10 us, 256 lists 8.2 and 11, 2048 lists 17 and 70.
  auto launch = [&](auto keys, auto threads) {
    constexpr int K = decltype(keys)::value, T = decltype(threads)::value;
    const auto kernel = size == 2 ? select_kernel<K, T, 2> : size == 4 ? select_kernel<K, T, 4> : select_kernel<K, T, 8>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)lists), dim3(T), 0, stream, a);
  };
  const std::integral_constant<int, 128> least{};
  const std::integral_constant<int, 256> small{};
  const std::integral_constant<int, 512> medium{};
  const std::integral_constant<int, 1024> large{};
  if (kv->max_pages > 8192) launch(std::integral_constant<int, LORA_BLOCKS_MAX_PAGES>{}, large);
  else if (kv->max_pages > kMostKeys) launch(std::integral_constant<int, 8192>{}, large);
  else if (lists <= 256) launch(std::integral_constant<int, kMostKeys>{}, medium);
  else if (lists <= 1280) launch(std::integral_constant<int, kMostKeys>{}, small);
  else launch(std::integral_constant<int, kMostKeys>{}, least);
  return launched("page selection launch");
}
