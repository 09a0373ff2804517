// Attention over the paged KV cache: the kernels, instantiated by kv_attn*.hip for each kind of cache (bf16 or 8-bit
// rows) and of mask.
//
// One pass over the positions with the running maximum m and sum l of each row's
// softmax: for a tile of positions, S = scale log2(e) K Q^T, m' = max(m, max S),
// P = 2^(S - m'), l = l 2^(m - m') + sum P, O = O 2^(m - m') + V^T P.  Products run on
// the matrix cores with positions as rows (S^T = K Q^T, O^T = V^T P^T): a lane then
// holds one row's scores in its registers, so maximum and sum are register
// operations and two exchanges between lane groups, and P^T is already the operand that
// its product with V needs, up to an order of positions that V's operand is read in too.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kv_internal.h"
#include "kv_debug.h"
#include "kv8.h"
#include "lds_load.h"

namespace lora {

// Which positions a row keeps of those that its item covers: the causal ones of a window (or all), a drafted tree's, or all
// up to its own on the pages that a list names.
enum class Mask { kCausal, kTree, kBlocks };

// n / d for 0 <= n < 2^31 by multiplication: m = floor(2^(31 + s) / d) + 1 with 2^s >= d > 2^(s - 1) exceeds
// 2^(31 + s) / d by at most 1, so n m / 2^(31 + s) exceeds n / d by less than 2^-s <= 1 / d: the same
// whole part.  m fits 32 bits, and so does 2 n.
struct Div {
  uint32_t m, s;
  Div(uint32_t d = 1) : s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)((1ull << (31 + s)) / d + 1);
  }
  __device__ __forceinline__ int operator()(int n) const { return (int)(__umulhi(2u * (uint32_t)n, m) >> s); }
};

struct AttnArgs {
  lora_kv_view kv;
  Div page_div;  // by kv.page_tokens
  uint32_t page16, token16;  // strides in units of 16 bytes
  const lora_attn_item *items;
  const uint16_t *q;
  uint16_t *out;
  float *lse;
  float *part_o;    // [num_part_rows][kv_heads][head_dim]: normalised results of one range
  float *part_lse;  // [num_part_rows][kv_heads]: base-2 logarithm of its sum
  int64_t q_ts, q_hs, o_ts, o_hs;
  float scale2;     // |scale| log2(e), 1 for a scale of 0
  uint32_t q_and, q_xor;  // see query()
  int32_t q_heads, group, causal, window, num_tokens, num_part_rows;
};
// What 8-bit rows and the other masks add; kernels that need none of it are not handed it.
struct AttnMoreArgs : AttnArgs {
  const uint8_t *k_scales, *v_scales;
  int64_t scale_hs;
  uint32_t scale_ps, scale_ts;
  const uint64_t *tree_mask;  // [num_tokens][tree_words]
  const int32_t *tree_depth;
  const int32_t *blocks;      // [num_tokens][kv_heads][count]
  const int32_t *token_pos;
  int32_t tree_words, count;
};

// The items of a plan, row items and then tile items (kv_attn.hip launches those over bf16 with a causal mask, and the joins).
void attn_items_tree(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream);
void attn_items_blocks(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream);
void attn8_items(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream);
void attn8_items_tree(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream);
void attn8_items_blocks(const AttnMoreArgs &a, const lora_attn_plan &plan, hipStream_t stream);

}  // namespace lora

namespace {

using namespace lora;
using Args = AttnArgs;
template <bool F8, Mask M>
using ArgsOf = std::conditional_t<!F8 && M == Mask::kCausal, AttnArgs, AttnMoreArgs>;

typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x2_t __attribute__((ext_vector_type(2)));

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));  // nearest even
}
__device__ __forceinline__ bool not_finite(uint16_t b) { return (b & 0x7f80u) == 0x7f80u; }
__device__ __forceinline__ float bf16_val(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// A query fragment times the sign of the scale (0 for a scale of 0), so that the factor left over is above 0.
__device__ __forceinline__ bf16x8_t query(const Args &a, uint4 u) {
  return __builtin_bit_cast(bf16x8_t, make_uint4((u.x & a.q_and) ^ a.q_xor, (u.y & a.q_and) ^ a.q_xor,
                                                 (u.z & a.q_and) ^ a.q_xor, (u.w & a.q_and) ^ a.q_xor));
}

// Maximum or sum over the four lane groups of 16 (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float max_groups(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_groups(float v) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// From a head's first exponent byte to that of a position.
__device__ __forceinline__ uint64_t scale_at(const AttnMoreArgs &a, int page, int slot) {
  return (uint64_t)(uint32_t)page * a.scale_ps + (uint64_t)(uint32_t)slot * a.scale_ts;
}

// Bits j0 .. j0 + 63 of a tree's mask row; those below 0 and behind its words are 0.
__device__ __forceinline__ uint64_t tree_bits(const uint64_t *row, int words, int64_t j0) {
  if (j0 < 0) return j0 > -64 ? row[0] << (int)-j0 : 0;
  const int64_t q = j0 >> 6;
  const int s = (int)(j0 & 63);
  const uint64_t lo = q < words ? row[q] : 0;
  return s == 0 ? lo : lo >> s | (q + 1 < words ? row[q + 1] << (64 - s) : 0);
}

// Whether an item read from the device lies within the plan and the view.  Items over listed pages are of one token each
// and have positions within its list.
template <Mask M, typename A>
__device__ __forceinline__ bool good_item(const A &a, const lora_attn_item &it, int max_rows) {
  int most = a.kv.max_pages * a.kv.page_tokens;
  if constexpr (M == Mask::kBlocks) {
    most = a.count * a.kv.page_tokens;
    if (it.row0 + (int64_t)it.rows > a.group) return false;
  }
  return it.rows >= 1 && it.rows <= max_rows && it.row0 >= 0 && it.q_begin >= 0 && it.row0 <= INT32_MAX - max_rows &&
         it.q_begin + (int64_t)(it.row0 + it.rows - 1) / a.group < a.num_tokens && it.seq >= 0 &&
         it.seq < a.kv.num_seqs && it.kv_begin >= 0 && it.kv_begin <= it.kv_end &&
         it.kv_end <= most && it.part >= -1 &&
         (int64_t)it.part + it.rows <= a.num_part_rows + (it.part < 0 ? (int64_t)INT32_MAX : 0);
}

// p, or where an absent row or column is read.
__device__ const uint4 g_zeros = {0, 0, 0, 0};
__device__ __forceinline__ const void *pick(bool use, const void *p) {
  const uintptr_t mask = (uintptr_t)0 - (uintptr_t)use;
  return reinterpret_cast<const void *>((reinterpret_cast<uintptr_t>(p) & mask) |
                                        (reinterpret_cast<uintptr_t>(&g_zeros) & ~mask));
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
  const int lo = __shfl((int)(uint32_t)v, lane), hi = __shfl((int)(v >> 32), lane);
  return (int64_t)(uint32_t)lo | ((int64_t)hi << 32);
}

constexpr float kSlack = 8.f;

// Chunks of 16 bytes of a row are stored permuted so that LDS reads spread over the banks: K
// is read as 8 rows of one chunk at a time, V as 4 rows of four neighbouring chunks (tile
// items) or 8 rows of two (row items).
template <int DP>
struct Layout {
  static constexpr int kRowBytes = 2 * DP;
  static constexpr int kCpr = DP / 8;  // chunks per row
  __device__ static __forceinline__ int k_slot(int row, int c) {
    return c ^ (row & (kCpr % 16 == 0 ? 15 : kCpr % 8 == 0 ? 7 : 3));
  }
  __device__ static __forceinline__ int v_slot(int row, int c) {
    if constexpr (kCpr % 16 == 0) return c ^ ((row & 3) << 2);
    else if constexpr (kCpr % 8 == 0) return c ^ ((row & 2) << 1);
    else return c;  // rows of 192 bytes are spread by themselves
  }
};
template <int DP>
struct RowLayout : Layout<DP> {
  __device__ static __forceinline__ int v_slot(int row, int c) { return Layout<DP>::v_slot(row, c) ^ ((row & 4) >> 1); }
};
// Rows of 8-bit codes: K is read as 16 rows of one chunk, V as the 8 rows 4 g .. 4 g + 3 and 16 + 4 g .. of one chunk for
// two neighbouring g at a time.  Chunks lie in 16 groups of banks, those of the same chunk in 16 / kCpr rows after one
// another; the bits of the row above those choose a slot.
template <int DP>
struct Layout8 {
  static constexpr int kRowBytes = DP;
  static constexpr int kCpr = DP / 16;
  static_assert(kCpr == 4 || kCpr == 8 || kCpr == 12 || kCpr == 16);
  __device__ static __forceinline__ int k_slot(int row, int c) {
    return c ^ (kCpr == 16 ? row & 15 : kCpr == 8 ? row >> 1 & 7 : row >> 2 & 3);
  }
  __device__ static __forceinline__ int v_slot(int row, int c) {
    const int hi = row >> 4 & 1;
    return c ^ (kCpr == 16 ? (row & 7) | hi << 3 : kCpr == 8 ? (row >> 1 & 3) | hi << 2 : (row >> 2 & 1) | hi << 1);
  }
};

// Loads of one wave for a tile of positions: its rows of K and V, chunk c = 64 (S i + W) + lane of load i being row c / kCpr
// in LDS slot c % kCpr.  `at`: this lane's position's row in units of 16 bytes from the head's first, -1 where it is
// absent (`exist` has bit l for lane l's position); `first`: this wave's first chunk.
template <typename L, int LOADS, int STRIDE, int LANES, bool FULL>
__device__ __forceinline__ void load_tile(const char *k, const char *v, int64_t at, uint64_t exist, int first, int nch,
                                          uint32_t kb, uint32_t vb) {
  const int lane = threadIdx.x & 63;
  constexpr uint64_t kAll = LANES == 64 ? ~0ull : (1ull << LANES) - 1;
  if (FULL && (exist & kAll) == kAll) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int c = first + 64 * STRIDE * i + lane, r = c / L::kCpr, slot = c % L::kCpr;
      const int64_t ra = shfl64(at, r) << 4;
      load_lds16(k + L::k_slot(r, slot) * 16 + ra, kb + (first + 64 * STRIDE * i) * 16);
      load_lds16(v + L::v_slot(r, slot) * 16 + ra, vb + (first + 64 * STRIDE * i) * 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int c = first + 64 * STRIDE * i + lane, r = c / L::kCpr, slot = c % L::kCpr;
      const int64_t ra = shfl64(at, r);
      const int kc = L::k_slot(r, slot), vc = L::v_slot(r, slot);
      load_lds16(pick(ra >= 0 && kc < nch, k + kc * 16 + (ra << 4)), kb + (first + 64 * STRIDE * i) * 16);
      load_lds16(pick(ra >= 0 && vc < nch, v + vc * 16 + (ra << 4)), vb + (first + 64 * STRIDE * i) * 16);
    }
  }
}

// ----------------------------------------------------------------- row items
// Up to 16 rows (the query heads of one KV head, for one or a few tokens) against
// positions [kv_begin, kv_end), or the positions with these numbers in a list of pages.  The waves take tiles of 32
// positions in turn, each with a softmax of its own and two LDS stages of its own: while a wave computes on one stage
// its loads of the next tile go straight into the other (16 bytes a lane, whole lines, any page per
// lane), with no barrier between waves.  The waves' results are joined at the end in wave order.
//
// Bound by HBM: K and V cross the device once.  What counts is bytes in flight: W waves hold
// W tiles of K and V.  64 tokens over 256 to 8192 positions, 64 / 8 heads of 128, 1.35 GB: 250 us, 5.4 TB/s; loads
// through registers take 492 us.  One token over few positions is bound by its chain of item, page
// entry, K, maximum and V (8.8 us for 200).
//
// 8-bit rows stay codes in LDS, half the bytes for each tile.  K's are widened as they are read, times the row's power of two;
// V's without theirs, which multiplies the softmax weight instead (exactly, before it is rounded), since an
// operand of V holds many positions.  The batch of 64 tokens above in 8 bits, 680 MB: 126 us with its join, 5.4 TB/s.  Lists of
// 64 pages of 64, 32 tokens, 64 / 8 heads of 128 in bf16, 537 MB: 96.6 us, 5.6 TB/s.
constexpr int kRowPos = 32;

template <int DP, bool F8>
using RowL = std::conditional_t<F8, Layout8<DP>, RowLayout<DP>>;

template <int DP, int W, bool FULL, bool F8, Mask M>
__global__ __launch_bounds__(64 * W) void attn_rows_kernel(ArgsOf<F8, M> a) {
  using L = RowL<DP, F8>;
  constexpr int KS = DP / 32, DT = DP / 16, LOADS = kRowPos * L::kCpr / 64;
  constexpr int kTile = kRowPos * L::kRowBytes, kStage = 2 * kTile + (F8 ? 256 : 0);  // K, V, the exponents of both
  constexpr int kTileLoads = 2 * LOADS + (F8 ? 1 : 0);
  static_assert(2 * kStage >= 16 * DP * 4);
  __shared__ __attribute__((aligned(16))) char lds[2][W * kStage];
  __shared__ float sm[W][16], sl[W][16];
  const lora_kv_view &kv = a.kv;
  const int h = blockIdx.x % kv.kv_heads, ii = blockIdx.x / kv.kv_heads;
  const lora_attn_item it = a.items[ii];
  if (!good_item<M>(a, it, LORA_ATTN_ROWS)) {
    KV_CHECK(threadIdx.x != 0, LORA_DEBUG_BAD_ITEM);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int D = FULL ? DP : kv.head_dim, nch = D * (F8 ? 1 : 2) >> 4;  // chunks of a stored row

  // loads: chunk c of a tile is row c / kCpr, LDS slot c % kCpr; lane l of load i takes c = 64 i + l
  const int32_t *table = kv.page_table + (int64_t)it.seq * kv.max_pages;
  const int first = it.kv_begin / kRowPos * kRowPos;
  const int tiles = (int)(((int64_t)it.kv_end - first + kRowPos - 1) / kRowPos);
  auto inside = [&](int64_t p) { return p >= it.kv_begin && p < it.kv_end; };
  // Listed pages: lane l holds the id of the list's page page0 + l, and how many of its positions are up to the token's own.
  int page0 = 0, ids = -1, kept = 0;
  auto fetch = [&](int from) {
    if constexpr (M == Mask::kBlocks) {
      const int32_t *list = a.blocks + ((int64_t)it.q_begin * kv.kv_heads + h) * a.count;
      const int e = from + lane < a.count ? list[from + lane] : -1;
      const bool in = (unsigned)e < (unsigned)kv.max_pages;
      ids = in ? table[e] : -1;
      kept = in ? (int)min(max((int64_t)a.token_pos[it.q_begin] + 1 - (int64_t)e * kv.page_tokens, (int64_t)0), (int64_t)kv.page_tokens) : 0;
      page0 = from;
      // waited for here, not at their uses among the tiles' loads, which the compiler does not count
      asm volatile("" : "+v"(ids), "+v"(kept));
    }
  };
  if constexpr (M == Mask::kBlocks) fetch(a.page_div(it.kv_begin));
  auto lookup = [&](int tile) {  // the page-table entry of the tile's position lane & 31, unused where that is outside
    const int64_t p = first + (int64_t)tile * kRowPos + (lane & 31);
    return M == Mask::kBlocks ? 0 : table[inside(p) ? a.page_div((int)p) : 0];
  };
  const char *kh = (const char *)kv.k + h * kv.head_stride * (F8 ? 1 : 2), *vh = (const char *)kv.v + h * kv.head_stride * (F8 ? 1 : 2);
  const uint8_t *eh = nullptr;  // lanes 0 .. 31 fetch K's exponents, the others V's
  if constexpr (F8) eh = (lane < 32 ? a.k_scales : a.v_scales) + h * a.scale_hs;
  auto issue = [&](auto bufc, int tile, int page) -> uint32_t {
    const int p = first + tile * kRowPos + (lane & 31), off = p - a.page_div(p) * kv.page_tokens;
    bool ok = inside(p);
    if constexpr (M == Mask::kBlocks) {
      const int begin = max(first + tile * kRowPos, it.kv_begin), end = (int)min(first + ((int64_t)tile + 1) * kRowPos, (int64_t)it.kv_end);
      const int lo = a.page_div(begin);
      if (lo < page0 || a.page_div(end - 1) >= page0 + 64) fetch(lo);  // 32 positions lie on 32 pages at most
      page = __shfl(ids, a.page_div(p) - page0);
      const int n = __shfl(kept, a.page_div(p) - page0);
      ok = ok && off < n;
    }
    KV_CHECK(!ok || (unsigned)page < (unsigned)kv.num_pages, LORA_DEBUG_BAD_PAGE);
    ok = ok && (unsigned)page < (unsigned)kv.num_pages;
    const int64_t at = (uint64_t)(uint32_t)page * a.page16 + (uint64_t)(uint32_t)off * a.token16;
    const uint64_t exist = __ballot(ok);  // bit i: the tile's position i exists
    const uint32_t kb = lds_offset(&lds[decltype(bufc)::value][wave * kStage]);
    load_tile<L, LOADS, 1, 32, FULL>(kh, vh, ok ? at : -1, exist, 0, nch, kb, kb + kTile);
    if constexpr (F8) {
      load_lds1(pick(ok, eh + scale_at(a, page, off)), kb + 2 * kTile);
    }
    return (uint32_t)exist;
  };

  // The order of a wave's loads is tile t, pages of t + 2, tile t + 1, pages of t + 3, ...: loads end in
  // order, so a tile's pages are there while the tile before it is still on its way.
  const bool any = wave < tiles;
  int page[2] = {any ? lookup(wave) : -1, any ? lookup(wave + W) : -1};  // of the next tile of each stage

  // this lane's row (a row past the item's computes row 0's token and is not stored)
  const int row = it.row0 + (fr < it.rows ? fr : 0);
  const int tok = row / a.group, head = h * a.group + (row - tok * a.group);
  const int64_t pos = (int64_t)it.pos0 + tok;
  const int hi = a.causal ? (int)max(pos, (int64_t)-1) : INT32_MAX;
  int lo = a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0;
  // every row of the item keeps the positions in [lo_all, hi_all] (a node is at most as deep as its number)
  const int64_t last = (int64_t)it.pos0 + (it.row0 + it.rows - 1) / a.group;
  const int lo_all = a.window ? (int)max(last - a.window + 1, (int64_t)0) : 0;
  int hi_all = a.causal ? (int)max((int64_t)it.pos0 + it.row0 / a.group, (int64_t)-1) : INT32_MAX;
  if constexpr (M == Mask::kTree) hi_all = min(hi_all, max(it.pos0, 0) - 1);
  if constexpr (M == Mask::kTree)
    lo = a.window ? (int)max((int64_t)it.pos0 + min(max(a.tree_depth[it.q_begin + tok], 0), tok) - a.window + 1, (int64_t)0) : 0;
  bf16x8_t qf[KS];
  const uint16_t *qp = a.q + (it.q_begin + tok) * a.q_ts + head * a.q_hs;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    // a lane's 8 elements of k-step s, in whichever order K's are read: 8-bit rows give two k-steps with each 16 bytes
    const int c = F8 ? 8 * (s / 2) + 2 * fg + s % 2 : 4 * s + fg;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (c * 8 < D) u = *reinterpret_cast<const uint4 *>(qp + c * 8);
    qf[s] = query(a, u);
  }

  f32x4_t o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;  // l: this lane's share of the positions

  uint32_t exist[2] = {0, 0};     // per stage

  auto step = [&](auto bufc, int tile) {
    constexpr int BUF = decltype(bufc)::value;
    char *const kb = &lds[BUF][wave * kStage], *const vb = kb + kTile;
    const uint32_t there = exist[BUF];
    const int t0 = first + tile * kRowPos;
    // this tile has landed once no more loads than the next tile's are outstanding
    if (tile + W < tiles) wait_vm<kTileLoads>();
    else wait_vm<0>();
    __builtin_amdgcn_wave_barrier();
    f32x4_t sc[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
    float vs[8];  // 8-bit: the factors of this lane's positions' rows of V
    if constexpr (F8) {
      const uint32_t *e = reinterpret_cast<const uint32_t *>(kb + 2 * kTile);
      const float ks[2] = {exponent(e[fr]), exponent(e[16 + fr])};
      const uint4 e0 = *reinterpret_cast<const uint4 *>(e + 32 + 4 * fg), e1 = *reinterpret_cast<const uint4 *>(e + 48 + 4 * fg);
      const uint32_t ev[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) vs[i] = exponent(ev[i]);
#pragma unroll
      for (int s = 0; s < KS; s += 2)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = 16 * half + fr;
          const uint4 u = *reinterpret_cast<const uint4 *>(kb + r * DP + L::k_slot(r, 2 * s + fg) * 16);
          sc[half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(u.x, u.y, ks[half]), qf[s], sc[half], 0, 0, 0);
          sc[half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(u.z, u.w, ks[half]), qf[s + 1], sc[half], 0, 0, 0);
        }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int r = 16 * half + fr;
          const bf16x8_t kf = __builtin_bit_cast(
              bf16x8_t, *reinterpret_cast<const uint4 *>(kb + 2 * r * DP + L::k_slot(r, 4 * s + fg) * 16));
          sc[half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[s], sc[half], 0, 0, 0);
        }
    }
    // scores: element e of this lane is position t0 + 4 fg + e (e < 4) or t0 + 16 + 4 fg + e - 4
    float s8[8];
    uint32_t keep = 255;
    bool hole = false;  // an existing position that this row does not keep
    float mt = -INFINITY;
    if (there == ~0u && t0 + (kRowPos - 1) <= hi_all && t0 >= lo_all) {  // every row keeps all of the tile
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s8[e] = sc[e >> 2][e & 3];
        mt = fmaxf(mt, s8[e]);
      }
    } else {
      uint32_t nodes = 0;  // drafted nodes that this row keeps, once the tile reaches them
      if constexpr (M == Mask::kTree)
        if ((int64_t)t0 + kRowPos > it.pos0)
          nodes = (uint32_t)tree_bits(a.tree_mask + (int64_t)(it.q_begin + tok) * a.tree_words, a.tree_words, (int64_t)t0 - it.pos0);
      keep = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = (e < 4 ? 4 * fg + e : 16 + 4 * fg + e - 4), p = t0 + i;
        const bool ex = there >> i & 1;
        bool ok = ex;
        if constexpr (M == Mask::kCausal) ok = ex && p <= hi && p >= lo;
        if constexpr (M == Mask::kTree) ok = ex && p <= hi && (p < it.pos0 ? p >= lo : (nodes >> i & 1));
        s8[e] = ok ? sc[e >> 2][e & 3] : -INFINITY;
        keep |= (uint32_t)ok << e;
        hole |= ex && !ok;
        // a position that is not kept may have any byte for its factor; absent ones have 0
        if constexpr (F8 && M != Mask::kBlocks) vs[e] = ok ? vs[e] : 0.f;
        mt = fmaxf(mt, s8[e]);
      }
    }
    mt = max_groups(mt);
    // the running maximum may lag by kSlack (see the tile items)
    if (__ballot((mt - m) * a.scale2 > kSlack)) {
      const float mn = fmaxf(m, mt);
      const float corr = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * a.scale2);
      l *= corr;
#pragma unroll
      for (int t = 0; t < DT; ++t) o[t] *= corr;
      m = mn;
    }
    const float base = m == -INFINITY ? 0.f : m * a.scale2;
    float sum = 0.f, p8[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p8[e] = __builtin_amdgcn_exp2f(fmaf(s8[e], a.scale2, -base));
      sum += p8[e];
    }
    l += sum;
    if (M != Mask::kBlocks && __ballot(hole)) {
      // 0 * inf is NaN: values that are not finite are added where they are kept, one position at a
      // time, and are zeros in the product
      bool odd = false;
      for (int c = lane; c < kRowPos * L::kCpr; c += 64) {
        const uint4 u = *reinterpret_cast<const uint4 *>(vb + c * 16);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          odd |= F8 ? nan8(w[e]) != 0 : not_finite((uint16_t)w[e]) || not_finite((uint16_t)(w[e] >> 16));
      }
      if (__ballot(odd)) {
        for (int r = 0; r < kRowPos; ++r) {
          const int idx = 4 * (r >> 4) + (r & 3), from = 16 * ((r & 15) >> 2) + fr;
          float pv = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) pv = idx == e ? p8[e] : pv;
          pv = __shfl(pv, from);
          const bool ok = __shfl((int)(keep >> idx & 1), from);
#pragma unroll
          for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int d = 16 * t + 4 * fg + j;
              if constexpr (F8) {
                const uint32_t v = (uint8_t)vb[r * DP + L::v_slot(r, d >> 4) * 16 + (d & 15)];
                if (ok && (v & 0x7f) == 0x7f) o[t][j] += NAN;
              } else {
                const uint16_t v = *reinterpret_cast<const uint16_t *>(vb + 2 * r * DP + L::v_slot(r, d >> 3) * 16 + (d & 7) * 2);
                if (ok && not_finite(v)) o[t][j] += pv * bf16_val(v);
              }
            }
        }
        __builtin_amdgcn_wave_barrier();
        if constexpr (F8) {
          for (int i = lane; i < kTile / 4; i += 64) {
            const uint32_t w = reinterpret_cast<uint32_t *>(vb)[i], bad = nan8(w) >> 7;
            if (bad) reinterpret_cast<uint32_t *>(vb)[i] = w & ~(bad * 0xffu);
          }
        } else {
          for (int i = lane; i < kRowPos * DP; i += 64)
            if (not_finite(reinterpret_cast<uint16_t *>(vb)[i])) reinterpret_cast<uint16_t *>(vb)[i] = 0;
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
    if constexpr (F8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p8[e] *= vs[e];
    }
    // rounded for the product only, as in the tile items
    const bf16x8_t pf = __builtin_bit_cast(
        bf16x8_t, make_uint4(pack_bf16(p8[0], p8[1]), pack_bf16(p8[2], p8[3]), pack_bf16(p8[4], p8[5]), pack_bf16(p8[6], p8[7])));
    if constexpr (F8) {
      // transposed reads: a group of 16 lanes names 8 rows x 16 columns, lane i gets column i's 8 values
      const int vr = (fr & 8 ? 16 : 0) + 4 * fg + (fr >> 1 & 3);
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        const i32x2_t x = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
            (__attribute__((address_space(3))) i32x2_t *)(vb + vr * DP + L::v_slot(vr, t) * 16 + (fr & 1) * 8));
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8((uint32_t)x[0], (uint32_t)x[1], 1.f), pf, o[t], 0, 0, 0);
      }
    } else {
      const int vr = 4 * fg + (fr >> 2);
#pragma unroll
      for (int t = 0; t < DT; ++t) {
        // transposed reads: a group of 16 lanes names 4 rows x 16 columns, lane i gets column i's 4 values
        uint2 x[2];
#pragma unroll
        for (int half = 0; half < 2; ++half)
          x[half] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t *)(
              vb + 2 * (16 * half + vr) * DP + L::v_slot(vr, 2 * t + ((fr & 3) >> 1)) * 16 + (fr & 1) * 8)));
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8_t, make_uint4(x[0].x, x[0].y, x[1].x, x[1].y)), pf, o[t], 0, 0, 0);
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (tile + 2 * W < tiles) {
      wait_lds();  // the reads of this stage are done
      exist[BUF] = issue(bufc, tile + 2 * W, page[BUF]);
      page[BUF] = lookup(tile + 4 * W);
    }
  };

  if (any) {
    exist[0] = issue(std::integral_constant<int, 0>{}, wave, page[0]);
    page[0] = lookup(wave + 2 * W);
    if (wave + W < tiles) {
      exist[1] = issue(std::integral_constant<int, 1>{}, wave + W, page[1]);
      page[1] = lookup(wave + 3 * W);
    }
    for (int t = wave; t < tiles; t += 2 * W) {
      step(std::integral_constant<int, 0>{}, t);
      if (t + W < tiles) step(std::integral_constant<int, 1>{}, t + W);
    }
  }
  l = sum_groups(l);
  m *= a.scale2;  // base-2 units; -inf where nothing is kept

  // join the waves in order
  __syncthreads();
  float (*so)[16][DP] = reinterpret_cast<float (*)[16][DP]>(lds);
  if (fg == 0) {
    sm[wave][fr] = m;
    sl[wave][fr] = l;
  }
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) so[wave][fr][16 * t + 4 * fg + j] = o[t][j];
  __syncthreads();
  const int nco = D >> 3;
  for (int i = threadIdx.x; i < it.rows * nco; i += 64 * W) {
    const int r = i / nco, c = i % nco;
    float top = sm[0][r];
    for (int w = 1; w < W; ++w) top = fmaxf(top, sm[w][r]);
    float f[W], total = 0.f;
    for (int w = 0; w < W; ++w) {
      f[w] = sl[w][r] == 0.f ? 0.f : __builtin_amdgcn_exp2f(sm[w][r] - top);  // nothing kept: no weight
      total += f[w] * sl[w][r];
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x = 0.f;
      for (int w = 0; w < W; ++w)
        if (sl[w][r] != 0.f) x += f[w] * so[w][r][8 * c + e];
      v[e] = x * inv;
    }
    const float lse2 = total == 0.f ? -INFINITY : top + log2f(total);
    if (it.part >= 0) {
      const int64_t pr = (int64_t)(it.part + r) * kv.kv_heads + h;
      float *po = a.part_o + pr * D + 8 * c;
      *reinterpret_cast<f32x4_t *>(po) = f32x4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_t *>(po + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
      if (c == 0) a.part_lse[pr] = lse2;
    } else {
      const int rr = it.row0 + r, tk = rr / a.group, hd = h * a.group + rr % a.group;
      *reinterpret_cast<uint4 *>(a.out + (it.q_begin + tk) * a.o_ts + hd * a.o_hs + 8 * c) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
      if (c == 0 && a.lse) a.lse[(int64_t)(it.q_begin + tk) * a.q_heads + hd] = lse2 * kLn2;
    }
  }
}

// ----------------------------------------------------------------- tile items
// Up to 128 rows against positions [kv_begin, kv_end): four waves of 32 rows share tiles of
// 64 positions, which go from the pages straight into LDS (16 bytes a lane, any page
// per lane) while the tile before is multiplied.
//
// The matrix cores are busy for 43 % of the time and the vector units for 46 %, most of it exponentials and the rounding of
// the weights, and nearly in turn: two waves share a SIMD, and those of a workgroup leave every barrier in the same phase.
// A chunk of 4096 tokens over 16384 positions, 64 / 8 heads of 128: 2.02 to 2.07 ms, 930 to 950 TFLOP/s; in items of 16
// rows, each reading K and V for itself, 22.1 ms.  Heads above 128 leave a SIMD one wave, and those above 192 spill 78
// registers a lane (2048 tokens over 8192, 32 / 8 heads: of 128 0.29 ms, of 192 0.54, of 256 0.70).
constexpr int kTileWaves = 4;
constexpr unsigned kUnits = 256;  // compute units
constexpr int kTilePos = 64;
template <int DP>
struct TileLayout : Layout<DP> {
  static constexpr int kLoads = kTilePos * Layout<DP>::kCpr / 64 / kTileWaves;  // per wave and operand
};

// Runs matrix instructions 0 .. N - 1, each with its operand read from LDS kLead instructions earlier.
// The order is fixed: left to itself the compiler reads each operand just before its use and waits.
constexpr int kLead = 3;
template <int N, typename F, typename R, typename M>
__device__ __forceinline__ void pipelined(R read, M multiply) {
  F f[kLead + 1];
#pragma unroll
  for (int n = 0; n < kLead && n < N; ++n) f[n] = read(n);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (n + kLead < N) f[(n + kLead) % (kLead + 1)] = read(n + kLead);
    __builtin_amdgcn_sched_barrier(0);
    multiply(n, f[n % (kLead + 1)]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// GR: groups of four waves with the same rows that take tiles in turn, each group with stages of its own, and are
// joined at the end: for grids that leave compute units with one workgroup, half as many tiles one
// after the other (a ragged batch of windowed chunks, 12 heads of 64: 22.5 us with one group, 19.0 with two).
template <int DP, bool FULL, int GR, bool F8, Mask M>
__global__ __launch_bounds__(64 * kTileWaves * GR, DP <= 128 ? 2 : 1) void attn_tile_kernel(ArgsOf<F8, M> a) {
  using L = TileLayout<DP>;
  constexpr int KS = DP / 16, DB = DP / 32, SB = kTilePos / 32;
  constexpr int kStage = kTilePos * DP;
  __shared__ __attribute__((aligned(16))) uint16_t sk0[GR * kStage], sk1[GR * kStage];
  __shared__ __attribute__((aligned(16))) uint16_t sv0[GR * kStage], sv1[GR * kStage];
  __shared__ uint32_t any_odd[kTileWaves * GR], masked[2][GR];
  const lora_kv_view &kv = a.kv;
  const int h = blockIdx.x % kv.kv_heads, ii = blockIdx.x / kv.kv_heads;
  const lora_attn_item it = a.items[ii];
  if (!good_item<M>(a, it, LORA_ATTN_TILE_ROWS)) {
    KV_CHECK(threadIdx.x != 0, LORA_DEBUG_BAD_ITEM);
    return;
  }
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wid / kTileWaves, wave = wid % kTileWaves;
  // Two workgroups share a compute unit, a wave of each a SIMD.  At equal priority both end late and at once, and where the last
  // round of them is not full half the device then waits for it; with one favoured the next workgroup starts sooner (8
  // chunks of 256 over 4096, 64 / 8 heads of 128, 640 workgroups: 171 us, else 204; 32 / 8 of 64, 16 of 256 over 2048: 61 and
  // 72).  In full rounds it costs a little (a chunk of 4096 over 8192, 32 / 8 of 64, 1024 workgroups: 291 us, favoured
  // 309), and over many rounds it gives little.  Bits 3:0 of the hardware's id register are the wave's slot in its SIMD.
  if (GR == 1 && DP <= 128 && gridDim.x > 2 * kUnits && gridDim.x < 16 * kUnits && gridDim.x % (2 * kUnits) != 0 &&
      (__builtin_amdgcn_s_getreg(4 | 3 << 11) & 1))
    __builtin_amdgcn_s_setprio(1);
  const int fr = lane & 31, hf = lane >> 5;
  const int D = FULL ? DP : kv.head_dim, nch = D >> 3;

  // loads: lane l looks up the tile's position l; chunk c of a tile is row c / kCpr, LDS slot c % kCpr, and lane l
  // of the wave's load i takes c = 64 (4 i + wave) + l
  const int32_t *table = kv.page_table + (int64_t)it.seq * kv.max_pages;
  const int first = it.kv_begin / kTilePos * kTilePos;
  const int tiles = (int)(((int64_t)it.kv_end - first + kTilePos - 1) / kTilePos);
  auto inside = [&](int64_t p) { return p >= it.kv_begin && p < it.kv_end; };
  auto lookup = [&](int tile) {  // a page-table entry, unused where the position is outside
    const int64_t p = first + (int64_t)tile * kTilePos + lane;
    return table[inside(p) ? a.page_div((int)p) : 0];
  };
  const char *kh = (const char *)kv.k + h * kv.head_stride * (F8 ? 1 : 2), *vh = (const char *)kv.v + h * kv.head_stride * (F8 ? 1 : 2);
  // 8-bit rows pass through registers, from where they are widened into a stage: chunk c = 64 (4 i + wave) + lane of 16 codes
  using L8 = Layout8<F8 ? DP : 64>;
  constexpr int kLoads8 = F8 ? kTilePos * L8::kCpr / 64 / kTileWaves : 1;
  uint4 raw[2][kLoads8];
  uint32_t exps[2] = {0, 0};  // of the tile's position `lane`
  const uint8_t *keh = nullptr, *veh = nullptr;
  if constexpr (F8) {
    keh = a.k_scales + h * a.scale_hs;
    veh = a.v_scales + h * a.scale_hs;
  }
  auto issue = [&](auto bufc, int tile, int page) -> uint64_t {
    constexpr int BUF = decltype(bufc)::value;
    const int p = first + tile * kTilePos + lane;
    const bool ok = inside(p) && (unsigned)page < (unsigned)kv.num_pages;
    KV_CHECK(ok || !inside(p), LORA_DEBUG_BAD_PAGE);
    const int64_t at = (uint64_t)(uint32_t)page * a.page16 + (uint64_t)(uint32_t)(p - a.page_div(p) * kv.page_tokens) * a.token16;
    const uint64_t there = __ballot(ok);  // bit i: the tile's position i exists
    if constexpr (F8) {
      const uint64_t e = scale_at(a, page, p - a.page_div(p) * kv.page_tokens);
      if (FULL && there == ~0ull) {
        exps[0] = keh[e];
        exps[1] = veh[e];
#pragma unroll
        for (int i = 0; i < kLoads8; ++i) {
          const int c = 64 * (kTileWaves * i + wave) + lane, ch = c % L8::kCpr;
          const int64_t ra = shfl64(at, c / L8::kCpr) << 4;
          raw[0][i] = *reinterpret_cast<const uint4 *>(kh + ch * 16 + ra);
          raw[1][i] = *reinterpret_cast<const uint4 *>(vh + ch * 16 + ra);
        }
      } else {
        exps[0] = *(const uint8_t *)pick(ok, keh + e);
        exps[1] = *(const uint8_t *)pick(ok, veh + e);
#pragma unroll
        for (int i = 0; i < kLoads8; ++i) {
          const int c = 64 * (kTileWaves * i + wave) + lane, ch = c % L8::kCpr;
          const int64_t ra = shfl64(ok ? at : -1, c / L8::kCpr);
          const bool here = ra >= 0 && ch < D >> 4;
          raw[0][i] = *reinterpret_cast<const uint4 *>(pick(here, kh + ch * 16 + (ra << 4)));
          raw[1][i] = *reinterpret_cast<const uint4 *>(pick(here, vh + ch * 16 + (ra << 4)));
        }
      }
    } else {
      load_tile<L, L::kLoads, kTileWaves, 64, FULL>(kh, vh, ok ? at : -1, there, 64 * wave, nch,
                                                    lds_offset(BUF ? sk1 : sk0) + group * kStage * 2,
                                                    lds_offset(BUF ? sv1 : sv0) + group * kStage * 2);
    }
    return there;
  };
  // the rows in registers into a stage, in pieces of 8 codes a lane.  Where a row's chunks divide the lanes, a lane's places
  // of the next load are the first one's some rows further on, and the layouts repeat after 16.
  auto place = [&](int i, int is_v, int half) {
    const int c = 64 * (kTileWaves * i + wave) + lane, r = c / L8::kCpr, ch = 2 * (c % L8::kCpr) + half;
    return r * DP + (is_v ? L::v_slot(r, ch) : L::k_slot(r, ch)) * 8;
  };
  constexpr int kMoreRows = 64 * kTileWaves / L8::kCpr;
  constexpr bool kRegular = 64 * kTileWaves % L8::kCpr == 0 && (kLoads8 == 1 || kMoreRows % 16 == 0);
  const int places[2][2] = {{place(0, 0, 0), place(0, 0, 1)}, {place(0, 1, 0), place(0, 1, 1)}};
  auto widen = [&](auto bufc, int piece) {
    constexpr int BUF = decltype(bufc)::value;
    const int i = piece / 4, half = piece % 2, is_v = piece / 2 % 2;  // K's and V's pieces of each load in turn
    uint16_t *to = (is_v ? (BUF ? sv1 : sv0) : (BUF ? sk1 : sk0)) + group * kStage + (kRegular ? places[is_v][half] + i * kMoreRows * DP : place(i, is_v, half));
    const uint4 u = raw[is_v][i];
    const float e = exponent(__shfl(exps[is_v], (64 * (kTileWaves * i + wave) + lane) / L8::kCpr));
    *reinterpret_cast<bf16x8_t *>(to) = widen8(half ? u.z : u.x, half ? u.w : u.y, e);
  };
  constexpr int kPieces = 4 * kLoads8;
  int page = tiles > 0 ? lookup(group) : -1;

  // this lane's row (a row past the item's computes the item's first one and is not stored)
  const int my = wave * 32 + fr;
  const int row = it.row0 + (my < it.rows ? my : 0);
  const int tok = row / a.group, head = h * a.group + (row - tok * a.group);
  auto highest = [&](int64_t pos) { return a.causal ? (int)max(pos, (int64_t)-1) : INT32_MAX; };
  auto lowest = [&](int64_t pos) { return a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0; };
  const int hi = highest((int64_t)it.pos0 + tok);
  int lo = lowest((int64_t)it.pos0 + tok);
  // every row of the item keeps the positions in [lo_all, hi_all]
  int hi_all = highest((int64_t)it.pos0 + it.row0 / a.group);
  const int lo_all = lowest((int64_t)it.pos0 + (it.row0 + it.rows - 1) / a.group);
  if constexpr (M == Mask::kTree) {
    // a node is at most as deep as its number, and every node keeps all of the context but what its window leaves off
    if (a.window) lo = lowest((int64_t)it.pos0 + min(max(a.tree_depth[it.q_begin + tok], 0), tok));
    hi_all = min(hi_all, max(it.pos0, 0) - 1);
  }
  bf16x8_t qf[KS];
  const uint16_t *qp = a.q + (it.q_begin + tok) * a.q_ts + head * a.q_hs;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (s * 2 + hf < nch) u = *reinterpret_cast<const uint4 *>(qp + (s * 2 + hf) * 8);
    qf[s] = query(a, u);
  }

  f32x16_t o[DB];
#pragma unroll
  for (int t = 0; t < DB; ++t) o[t] = f32x16_t{};
  float m = -INFINITY, l = 0.f;  // m: of the unscaled scores; l: this lane's half of the positions
  uint64_t exist[2] = {0, 0};    // per stage
  uint64_t ahead = 0;            // 8-bit: of the tile whose rows are in registers

  auto step = [&](auto bufc, int tile) {
    constexpr int BUF = decltype(bufc)::value;
    const uint16_t *kb = (BUF ? sk1 : sk0) + group * kStage;
    uint16_t *vb = (BUF ? sv1 : sv0) + group * kStage;
    const bool mine = GR == 1 || tile < tiles, active = mine && wave * 32 < it.rows;
    const int t0 = first + tile * kTilePos;
    bool whole = !mine || (exist[BUF] == ~0ull && hi_all >= t0 + (kTilePos - 1) && lo_all <= t0);
    if (GR > 1 && wave == 0 && lane == 0) masked[BUF][group] = !whole;
    if constexpr (!F8) wait_vm<0>();  // this wave's loads of the tile have landed
    __syncthreads();                  // everybody's have, and nobody reads the other stage any more
    if constexpr (GR > 1) whole = (masked[BUF][0] | masked[BUF][GR - 1]) == 0;  // the groups mask together: there are barriers
    const std::integral_constant<int, 1 - BUF> other{};
    if (!F8 && tile + GR < tiles) {
      exist[1 - BUF] = issue(other, tile + GR, page);
      page = lookup(tile + 2 * GR);
    }
    // element i of block b is position t0 + 32 b + 8 (i / 4) + 4 hf + i % 4
    f32x16_t s[SB];
    uint32_t keep = ~0u;
    float base = 0.f;
    if (active) {
      // S^T: positions are operand rows; the blocks in turn, so that no product waits for the one before
#pragma unroll
      for (int b = 0; b < SB; ++b) s[b] = f32x16_t{};
      pipelined<SB * KS, uint4>(
          [&](int n) {
            const int r = 32 * (n % SB) + fr, ks = n / SB;
            return *reinterpret_cast<const uint4 *>(kb + r * DP + L::k_slot(fr, 2 * ks + hf) * 8);
          },
          [&](int n, uint4 kf) {
            s[n % SB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, kf), qf[n / SB], s[n % SB], 0, 0, 0);
            // 8-bit: the next tile (behind the last, whatever the registers hold, which nobody reads) is widened while the
            // matrix instructions leave the vector units free
            static_assert(!F8 || SB * KS == 2 * kPieces);
            if (F8 && n % 2 == 0) widen(other, n / 2);
          });
    } else if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) widen(other, i);
    }
    if constexpr (F8) {
      exist[1 - BUF] = ahead;
      if (tile + 2 * GR < tiles) {
        ahead = issue(other, tile + 2 * GR, page);
        page = lookup(tile + 3 * GR);
      }
    }
    if (active) {
      if (!whole) {
        keep = 0;
        uint64_t nodes = 0;  // drafted nodes that this row keeps, once the tile reaches them
        if constexpr (M == Mask::kTree)
          if ((int64_t)t0 + kTilePos > it.pos0)
            nodes = tree_bits(a.tree_mask + (int64_t)(it.q_begin + tok) * a.tree_words, a.tree_words, (int64_t)t0 - it.pos0);
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = 32 * b + 8 * (i / 4) + 4 * hf + i % 4, p = t0 + r;
            bool ok = p <= hi && (exist[BUF] >> r & 1);
            if constexpr (M == Mask::kTree) ok = ok && (p < it.pos0 ? p >= lo : (nodes >> r & 1));
            else ok = ok && p >= lo;
            s[b][i] = ok ? s[b][i] : -INFINITY;
            keep |= (uint32_t)ok << (16 * b + i);
          }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < SB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[b][i]);
      auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
      mx = fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1]));
      // the running maximum may lag by kSlack (in powers of two): weights then stay below 2^kSlack, and the
      // rescaling of o, which most tiles would do for some row, is rare
      if (__ballot((mx - m) * a.scale2 > kSlack)) {
        const float mn = fmaxf(m, mx);
        const float corr = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * a.scale2);
        l *= corr;
#pragma unroll
        for (int t = 0; t < DB; ++t) o[t] *= corr;
        m = mn;
      }
      base = m == -INFINITY ? 0.f : m * a.scale2;
    }
    if (!whole) {
      // 0 * inf is NaN: values of V that are not finite are added where they are kept, one position at a
      // time, and are zeros in the product
      bool odd = false;
      for (int c = 64 * wave + lane; mine && c < kTilePos * L::kCpr; c += 64 * kTileWaves) {
        const uint4 u = *reinterpret_cast<const uint4 *>(vb + c * 8);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= not_finite((uint16_t)w[e]) || not_finite((uint16_t)(w[e] >> 16));
      }
      odd = __ballot(odd) != 0;
      if (lane == 0) any_odd[wid] = odd;
      __syncthreads();
      odd = false;
      for (int w = 0; w < kTileWaves * GR; ++w) odd |= any_odd[w] != 0;
      if (odd) {
        if (active) {
          for (int r = 0; r < kTilePos; ++r) {
            const int idx = 16 * (r >> 5) + 4 * ((r & 31) >> 3) + (r & 3), from = fr + 32 * (r >> 2 & 1);
            float pv = 0.f;
#pragma unroll
            for (int b = 0; b < SB; ++b)
#pragma unroll
              for (int i = 0; i < 16; ++i) pv = idx == 16 * b + i ? s[b][i] : pv;
            pv = __shfl(__builtin_amdgcn_exp2f(fmaf(pv, a.scale2, -base)), from);
            const bool ok = __shfl((int)(keep >> idx & 1), from);
#pragma unroll
            for (int t = 0; t < DB; ++t)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int d = 32 * t + 8 * (i / 4) + 4 * hf + i % 4;
                const uint16_t v = vb[r * DP + L::v_slot(r, d >> 3) * 8 + (d & 7)];
                if (ok && not_finite(v)) o[t][i] += pv * bf16_val(v);
              }
          }
        }
        __syncthreads();
        for (int i = 64 * wave + lane; i < kTilePos * DP; i += 64 * kTileWaves)
          if (not_finite(vb[i])) vb[i] = 0;
        __syncthreads();
      }
    }
    if (active) {
      // The weights are rounded to bf16 for this product, the sum takes them unrounded: out is 1.3 times as far from 64 bits
      // as its own rounding alone leaves it (0.0023 and 0.0017 of it).  A second product with what the rounding leaves off
      // would take as many matrix instructions again, and 0 * inf would make NaN of a kept infinite V.
      // O^T += V^T P^T: k-step ks holds positions 16 ks ..; this lane's half of P has 4 hf .. + 3 and 8 + 4 hf .. + 3
      const int li = lane & 15, vr = 4 * hf + (li >> 2);
      // The second block's weights are computed between the first block's products, which leave the vector
      // units free.
      bf16x8_t pf[kTilePos / 16];
      float sum[2] = {0.f, 0.f};
      auto weigh = [&](int b, int i) {
        s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], a.scale2, -base));
        sum[i & 1] += s[b][i];
      };
      auto round8 = [&](int ks) {
        const int b = ks / 2, e = 8 * (ks % 2);
        pf[ks] = __builtin_bit_cast(
            bf16x8_t, make_uint4(pack_bf16(s[b][e], s[b][e + 1]), pack_bf16(s[b][e + 2], s[b][e + 3]),
                                 pack_bf16(s[b][e + 4], s[b][e + 5]), pack_bf16(s[b][e + 6], s[b][e + 7])));
      };
#pragma unroll
      for (int i = 0; i < 16; ++i) weigh(0, i);
      round8(0);
      round8(1);
      pipelined<kTilePos / 16 * DB, uint4>(
          [&](int n) {
            const int ks = n / DB, c = 4 * (n % DB) + 2 * (lane >> 4 & 1) + ((li & 3) >> 1);
            uint2 x[2];
#pragma unroll
            for (int half = 0; half < 2; ++half)
              x[half] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4_t *)(vb + (16 * ks + 8 * half + vr) * DP + L::v_slot(vr, c) * 8 +
                                                                (li & 1) * 4)));
            return make_uint4(x[0].x, x[0].y, x[1].x, x[1].y);
          },
          [&](int n, uint4 vf) {
            o[n % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, vf), pf[n / DB], o[n % DB], 0, 0, 0);
            // 16 weights over the 2 DB products of the first block
#pragma unroll
            for (int i = 16 * n / (2 * DB); i < 16 * (n + 1) / (2 * DB) && i < 16; ++i) {
              weigh(1, i);
              if (i % 8 == 7) round8(2 + i / 8);
            }
          });
      l += sum[0] + sum[1];
    }
  };

  if (group < tiles) {
    exist[0] = issue(std::integral_constant<int, 0>{}, group, page);
    page = lookup(group + GR);
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) widen(std::integral_constant<int, 0>{}, i);
      if (group + GR < tiles) {
        ahead = issue(std::integral_constant<int, 0>{}, group + GR, page);
        page = lookup(group + 2 * GR);
      }
    }
  }
  for (int t = 0; t < tiles; t += 2 * GR) {
    step(std::integral_constant<int, 0>{}, t + group);
    if (t + GR < tiles) step(std::integral_constant<int, 1>{}, t + GR + group);
  }
  auto ls = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
  l = __uint_as_float(ls[0]) + __uint_as_float(ls[1]);
  if constexpr (GR > 1) {
    // the second group's results through LDS, lane by lane: the stages hold them
    static_assert(GR == 2 && 4 * GR * kStage * 2 >= kTileWaves * 64 * (16 * DB + 2) * 4);
    constexpr int kHalf = 16 * DB / 2 * 64 * kTileWaves;  // floats of half the rows' results: one of the four arrays
    static_assert(kHalf * 4 <= GR * kStage * 2 && 2 * 64 * kTileWaves * 4 <= GR * kStage * 2);
    float *part[2] = {reinterpret_cast<float *>(sk0), reinterpret_cast<float *>(sk1)};
    float *ml = reinterpret_cast<float *>(sv0);
    const int at = 64 * wave + lane;
    __syncthreads();
    if (group == 1) {
#pragma unroll
      for (int t = 0; t < DB; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(t * 16 + i) / (8 * DB)][(t * 16 + i) % (8 * DB) * 64 * kTileWaves + at] = o[t][i];
      ml[at] = m;
      ml[64 * kTileWaves + at] = l;
    }
    __syncthreads();
    if (group == 1) return;
    const float m1 = ml[at], l1 = ml[64 * kTileWaves + at], mn = fmaxf(m, m1);
    const float f0 = l == 0.f ? 0.f : __builtin_amdgcn_exp2f((m - mn) * a.scale2);  // nothing kept: no weight
    const float f1 = l1 == 0.f ? 0.f : __builtin_amdgcn_exp2f((m1 - mn) * a.scale2);
#pragma unroll
    for (int t = 0; t < DB; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float o1 = part[(t * 16 + i) / (8 * DB)][(t * 16 + i) % (8 * DB) * 64 * kTileWaves + at];
        o[t][i] = (l == 0.f ? 0.f : o[t][i] * f0) + (l1 == 0.f ? 0.f : o1 * f1);
      }
    l = l * f0 + l1 * f1;
    m = mn;
  }
  if (my >= it.rows) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float lse2 = l == 0.f ? -INFINITY : m * a.scale2 + log2f(l);
  const int64_t pr = (int64_t)(it.part + my) * kv.kv_heads + h;
  uint16_t *op = a.out + (it.q_begin + tok) * a.o_ts + head * a.o_hs;
#pragma unroll
  for (int t = 0; t < DB; ++t)
#pragma unroll
    for (int q4 = 0; q4 < 4; ++q4) {
      const int d = 32 * t + 8 * q4 + 4 * hf;
      if (d >= D) continue;
      f32x4_t v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = l == 0.f ? 0.f : o[t][4 * q4 + j] * inv;
      if (it.part >= 0) *reinterpret_cast<f32x4_t *>(a.part_o + pr * D + d) = v;
      else *reinterpret_cast<uint2 *>(op + d) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
  if (hf == 0) {
    if (it.part >= 0) a.part_lse[pr] = lse2;
    else if (a.lse) a.lse[(int64_t)(it.q_begin + tok) * a.q_heads + head] = lse2 * kLn2;
  }
}

// Heads of 64, 128 and 256, the usual ones, have kernels without the checks that shorter rows need (chunks of 64
// over 512 positions, 12 heads of 64: 12.8 us, with the checks 13.8; 8 chunks of 128 over 4096: 171 and 178).
template <int DP>
constexpr bool kFull = DP == 64 || DP == 128 || DP == 256;
template <int DP>
bool full(const Args &a) { return kFull<DP> && a.kv.head_dim == DP; }

template <int DP, bool F8, Mask M>
void launch_rows(const ArgsOf<F8, M> &a, unsigned grid, hipStream_t stream) {
  // two workgroups of half the waves share a compute unit's LDS and overlap their ends; a grid that gives
  // every compute unit one at most takes all the waves at once, for a shorter chain of tiles (heads of 128, 4 tokens
  // over 300 positions: 10.2 us, with half the waves 11.2; 8 tokens over 2048, 512 units: 32 us and 26)
  constexpr int W = (DP <= 64 ? 4 : DP <= 128 ? 2 : 1) * (F8 && DP > 64 ? 2 : 1);  // 8-bit stages take half the LDS
  const auto wide = full<DP>(a) ? attn_rows_kernel<DP, 2 * W, kFull<DP>, F8, M> : attn_rows_kernel<DP, 2 * W, false, F8, M>;
  const auto slim = full<DP>(a) ? attn_rows_kernel<DP, W, kFull<DP>, F8, M> : attn_rows_kernel<DP, W, false, F8, M>;
  // Many workgroups of half the waves again, where there are more than a compute unit holds: what counts for short items is how
  // many begin and end side by side (in 8 bits, 256 tokens over 75 to 300, 32 / 8 heads of 128: 29 us, else 40;
  // 64 over 128 to 512, 64 / 64: 73 and 92; 64 over 8192, 64 / 8, 1000 workgroups: 145 and 135.  Lists of 480 positions, 1812
  // workgroups, heads of 64: 21.1 and 25.4, bf16 27.4 and 36.6; of 2048 positions in 8 bits, 2048 workgroups, heads of
  // 128: 181 and 167).  The rule does not know how long the items of tokens are, and long ones are slower by it with heads of
  // 256, and with others in the first such grids alone (8-bit, 1280 workgroups, up to 1024 / 2048 / 8192 positions, half and all:
  // 64 / 8 of 128 41 and 47, 79 and 86, 285 and 283; 32 / 8 of 64 23 and 26, 41 and 42, 163 and 143; 16 / 8 of 256 93 and 95, 181
  // and 167, 707 and 602; 4096 workgroups of up to 8192, 64 / 8 of 128: 871 and 851).  bf16 rows with causal masks keep the waves that their sums have always been joined in.
  bool many = (F8 || M != Mask::kCausal) && W > 1 && grid >= (M == Mask::kBlocks ? 4 : 5) * kUnits;
  if constexpr (M == Mask::kBlocks) many = many && !(F8 && (int64_t)a.count * a.kv.page_tokens > 1024);
  if (many) {
    if constexpr ((F8 || M != Mask::kCausal) && W > 1) {
      const auto thin = full<DP>(a) ? attn_rows_kernel<DP, W / 2, kFull<DP>, F8, M> : attn_rows_kernel<DP, W / 2, false, F8, M>;
      hipLaunchKernelGGL(thin, dim3(grid), dim3(32 * W), 0, stream, a);
    }
  } else if (grid <= kUnits) {
    hipLaunchKernelGGL(wide, dim3(grid), dim3(128 * W), 0, stream, a);
  } else {
    hipLaunchKernelGGL(slim, dim3(grid), dim3(64 * W), 0, stream, a);
  }
}

template <int DP, bool F8, Mask M>
void launch_tiles(const ArgsOf<F8, M> &a, unsigned grid, hipStream_t stream) {
  // a grid of one workgroup per compute unit at most takes two groups of waves (4 chunks of 64 over 512 positions, 12
  // heads of 64: 12.8 us, with one group 13.9; 40 such chunks, 480 units: 86 us and 20)
  constexpr int G2 = DP <= 128 ? 2 : 1;  // what the LDS holds
  const auto one = full<DP>(a) ? attn_tile_kernel<DP, kFull<DP>, 1, F8, M> : attn_tile_kernel<DP, false, 1, F8, M>;
  const auto two = full<DP>(a) ? attn_tile_kernel<DP, kFull<DP>, G2, F8, M> : attn_tile_kernel<DP, false, G2, F8, M>;
  if (grid <= kUnits) hipLaunchKernelGGL(two, dim3(grid), dim3(64 * kTileWaves * G2), 0, stream, a);
  else hipLaunchKernelGGL(one, dim3(grid), dim3(64 * kTileWaves), 0, stream, a);
}


// A plan's row items, then its tile items, for the smallest padded head that holds this one.
template <bool F8, Mask M>
void launch_items(ArgsOf<F8, M> a, const lora_attn_plan &plan, hipStream_t stream) {
  const int dp = (a.kv.head_dim + 31) / 32 * 32;
  if (plan.num_row_items) {
    const unsigned grid = (unsigned)(plan.num_row_items * a.kv.kv_heads);
    if (dp <= 64) launch_rows<64, F8, M>(a, grid, stream);
    else if (!F8 && dp <= 96) launch_rows<F8 ? 128 : 96, F8, M>(a, grid, stream);
    else if (dp <= 128) launch_rows<128, F8, M>(a, grid, stream);
    else if (dp <= 192) launch_rows<192, F8, M>(a, grid, stream);
    else launch_rows<256, F8, M>(a, grid, stream);
  }
  if constexpr (M != Mask::kBlocks)
    if (plan.num_tile_items) {
      a.items += plan.num_row_items;
      const unsigned grid = (unsigned)(plan.num_tile_items * a.kv.kv_heads);
      if (dp <= 64) launch_tiles<64, F8, M>(a, grid, stream);
      else if (!F8 && dp <= 96) launch_tiles<F8 ? 128 : 96, F8, M>(a, grid, stream);
      else if (dp <= 128) launch_tiles<128, F8, M>(a, grid, stream);
      else if (dp <= 192) launch_tiles<192, F8, M>(a, grid, stream);
      else launch_tiles<256, F8, M>(a, grid, stream);
    }
}

}  // namespace
