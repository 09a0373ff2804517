// Attention of new tokens over the paged KV cache (lora_kv.h).
//
// One pass over the positions with the running maximum m and sum l of each row's
// softmax: for a tile of positions, S = scale log2(e) K Q^T, m' = max(m, max S),
// P = 2^(S - m'), l = l 2^(m - m') + sum P, O = O 2^(m - m') + V^T P.  Products run on
// the matrix cores with positions as rows (S^T = K Q^T, O^T = V^T P^T): a lane then
// holds one row's scores in its registers, so maximum and sum are register
// operations and two exchanges between lane groups, and P^T is already the operand that
// its product with V needs, up to an order of positions that V's operand is read in too.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kv_internal.h"
#include "kv_debug.h"
#include "lds_load.h"

using namespace lora;

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(2))) float f32x2_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;

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

struct Args {
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

// Whether an item read from the device lies within the plan and the view.
__device__ __forceinline__ bool good_item(const Args &a, const lora_attn_item &it, int max_rows) {
  return it.rows >= 1 && it.rows <= max_rows && it.row0 >= 0 && it.q_begin >= 0 && it.row0 <= INT32_MAX - max_rows &&
         it.q_begin + (int64_t)(it.row0 + it.rows - 1) / a.group < a.num_tokens && it.seq >= 0 &&
         it.seq < a.kv.num_seqs && it.kv_begin >= 0 && it.kv_begin <= it.kv_end &&
         it.kv_end <= a.kv.max_pages * a.kv.page_tokens && it.part >= -1 &&
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
// positions [kv_begin, kv_end).  The waves take tiles of 32 positions in turn, each with a
// softmax of its own and two LDS stages of its own: while a wave computes on one stage its
// loads of the next tile go straight into the other (16 bytes a lane, whole lines, any page per
// lane), with no barrier between waves.  The waves' results are joined at the end in wave order.
//
// Bound by HBM: K and V cross the device once.  What counts is bytes in flight: W waves hold
// W tiles of K and V.  64 tokens over 256 to 8192 positions, 64 / 8 heads of 128, 1.35 GB: 250 us, 5.4 TB/s; loads
// through registers take 492 us.  One token over few positions is bound by its chain of item, page
// entry, K, maximum and V (8.8 us for 200).
constexpr int kRowPos = 32;

template <int DP, int W, bool FULL>
__global__ __launch_bounds__(64 * W) void attn_rows_kernel(Args a) {
  using L = RowLayout<DP>;
  constexpr int KS = DP / 32, DT = DP / 16, LOADS = kRowPos * L::kCpr / 64;
  __shared__ __attribute__((aligned(16))) uint16_t sk0[W * kRowPos * DP], sk1[W * kRowPos * DP];
  __shared__ __attribute__((aligned(16))) uint16_t sv0[W * kRowPos * DP], sv1[W * kRowPos * DP];
  __shared__ float sm[W][16], sl[W][16];
  const lora_kv_view &kv = a.kv;
  const int h = blockIdx.x % kv.kv_heads, ii = blockIdx.x / kv.kv_heads;
  const lora_attn_item it = a.items[ii];
  if (!good_item(a, it, LORA_ATTN_ROWS)) {
    KV_CHECK(threadIdx.x != 0, LORA_DEBUG_BAD_ITEM);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int fr = lane & 15, fg = lane >> 4;
  const int D = FULL ? DP : kv.head_dim, nch = D >> 3;
  const int off = wave * kRowPos * DP;  // this wave's part of each stage

  // loads: chunk c of a tile is row c / kCpr, LDS slot c % kCpr; lane l of load i takes c = 64 i + l
  const int32_t *table = kv.page_table + (int64_t)it.seq * kv.max_pages;
  const int first = it.kv_begin / kRowPos * kRowPos;
  const int tiles = (int)(((int64_t)it.kv_end - first + kRowPos - 1) / kRowPos);
  auto inside = [&](int64_t p) { return p >= it.kv_begin && p < it.kv_end; };
  auto lookup = [&](int tile) {  // the page-table entry of the tile's position lane & 31, unused where that is outside
    const int64_t p = first + (int64_t)tile * kRowPos + (lane & 31);
    return table[inside(p) ? a.page_div((int)p) : 0];
  };
  const char *kh = (const char *)kv.k + h * kv.head_stride * 2, *vh = (const char *)kv.v + h * kv.head_stride * 2;
  auto issue = [&](auto bufc, int tile, int page) -> uint32_t {
    constexpr int BUF = decltype(bufc)::value;
    const int p = first + tile * kRowPos + (lane & 31);
    const bool ok = inside(p) && (unsigned)page < (unsigned)kv.num_pages;
    KV_CHECK(ok || !inside(p), LORA_DEBUG_BAD_PAGE);
    const int64_t at = (uint64_t)(uint32_t)page * a.page16 + (uint64_t)(uint32_t)(p - a.page_div(p) * kv.page_tokens) * a.token16;
    const uint64_t exist = __ballot(ok);  // bit i: the tile's position i exists
    load_tile<L, LOADS, 1, 32, FULL>(kh, vh, ok ? at : -1, exist, 0, nch, lds_offset(BUF ? sk1 : sk0) + off * 2,
                                     lds_offset(BUF ? sv1 : sv0) + off * 2);
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
  const int lo = a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0;
  bf16x8_t qf[KS];
  const uint16_t *qp = a.q + (it.q_begin + tok) * a.q_ts + head * a.q_hs;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (s * 4 + fg < nch) u = *reinterpret_cast<const uint4 *>(qp + (s * 4 + fg) * 8);
    qf[s] = query(a, u);
  }

  f32x4_t o[DT];
#pragma unroll
  for (int t = 0; t < DT; ++t) o[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;  // l: this lane's share of the positions
  uint32_t exist[2] = {0, 0};     // per stage

  auto step = [&](auto bufc, int tile) {
    constexpr int BUF = decltype(bufc)::value;
    const uint16_t *kb = (BUF ? sk1 : sk0) + off;
    uint16_t *vb = (BUF ? sv1 : sv0) + off;
    const int t0 = first + tile * kRowPos;
    const uint32_t there = exist[BUF];
    // this tile has landed once no more loads than the next tile's are outstanding
    if (tile + W < tiles) wait_vm<2 * LOADS>();
    else wait_vm<0>();
    __builtin_amdgcn_wave_barrier();
    f32x4_t sc[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int r = 16 * half + fr;
        const bf16x8_t kf = __builtin_bit_cast(
            bf16x8_t, *reinterpret_cast<const uint4 *>(kb + r * DP + L::k_slot(r, 4 * s + fg) * 8));
        sc[half] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[s], sc[half], 0, 0, 0);
      }
    // scores: element e of this lane is position t0 + 4 fg + e (e < 4) or t0 + 16 + 4 fg + e - 4
    float s8[8];
    uint32_t keep = 0;
    bool hole = false;  // an existing position that this row does not keep
    float mt = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = (e < 4 ? 4 * fg + e : 16 + 4 * fg + e - 4), p = t0 + i;
      const bool ex = there >> i & 1, ok = ex && p <= hi && p >= lo;
      s8[e] = ok ? sc[e >> 2][e & 3] : -INFINITY;
      keep |= (uint32_t)ok << e;
      hole |= ex && !ok;
      mt = fmaxf(mt, s8[e]);
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
    if (__ballot(hole)) {
      // 0 * inf is NaN: values that are not finite are added where they are kept, one position at a
      // time, and are zeros in the product
      bool odd = false;
      for (int c = lane; c < kRowPos * L::kCpr; c += 64) {
        const uint4 u = *reinterpret_cast<const uint4 *>(vb + c * 8);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= not_finite((uint16_t)w[e]) || not_finite((uint16_t)(w[e] >> 16));
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
              const uint16_t v = vb[r * DP + L::v_slot(r, d >> 3) * 8 + (d & 7)];
              if (ok && not_finite(v)) o[t][j] += pv * bf16_val(v);
            }
        }
        __builtin_amdgcn_wave_barrier();
        for (int i = lane; i < kRowPos * DP; i += 64)
          if (not_finite(vb[i])) vb[i] = 0;
        __builtin_amdgcn_wave_barrier();
      }
    }
    // rounded for the product only, as in the tile items
    const bf16x8_t pf = __builtin_bit_cast(
        bf16x8_t, make_uint4(pack_bf16(p8[0], p8[1]), pack_bf16(p8[2], p8[3]), pack_bf16(p8[4], p8[5]), pack_bf16(p8[6], p8[7])));
    const int vr = 4 * fg + (fr >> 2);
#pragma unroll
    for (int t = 0; t < DT; ++t) {
      // transposed reads: a group of 16 lanes names 4 rows x 16 columns, lane i gets column i's 4 values
      uint2 x[2];
#pragma unroll
      for (int half = 0; half < 2; ++half)
        x[half] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t *)(
            vb + (16 * half + vr) * DP + L::v_slot(vr, 2 * t + ((fr & 3) >> 1)) * 8 + (fr & 1) * 4)));
      o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          __builtin_bit_cast(bf16x8_t, make_uint4(x[0].x, x[0].y, x[1].x, x[1].y)), pf, o[t], 0, 0, 0);
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
  float (*so)[16][DP] = reinterpret_cast<float (*)[16][DP]>(sk0);  // the same size
  if (fg == 0) {
    sm[wave][fr] = m;
    sl[wave][fr] = l;
  }
#pragma unroll
  for (int t = 0; t < DT; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) so[wave][fr][16 * t + 4 * fg + j] = o[t][j];
  __syncthreads();
  for (int i = threadIdx.x; i < it.rows * nch; i += 64 * W) {
    const int r = i / nch, c = i % nch;
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
template <int DP, bool FULL, int GR>
__global__ __launch_bounds__(64 * kTileWaves * GR, DP <= 128 ? 2 : 1) void attn_tile_kernel(Args a) {
  using L = TileLayout<DP>;
  constexpr int KS = DP / 16, DB = DP / 32, SB = kTilePos / 32;
  constexpr int kStage = kTilePos * DP;
  __shared__ __attribute__((aligned(16))) uint16_t sk0[GR * kStage], sk1[GR * kStage];
  __shared__ __attribute__((aligned(16))) uint16_t sv0[GR * kStage], sv1[GR * kStage];
  __shared__ uint32_t any_odd[kTileWaves * GR], masked[2][GR];
  const lora_kv_view &kv = a.kv;
  const int h = blockIdx.x % kv.kv_heads, ii = blockIdx.x / kv.kv_heads;
  const lora_attn_item it = a.items[ii];
  if (!good_item(a, it, LORA_ATTN_TILE_ROWS)) {
    KV_CHECK(threadIdx.x != 0, LORA_DEBUG_BAD_ITEM);
    return;
  }
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wid / kTileWaves, wave = wid % kTileWaves;
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
  const char *kh = (const char *)kv.k + h * kv.head_stride * 2, *vh = (const char *)kv.v + h * kv.head_stride * 2;
  auto issue = [&](auto bufc, int tile, int page) -> uint64_t {
    constexpr int BUF = decltype(bufc)::value;
    const int p = first + tile * kTilePos + lane;
    const bool ok = inside(p) && (unsigned)page < (unsigned)kv.num_pages;
    KV_CHECK(ok || !inside(p), LORA_DEBUG_BAD_PAGE);
    const int64_t at = (uint64_t)(uint32_t)page * a.page16 + (uint64_t)(uint32_t)(p - a.page_div(p) * kv.page_tokens) * a.token16;
    const uint64_t there = __ballot(ok);  // bit i: the tile's position i exists
    load_tile<L, L::kLoads, kTileWaves, 64, FULL>(kh, vh, ok ? at : -1, there, 64 * wave, nch,
                                                  lds_offset(BUF ? sk1 : sk0) + group * kStage * 2,
                                                  lds_offset(BUF ? sv1 : sv0) + group * kStage * 2);
    return there;
  };
  int page = tiles > 0 ? lookup(group) : -1;

  // this lane's row (a row past the item's computes the item's first one and is not stored)
  const int my = wave * 32 + fr;
  const int row = it.row0 + (my < it.rows ? my : 0);
  const int tok = row / a.group, head = h * a.group + (row - tok * a.group);
  auto highest = [&](int64_t pos) { return a.causal ? (int)max(pos, (int64_t)-1) : INT32_MAX; };
  auto lowest = [&](int64_t pos) { return a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0; };
  const int hi = highest((int64_t)it.pos0 + tok), lo = lowest((int64_t)it.pos0 + tok);
  // every row of the item keeps the positions in [lo_all, hi_all]
  const int hi_all = highest((int64_t)it.pos0 + it.row0 / a.group);
  const int lo_all = lowest((int64_t)it.pos0 + (it.row0 + it.rows - 1) / a.group);
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

  auto step = [&](auto bufc, int tile) {
    constexpr int BUF = decltype(bufc)::value;
    const uint16_t *kb = (BUF ? sk1 : sk0) + group * kStage;
    uint16_t *vb = (BUF ? sv1 : sv0) + group * kStage;
    const bool mine = GR == 1 || tile < tiles, active = mine && wave * 32 < it.rows;
    const int t0 = first + tile * kTilePos;
    bool whole = !mine || (exist[BUF] == ~0ull && hi_all >= t0 + (kTilePos - 1) && lo_all <= t0);
    if (GR > 1 && wave == 0 && lane == 0) masked[BUF][group] = !whole;
    wait_vm<0>();     // this wave's loads of the tile have landed
    __syncthreads();  // everybody's have, and nobody reads the other stage any more
    if constexpr (GR > 1) whole = (masked[BUF][0] | masked[BUF][GR - 1]) == 0;  // the groups mask together: there are barriers
    if (tile + GR < tiles) {
      exist[1 - BUF] = issue(std::integral_constant<int, 1 - BUF>{}, tile + GR, page);
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
          });
      if (!whole) {
        keep = 0;
#pragma unroll
        for (int b = 0; b < SB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = 32 * b + 8 * (i / 4) + 4 * hf + i % 4, p = t0 + r;
            const bool ok = p <= hi && p >= lo && (exist[BUF] >> r & 1);
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

// ----------------------------------------------------------------- join
// An item's parts, each weighted with 2^(lse_part - lse).  The weights first, in LDS; then a thread adds 8 columns
// of a row over a slice of the parts, and the slices are added in order.  As many slices as the
// threads allow: one thread going through all the parts of its columns would wait for each of them
// in turn (64 / 8 heads of 128, one token over 8192 positions in 32 parts: 41 us in all, so 18).
constexpr int kJoinThreads = 1024;

__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(Args a) {
  __shared__ float sw[LORA_ATTN_MAX_PARTS * LORA_ATTN_TILE_ROWS], slse[LORA_ATTN_TILE_ROWS];
  __shared__ __attribute__((aligned(16))) f32x4_t sv[2][kJoinThreads];
  const lora_kv_view &kv = a.kv;
  const int h = blockIdx.x % kv.kv_heads, ii = blockIdx.x / kv.kv_heads;
  lora_attn_item it = a.items[ii];
  const int parts = it.part, base = it.kv_begin;
  it.part = -1;
  it.kv_begin = 0;  // kv_end stays: a join past the view has parts that were skipped
  if (!good_item(a, it, LORA_ATTN_TILE_ROWS) || parts < 1 || parts > LORA_ATTN_MAX_PARTS || base < 0 ||
      base + (int64_t)parts * it.rows > a.num_part_rows) {
    KV_CHECK(threadIdx.x != 0, LORA_DEBUG_BAD_ITEM);
    return;
  }
  const int D = kv.head_dim, nch = D >> 3, units = it.rows * nch;
  // a wave per row, a lane per part
  constexpr int kWaves = kJoinThreads / 64, kTurns = LORA_ATTN_TILE_ROWS / kWaves;
  static_assert(LORA_ATTN_MAX_PARTS <= 64 && kTurns * kWaves == LORA_ATTN_TILE_ROWS);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float lp[kTurns];
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const int r = wave + t * kWaves;
    lp[t] = r < it.rows && lane < parts ? a.part_lse[(int64_t)(base + lane * it.rows + r) * kv.kv_heads + h] : -INFINITY;
  }
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    const int r = wave + t * kWaves;
    if (r >= it.rows) break;
    float top = lp[t];
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float f = lp[t] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(lp[t] - top);  // the range kept nothing: no weight
    float total = f;
    for (int x = 1; x < 64; x <<= 1) total += __shfl_xor(total, x);
    if (lane < parts) sw[lane * it.rows + r] = total == 0.f ? 0.f : f / total;
    if (lane == 0) slse[r] = total == 0.f ? -INFINITY : top + log2f(total);
  }
  __syncthreads();
  const int slices = max(1, min(parts, kJoinThreads / units)), per = (parts + slices - 1) / slices;
  // with one slice several turns, else the threads behind the last slice have none
  for (int i0 = 0; i0 < units; i0 += slices > 1 ? units : kJoinThreads) {
    const int slice = slices > 1 ? (int)threadIdx.x / units : 0, i = slices > 1 ? (int)threadIdx.x % units : i0 + (int)threadIdx.x;
    const int r = i / nch, c = i % nch;
    f32x4_t v[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
    if (slice < slices && i < units) {
#pragma unroll 4
      for (int p = slice * per; p < min(parts, (slice + 1) * per); ++p) {
        const float f = sw[p * it.rows + r];
        const f32x4_t *po = reinterpret_cast<const f32x4_t *>(a.part_o + ((int64_t)(base + p * it.rows + r) * kv.kv_heads + h) * D + 8 * c);
        v[0] += f * po[0];
        v[1] += f * po[1];
      }
    }
    if (slices > 1) {
      sv[0][threadIdx.x] = v[0];
      sv[1][threadIdx.x] = v[1];
      __syncthreads();
      if (slice == 0)
        for (int w = 1; w < slices; ++w) {
          v[0] += sv[0][w * units + i];
          v[1] += sv[1][w * units + i];
        }
    }
    if (slice > 0 || i >= units) continue;
    const int rr = it.row0 + r, tk = rr / a.group, hd = h * a.group + rr % a.group;
    *reinterpret_cast<uint4 *>(a.out + (it.q_begin + tk) * a.o_ts + hd * a.o_hs + 8 * c) =
        make_uint4(pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3]), pack_bf16(v[1][0], v[1][1]), pack_bf16(v[1][2], v[1][3]));
    if (c == 0 && a.lse) a.lse[(int64_t)(it.q_begin + tk) * a.q_heads + hd] = slse[r] * kLn2;
  }
}

constexpr unsigned kComputeUnits = 256;

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Heads of 64, 128 and 256, the usual ones, have kernels without the checks that shorter rows need (chunks of 64
// over 512 positions, 12 heads of 64: 12.8 us, with the checks 13.8; 8 chunks of 128 over 4096: 171 and 178).
template <int DP>
constexpr bool kFull = DP == 64 || DP == 128 || DP == 256;
template <int DP>
bool full(const Args &a) { return kFull<DP> && a.kv.head_dim == DP; }

template <int DP>
void launch_rows(const Args &a, unsigned grid, hipStream_t stream) {
  // two workgroups of half the waves share a compute unit's LDS and overlap their ends; a grid that gives
  // every compute unit one at most takes all the waves at once, for a shorter chain of tiles (heads of 128, 4 tokens
  // over 300 positions: 10.2 us, with half the waves 11.2; 8 tokens over 2048, 512 units: 32 us and 26)
  constexpr int W = DP <= 64 ? 4 : DP <= 128 ? 2 : 1;
  const auto wide = full<DP>(a) ? attn_rows_kernel<DP, 2 * W, kFull<DP>> : attn_rows_kernel<DP, 2 * W, false>;
  const auto slim = full<DP>(a) ? attn_rows_kernel<DP, W, kFull<DP>> : attn_rows_kernel<DP, W, false>;
  if (grid <= kComputeUnits) hipLaunchKernelGGL(wide, dim3(grid), dim3(128 * W), 0, stream, a);
  else hipLaunchKernelGGL(slim, dim3(grid), dim3(64 * W), 0, stream, a);
}

template <int DP>
void launch_tiles(const Args &a, unsigned grid, hipStream_t stream) {
  // a grid of one workgroup per compute unit at most takes two groups of waves (4 chunks of 64 over 512 positions, 12
  // heads of 64: 12.8 us, with one group 13.9; 40 such chunks, 480 units: 86 us and 20)
  constexpr int G2 = DP <= 128 ? 2 : 1;  // what the LDS holds
  const auto one = full<DP>(a) ? attn_tile_kernel<DP, kFull<DP>, 1> : attn_tile_kernel<DP, false, 1>;
  const auto two = full<DP>(a) ? attn_tile_kernel<DP, kFull<DP>, G2> : attn_tile_kernel<DP, false, G2>;
  if (grid <= kComputeUnits) hipLaunchKernelGGL(two, dim3(grid), dim3(64 * kTileWaves * G2), 0, stream, a);
  else hipLaunchKernelGGL(one, dim3(grid), dim3(64 * kTileWaves), 0, stream, a);
}

}  // namespace

lora_status lora::kv_attn_debug(uint32_t *flags, int32_t clear) { return kv_debug_word(flags, clear); }

extern "C" lora_status lora_kv_attn(const lora_kv_view *kv, const lora_attn_plan *plan, const lora_attn_item *items,
                                    const void *q, int64_t q_token_stride, int64_t q_head_stride, void *out,
                                    int64_t out_token_stride, int64_t out_head_stride, float *lse, float scale,
                                    void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  lora_status st = check_view(kv);
  if (st != LORA_OK) return st;
  if (!plan) return fail(LORA_EINVAL, "null plan");
  if (plan->kv_heads != kv->kv_heads || plan->head_dim != kv->head_dim)
    return fail(LORA_EINVAL, "the plan is for %d KV heads of %d, the cache holds %d of %d", plan->kv_heads,
                plan->head_dim, kv->kv_heads, kv->head_dim);
  if (plan->q_heads < 1 || plan->q_heads % plan->kv_heads || plan->num_tokens < 0 || plan->num_row_items < 0 ||
      plan->num_tile_items < 0 || plan->num_joins < 0 || plan->num_part_rows < 0 || plan->window < 0 ||
      (plan->flags & ~LORA_ATTN_CAUSAL))
    return fail(LORA_EINVAL, "not a plan");
  const int64_t strides[4] = {q_token_stride, q_head_stride, out_token_stride, out_head_stride};
  for (int64_t s : strides)
    if (s < 0 || s % 8) return fail(LORA_EINVAL, "strides of q and out must be multiples of 8 elements, not negative");
  if (kv->page_stride / 8 > UINT32_MAX || kv->token_stride / 8 > UINT32_MAX)
    return fail(LORA_EUNSUPPORTED, "KV strides of 2^35 elements and more");
  if (!std::isfinite(scale)) return fail(LORA_EINVAL, "scale is not finite");
  const int64_t part_floats = (int64_t)plan->num_part_rows * kv->kv_heads * kv->head_dim;
  const int64_t need = plan->num_part_rows * (int64_t)kv->kv_heads * (kv->head_dim + 4) * (int64_t)sizeof(float);
  if (workspace_bytes < need || (need > 0 && (!workspace || !aligned16(workspace))))
    return fail(LORA_EINVAL, "workspace of %lld bytes, 16-byte aligned, needed (got %lld)", (long long)need,
                (long long)workspace_bytes);
  const int64_t all = (int64_t)plan->num_row_items + plan->num_tile_items + plan->num_joins;
  if (all * kv->kv_heads > INT32_MAX) return fail(LORA_EINVAL, "not a plan");
  // row and tile items have at most 256 threads where their grid is large
  if (too_many((int64_t)plan->num_row_items * kv->kv_heads, 256) || too_many((int64_t)plan->num_tile_items * kv->kv_heads, 256) ||
      too_many((int64_t)plan->num_joins * kv->kv_heads, kJoinThreads))
    return fail(LORA_EUNSUPPORTED, "too many items for one launch");
  if (plan->num_tokens == 0 || all == 0) return ok();
  if (!items || !q || !out) return fail(LORA_EINVAL, "null pointer");
  if (!aligned16(items) || !aligned16(q) || !aligned16(out) || ((uintptr_t)lse & 3))
    return fail(LORA_EINVAL, "q, out and items must be 16-byte aligned");
  Args a{};
  a.kv = *kv;
  a.q = (const uint16_t *)q;
  a.out = (uint16_t *)out;
  a.lse = lse;
  a.part_o = (float *)workspace;
  a.part_lse = (float *)workspace + part_floats;
  a.q_ts = q_token_stride;
  a.q_hs = q_head_stride;
  a.o_ts = out_token_stride;
  a.o_hs = out_head_stride;
  a.page_div = Div((uint32_t)kv->page_tokens);
  a.page16 = (uint32_t)(kv->page_stride / 8);
  a.token16 = (uint32_t)(kv->token_stride / 8);
  a.scale2 = scale == 0.f ? 1.f : std::fabs(scale) * kLog2e;
  a.q_and = scale == 0.f ? 0u : ~0u;
  a.q_xor = scale < 0.f ? 0x80008000u : 0u;
  a.q_heads = plan->q_heads;
  a.group = plan->q_heads / plan->kv_heads;
  a.causal = plan->flags & LORA_ATTN_CAUSAL;
  a.window = plan->window;
  a.num_tokens = plan->num_tokens;
  a.num_part_rows = plan->num_part_rows;
  const int dp = (kv->head_dim + 31) / 32 * 32;
  if (plan->num_row_items) {
    a.items = items;
    const unsigned grid = (unsigned)(plan->num_row_items * kv->kv_heads);
    if (dp <= 64) launch_rows<64>(a, grid, stream);
    else if (dp <= 96) launch_rows<96>(a, grid, stream);
    else if (dp <= 128) launch_rows<128>(a, grid, stream);
    else if (dp <= 192) launch_rows<192>(a, grid, stream);
    else launch_rows<256>(a, grid, stream);
  }
  if (plan->num_tile_items) {
    a.items = items + plan->num_row_items;
    const unsigned grid = (unsigned)(plan->num_tile_items * kv->kv_heads);
    if (dp <= 64) launch_tiles<64>(a, grid, stream);
    else if (dp <= 96) launch_tiles<96>(a, grid, stream);
    else if (dp <= 128) launch_tiles<128>(a, grid, stream);
    else if (dp <= 192) launch_tiles<192>(a, grid, stream);
    else launch_tiles<256>(a, grid, stream);
  }
  if (plan->num_joins) {
    a.items = items + plan->num_row_items + plan->num_tile_items;
    hipLaunchKernelGGL(attn_join_kernel, dim3((unsigned)(plan->num_joins * kv->kv_heads)), dim3(kJoinThreads), 0,
                       stream, a);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, "attention launch");
}
