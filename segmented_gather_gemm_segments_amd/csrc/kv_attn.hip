// Attention of new tokens over the paged KV cache (lora_kv.h, lora_tree.h, lora_blocks.h): the kernels over bf16
// rows with a causal mask, the join of ranges, and the entry points.
#include "kv_attn.h"

#include "lora_blocks.h"
#include "lora_tree.h"

namespace {

// ----------------------------------------------------------------- join
// An item's parts, each weighted with 2^(lse_part - lse).  The weights first, in LDS; then a thread adds 8 columns
// of a row over a slice of the parts, and the slices are added in order.  As many slices as the
// threads allow: one thread going through all the parts of its columns would wait for each of them
// in turn (64 / 8 heads of 128, one token over 8192 positions in 32 parts: 41 us in all, so 18).
constexpr int kJoinThreads = 1024;

template <Mask M>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(ArgsOf<false, M> a) {
  __shared__ float sw[LORA_ATTN_MAX_PARTS * LORA_ATTN_TILE_ROWS], slse[LORA_ATTN_TILE_ROWS];
  __shared__ __attribute__((aligned(16))) f32x4_t sv[2][kJoinThreads];
  const lora_kv_view &kv = a.kv;
  const int h = blockIdx.x % kv.kv_heads, ii = blockIdx.x / kv.kv_heads;
  lora_attn_item it = a.items[ii];
  const int parts = it.part, base = it.kv_begin;
  it.part = -1;
  it.kv_begin = 0;  // kv_end stays: a join past the view has parts that were skipped
  if (!good_item<M>(a, it, LORA_ATTN_TILE_ROWS) || parts < 1 || parts > LORA_ATTN_MAX_PARTS || base < 0 ||
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

}  // namespace

lora_status lora::kv_attn_debug(uint32_t *flags, int32_t clear) { return kv_debug_word(flags, clear); }

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// A call of any of the three entry points: exactly the mask of its own kind is given, and the plan's flags say the same.
struct Call {
  const lora_kv_view *kv;
  const lora_attn_plan *plan;
  const lora_attn_item *items;
  const void *q;
  int64_t q_token_stride, q_head_stride;
  void *out;
  int64_t out_token_stride, out_head_stride;
  float *lse;
  float scale;
  void *workspace;
  int64_t workspace_bytes;
  hipStream_t stream;
};

lora_status run(const Call &c, Mask mask, AttnMoreArgs a) {
  const lora_kv_view *kv = c.kv;
  const lora_attn_plan *plan = c.plan;
  if (plan->kv_heads != kv->kv_heads || plan->head_dim != kv->head_dim)
    return fail(LORA_EINVAL, "the plan is for %d KV heads of %d, the cache holds %d of %d", plan->kv_heads,
                plan->head_dim, kv->kv_heads, kv->head_dim);
  if (plan->q_heads < 1 || plan->q_heads % plan->kv_heads || plan->num_tokens < 0 || plan->num_row_items < 0 ||
      plan->num_tile_items < 0 || plan->num_joins < 0 || plan->num_part_rows < 0 || plan->window < 0 ||
      (plan->flags & ~LORA_ATTN_CAUSAL) != (mask == Mask::kTree ? LORA_ATTN_TREE : mask == Mask::kBlocks ? LORA_ATTN_BLOCKS : 0) ||
      (mask == Mask::kBlocks && (plan->flags != LORA_ATTN_BLOCKS || plan->window || plan->num_tile_items)))
    return fail(LORA_EINVAL, "not a plan for this call");
  const int64_t strides[4] = {c.q_token_stride, c.q_head_stride, c.out_token_stride, c.out_head_stride};
  for (int64_t s : strides)
    if (s < 0 || s % 8) return fail(LORA_EINVAL, "strides of q and out must be multiples of 8 elements, not negative");
  const bool f8 = kv->dtype == LORA_FP8_E4M3;
  const int64_t unit = f8 ? 16 : 8;  // elements in 16 bytes
  if (kv->page_stride / unit > UINT32_MAX || kv->token_stride / unit > UINT32_MAX)
    return fail(LORA_EUNSUPPORTED, "KV strides of 2^35 elements (8-bit: 2^36) and more");
  if (!std::isfinite(c.scale)) return fail(LORA_EINVAL, "scale is not finite");
  const int64_t part_floats = (int64_t)plan->num_part_rows * kv->kv_heads * kv->head_dim;
  const int64_t need = plan->num_part_rows * (int64_t)kv->kv_heads * (kv->head_dim + 4) * (int64_t)sizeof(float);
  if (c.workspace_bytes < need || (need > 0 && (!c.workspace || !aligned16(c.workspace))))
    return fail(LORA_EINVAL, "workspace of %lld bytes, 16-byte aligned, needed (got %lld)", (long long)need,
                (long long)c.workspace_bytes);
  const int64_t all = (int64_t)plan->num_row_items + plan->num_tile_items + plan->num_joins;
  if (all * kv->kv_heads > INT32_MAX) return fail(LORA_EINVAL, "not a plan");
  // row and tile items have at most 256 threads where their grid is large
  if (too_many((int64_t)plan->num_row_items * kv->kv_heads, 256) || too_many((int64_t)plan->num_tile_items * kv->kv_heads, 256) ||
      too_many((int64_t)plan->num_joins * kv->kv_heads, kJoinThreads))
    return fail(LORA_EUNSUPPORTED, "too many items for one launch");
  if (plan->num_tokens == 0 || all == 0) return ok();
  if (!c.items || !c.q || !c.out) return fail(LORA_EINVAL, "null pointer");
  if (!aligned16(c.items) || !aligned16(c.q) || !aligned16(c.out) || ((uintptr_t)c.lse & 3))
    return fail(LORA_EINVAL, "q, out and items must be 16-byte aligned");
  a.kv = *kv;
  a.items = c.items;
  a.q = (const uint16_t *)c.q;
  a.out = (uint16_t *)c.out;
  a.lse = c.lse;
  a.part_o = (float *)c.workspace;
  a.part_lse = (float *)c.workspace + part_floats;
  a.q_ts = c.q_token_stride;
  a.q_hs = c.q_head_stride;
  a.o_ts = c.out_token_stride;
  a.o_hs = c.out_head_stride;
  a.page_div = Div((uint32_t)kv->page_tokens);
  a.page16 = (uint32_t)(kv->page_stride / unit);
  a.token16 = (uint32_t)(kv->token_stride / unit);
  if (f8) {
    const lora_kv8_view *kv8 = reinterpret_cast<const lora_kv8_view *>(kv);
    if (kv8->scale_page_stride > UINT32_MAX || kv8->scale_token_stride > UINT32_MAX)
      return fail(LORA_EUNSUPPORTED, "strides of scales of 2^32 bytes and more");
    a.k_scales = kv8->k_scales;
    a.v_scales = kv8->v_scales;
    a.scale_ps = (uint32_t)kv8->scale_page_stride;
    a.scale_hs = kv8->scale_head_stride;
    a.scale_ts = (uint32_t)kv8->scale_token_stride;
  }
  a.scale2 = c.scale == 0.f ? 1.f : std::fabs(c.scale) * kLog2e;
  a.q_and = c.scale == 0.f ? 0u : ~0u;
  a.q_xor = c.scale < 0.f ? 0x80008000u : 0u;
  a.q_heads = plan->q_heads;
  a.group = plan->q_heads / plan->kv_heads;
  a.causal = plan->flags & LORA_ATTN_CAUSAL;
  a.window = plan->window;
  a.num_tokens = plan->num_tokens;
  a.num_part_rows = plan->num_part_rows;
  if (mask == Mask::kTree) (f8 ? attn8_items_tree : attn_items_tree)(a, *plan, c.stream);
  else if (mask == Mask::kBlocks) (f8 ? attn8_items_blocks : attn_items_blocks)(a, *plan, c.stream);
  else if (f8) attn8_items(a, *plan, c.stream);
  else launch_items<false, Mask::kCausal>(a, *plan, c.stream);
  if (plan->num_joins) {
    a.items = c.items + plan->num_row_items + plan->num_tile_items;
    const dim3 grid((unsigned)(plan->num_joins * kv->kv_heads));
    if (mask == Mask::kBlocks) hipLaunchKernelGGL(attn_join_kernel<Mask::kBlocks>, grid, dim3(kJoinThreads), 0, c.stream, a);
    else hipLaunchKernelGGL(attn_join_kernel<Mask::kCausal>, grid, dim3(kJoinThreads), 0, c.stream, a);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, "attention launch");
}

lora_status check(const Call &c) {
  const lora_status st = check_view(c.kv);
  return st != LORA_OK ? st : c.plan ? LORA_OK : fail(LORA_EINVAL, "null plan");
}

}  // namespace

extern "C" lora_status lora_kv_attn(const lora_kv_view *kv, const lora_attn_plan *plan, const lora_attn_item *items,
                                    const void *q, int64_t q_token_stride, int64_t q_head_stride, void *out,
                                    int64_t out_token_stride, int64_t out_head_stride, float *lse, float scale,
                                    void *workspace, int64_t workspace_bytes, hipStream_t stream) {
  const Call c = {kv, plan, items, q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse,
                  scale, workspace, workspace_bytes, stream};
  const lora_status st = check(c);
  return st != LORA_OK ? st : run(c, Mask::kCausal, AttnMoreArgs{});
}

extern "C" lora_status lora_kv_attn_tree(const lora_kv_view *kv, const lora_attn_plan *plan, const lora_attn_item *items,
                                         const lora_tree *tree, const void *q, int64_t q_token_stride,
                                         int64_t q_head_stride, void *out, int64_t out_token_stride,
                                         int64_t out_head_stride, float *lse, float scale, void *workspace,
                                         int64_t workspace_bytes, hipStream_t stream) {
  const Call c = {kv, plan, items, q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse,
                  scale, workspace, workspace_bytes, stream};
  lora_status st = check(c);
  if (st == LORA_OK) st = check_tree(tree);
  if (st != LORA_OK) return st;
  if (tree->num_tokens < plan->num_tokens)
    return fail(LORA_EINVAL, "a tree of %d tokens for a plan of %d", tree->num_tokens, plan->num_tokens);
  AttnMoreArgs a{};
  a.tree_mask = tree->mask;
  a.tree_depth = tree->depth;
  a.tree_words = tree->words;
  return run(c, Mask::kTree, a);
}

extern "C" lora_status lora_kv_attn_blocks(const lora_kv_view *kv, const lora_attn_plan *plan,
                                           const lora_attn_item *items, const int32_t *blocks, int32_t count,
                                           const int32_t *token_pos, const void *q, int64_t q_token_stride,
                                           int64_t q_head_stride, void *out, int64_t out_token_stride,
                                           int64_t out_head_stride, float *lse, float scale, void *workspace,
                                           int64_t workspace_bytes, hipStream_t stream) {
  const Call c = {kv, plan, items, q, q_token_stride, q_head_stride, out, out_token_stride, out_head_stride, lse,
                  scale, workspace, workspace_bytes, stream};
  const lora_status st = check(c);
  if (st != LORA_OK) return st;
  if (count < 1 || count > LORA_BLOCKS_MAX_COUNT)
    return fail(LORA_EUNSUPPORTED, "lists of %d pages, not 1..%d", count, LORA_BLOCKS_MAX_COUNT);
  if ((int64_t)count * kv->page_tokens > INT32_MAX) return fail(LORA_EUNSUPPORTED, "lists of more than 2^31 - 1 positions");
  if (plan->num_tokens > 0 && (!blocks || !token_pos)) return fail(LORA_EINVAL, "null pointer");
  if (((uintptr_t)blocks & 3) || ((uintptr_t)token_pos & 3)) return fail(LORA_EINVAL, "blocks and token_pos must be 4-byte aligned");
  AttnMoreArgs a{};
  a.blocks = blocks;
  a.count = count;
  a.token_pos = token_pos;
  return run(c, Mask::kBlocks, a);
}
