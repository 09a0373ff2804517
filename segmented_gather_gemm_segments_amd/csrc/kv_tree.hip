// Trees of drafted tokens over the paged KV cache (lora_tree.h): their masks, and the accepted path's rows moved.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kv_internal.h"
#include "kv_debug.h"
#include "kv_rows.h"

using namespace lora;

namespace {

constexpr int kThreads = 256;

// A workgroup per request, a thread per node: it walks up to the context through the parents in LDS.  Ancestors come in
// falling order, so the words of its mask do too, and each is written once.
__global__ __launch_bounds__(kThreads) void tree_mask_kernel(const int32_t *__restrict__ q_starts,
                                                             const int32_t *__restrict__ parent, int window, lora_tree tree) {
  __shared__ int up[LORA_TREE_MAX_NODES];
  const int begin = q_starts[blockIdx.x], end = q_starts[blockIdx.x + 1], n = end - begin;
  const bool good = begin >= 0 && end >= begin && end <= tree.num_tokens && n <= 64 * tree.words;
  KV_CHECK(good || threadIdx.x != 0, LORA_DEBUG_BAD_TOKEN);
  if (!good) return;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int p = parent[begin + i];
    KV_CHECK(p >= -1 && p < i, LORA_DEBUG_BAD_TOKEN);
    up[i] = p >= -1 && p < i ? p : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    uint64_t *row = tree.mask + (int64_t)(begin + i) * tree.words;
    int depth = 0, w = i >> 6;
    uint64_t bits = 0;
    for (int x = w + 1; x < tree.words; ++x) row[x] = 0;
    for (int a = i;; ++depth) {
      if (window == 0 || depth < window) {
        for (; w > a >> 6; --w) {
          row[w] = bits;
          bits = 0;
        }
        bits |= 1ull << (a & 63);
      }
      a = up[a];
      if (a < 0) break;
    }
    for (; w >= 0; --w) {
      row[w] = bits;
      bits = 0;
    }
    tree.depth[begin + i] = depth;
  }
}

// A thread moves one piece (16 bytes of a row, or a scale byte) of every row of its request's path, in the path's order.
// Entries ascend, so path[i] >= i: what position base + i receives is never read later, only by copies before it, and
// pieces of kAhead entries may be read before the first of them is written.
constexpr int kAhead = 8;

template <typename T>
__device__ __forceinline__ void move_piece(const lora_kv_view &kv, int s, int base, const int32_t *path, int max_path, T *store,
                                           int64_t page_stride, int64_t token_stride) {
  int before = -1;
  for (int i0 = 0; i0 < max_path; i0 += kAhead) {
    T piece[kAhead];
    int64_t to[kAhead];
    bool more = true;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int e = more && i0 + j < max_path ? path[i0 + j] : -1;
      KV_CHECK(e < 0 || e > before, LORA_DEBUG_BAD_TOKEN);
      more = e > before && e >= 0;
      to[j] = -1;
      if (more) {
        before = e;
        const int64_t src = (int64_t)base + e, dst = (int64_t)base + i0 + j;
        if (src != dst) {
          const Place a = place_of(kv, s, (int)min(src, (int64_t)INT32_MAX)), b = place_of(kv, s, (int)min(dst, (int64_t)INT32_MAX));
          if (a.page >= 0 && b.page >= 0) {
            piece[j] = store[a.page * page_stride + a.slot * token_stride];
            to[j] = b.page * page_stride + b.slot * token_stride;
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (to[j] >= 0) store[to[j]] = piece[j];
    if (!more) return;
  }
}

__global__ __launch_bounds__(kThreads) void keep_path_kernel(lora_kv8_view v, const int32_t *__restrict__ seq,
                                                             const int32_t *__restrict__ bases,
                                                             const int32_t *__restrict__ path, int max_path, int chunks,
                                                             int size, int units, int groups) {
  const lora_kv_view &kv = v.kv;
  const int r = blockIdx.x / groups, u = (int)(blockIdx.x % groups) * kThreads + (int)threadIdx.x;
  if (u >= units) return;
  const int s = seq[r], base = bases[r];
  KV_CHECK(s < kv.num_seqs && (s < 0 || base >= 0), LORA_DEBUG_BAD_TOKEN);
  if (s < 0 || s >= kv.num_seqs || base < 0) return;
  const int rows = 2 * kv.kv_heads;  // of K, then of V
  path += (int64_t)r * max_path;
  if (u < rows * chunks) {
    const int row = u / chunks, c = u % chunks, h = row % kv.kv_heads;
    uint4 *store = (uint4 *)((char *)(row < kv.kv_heads ? kv.k : kv.v) + (int64_t)h * kv.head_stride * size) + c;
    move_piece(kv, s, base, path, max_path, store, kv.page_stride * size / 16, kv.token_stride * size / 16);
  } else {
    const int row = u - rows * chunks, h = row % kv.kv_heads;
    uint8_t *store = (row < kv.kv_heads ? v.k_scales : v.v_scales) + (int64_t)h * v.scale_head_stride;
    move_piece(kv, s, base, path, max_path, store, v.scale_page_stride, v.scale_token_stride);
  }
}

}  // namespace

lora_status lora::kv_tree_debug(uint32_t *flags, int32_t clear) { return kv_debug_word(flags, clear); }

lora_status lora::check_tree(const lora_tree *tree) {
  if (!tree) return fail(LORA_EINVAL, "null tree");
  if (tree->num_tokens < 0) return fail(LORA_EINVAL, "a tree of %d tokens", tree->num_tokens);
  if (tree->words < 1 || tree->words > LORA_TREE_MAX_NODES / 64)
    return fail(LORA_EUNSUPPORTED, "%d words for each node's mask, not 1..%d", tree->words, LORA_TREE_MAX_NODES / 64);
  if (tree->num_tokens > 0 && (!tree->mask || !tree->depth)) return fail(LORA_EINVAL, "null mask or depth");
  if (((uintptr_t)tree->mask & 7) || ((uintptr_t)tree->depth & 3))
    return fail(LORA_EINVAL, "masks must be 8-byte aligned, depths 4-byte");
  return LORA_OK;
}

extern "C" lora_status lora_tree_mask(const int32_t *q_starts, int32_t num_reqs, const int32_t *parent, int32_t window,
                                      const lora_tree *tree, hipStream_t stream) {
  const lora_status st = check_tree(tree);
  if (st != LORA_OK) return st;
  if (num_reqs < 0 || window < 0) return fail(LORA_EINVAL, "%d requests, window %d", num_reqs, window);
  if (num_reqs >= 1 << 24) return fail(LORA_EUNSUPPORTED, "%d requests", num_reqs);
  if (num_reqs == 0 || tree->num_tokens == 0) return ok();
  if (!q_starts || !parent) return fail(LORA_EINVAL, "null pointer");
  if (((uintptr_t)q_starts & 3) || ((uintptr_t)parent & 3)) return fail(LORA_EINVAL, "q_starts and parent must be 4-byte aligned");
  hipLaunchKernelGGL(tree_mask_kernel, dim3((unsigned)num_reqs), dim3(kThreads), 0, stream, q_starts, parent, window, *tree);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, "tree mask launch");
}

extern "C" lora_status lora_kv_keep_path(const lora_kv_view *kv, const int32_t *seq, const int32_t *base,
                                         const int32_t *path, int32_t num_reqs, int32_t max_path, hipStream_t stream) {
  const lora_status st = check_view(kv);
  if (st != LORA_OK) return st;
  if (num_reqs < 0 || max_path < 0) return fail(LORA_EINVAL, "%d requests, paths of %d", num_reqs, max_path);
  if (num_reqs == 0 || max_path == 0 || kv->num_pages == 0 || kv->num_seqs == 0 || kv->max_pages == 0) return ok();
  if (!seq || !base || !path) return fail(LORA_EINVAL, "null pointer");
  if (((uintptr_t)seq & 3) || ((uintptr_t)base & 3) || ((uintptr_t)path & 3))
    return fail(LORA_EINVAL, "seq, base and path must be 4-byte aligned");
  const bool f8 = kv->dtype == LORA_FP8_E4M3;
  const int size = f8 ? 1 : 2, chunks = kv->head_dim * size / 16;
  const int64_t units = 2 * (int64_t)kv->kv_heads * (chunks + (f8 ? 1 : 0)), groups = (units + kThreads - 1) / kThreads;
  if (groups * num_reqs >= 1 << 24) return fail(LORA_EUNSUPPORTED, "paths too many for one launch");
  hipLaunchKernelGGL(keep_path_kernel, dim3((unsigned)(groups * num_reqs)), dim3(kThreads), 0, stream, view8(kv), seq, base,
                     path, max_path, chunks, size, (int)units, (int)groups);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, "path launch");
}
