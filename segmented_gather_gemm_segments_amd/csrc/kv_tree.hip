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
// falling order, so the words of its mask do too, and each is written once.  Bound by its chain of loads: one tree of 26
// nodes 2.1 us, 32 of up to 61 5.8 us; a thread's walk in LDS is as long as the tree is deep.
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
//
// A wave looks up 64 entries' places side by side (path, then two page ids: a chain of two loads for
// all of them) into LDS.  Paths of up to 8 in 128 trees, 64 heads of 128 in 8 bits, 34 MB: 9.8 us; of 5 in one tree, 8 heads
// in bf16: 4.4 us, the chain of seq, path, page and row.  A place looked up by each thread for itself, entry by entry, took 17.
constexpr int kAhead = 8;  // divides 64
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

__device__ const u32x4_t g_zeros = {0, 0, 0, 0};

// Pieces of entries [0, n) of up to 64; to[j].page < 0: not copied (and zeros read, so that no load waits for a branch).
template <typename T>
__device__ __forceinline__ void move_pieces(T *store, int64_t page_stride, int64_t token_stride, const Place *from,
                                            const Place *to, int n) {
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    T piece[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const Place x = from[j0 + j];
      const T *at = store + (x.page * page_stride + x.slot * token_stride);
      piece[j] = *(j0 + j < n && to[j0 + j].page >= 0 ? at : reinterpret_cast<const T *>(&g_zeros));
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const Place x = to[j0 + j];
      if (j0 + j < n && x.page >= 0) store[x.page * page_stride + x.slot * token_stride] = piece[j];
    }
  }
}

__global__ __launch_bounds__(kThreads) void keep_path_kernel(lora_kv8_view v, const int32_t *__restrict__ seq,
                                                             const int32_t *__restrict__ bases,
                                                             const int32_t *__restrict__ path, int max_path, int chunks,
                                                             int size, int units, int groups) {
  __shared__ Place from[64], to[64];
  __shared__ int count, last;
  const lora_kv_view &kv = v.kv;
  const int r = blockIdx.x / groups, u = (int)(blockIdx.x % groups) * kThreads + (int)threadIdx.x;
  const int s = seq[r], base = bases[r], lane = threadIdx.x;
  KV_CHECK(s < kv.num_seqs && (s < 0 || base >= 0), LORA_DEBUG_BAD_TOKEN);
  if (s < 0 || s >= kv.num_seqs || base < 0) return;
  const int rows = 2 * kv.kv_heads;  // of K, then of V
  // this thread's piece of a row, or its scale byte
  const bool piece = u < rows * chunks, scale = !piece && u < units;
  const int row = piece ? u / chunks : scale ? u - rows * chunks : 0, h = row % kv.kv_heads;
  const bool is_v = row >= kv.kv_heads;
  u32x4_t *store = (u32x4_t *)((char *)(is_v ? kv.v : kv.k) + (int64_t)h * kv.head_stride * size) + (piece ? u % chunks : 0);
  uint8_t *scales = (is_v ? v.v_scales : v.k_scales) + (int64_t)h * v.scale_head_stride;
  path += (int64_t)r * max_path;
  for (int i0 = 0; i0 < max_path; i0 += 64) {
    if (lane < 64) {
      const int e = i0 + lane < max_path ? path[i0 + lane] : -1;
      const int prev = lane ? __shfl_up(e, 1) : i0 ? last : -1;
      const uint64_t stop = __ballot(e <= prev || e < 0);
      const int n = stop ? __builtin_ctzll(stop) : 64;
      KV_CHECK(lane != n || e < 0, LORA_DEBUG_BAD_TOKEN);
      Place a = {-1, 0}, b = {-1, 0};
      if (lane < n && e != i0 + lane) {  // not where it stands already
        a = place_of(kv, s, (int)min((int64_t)base + e, (int64_t)INT32_MAX));
        b = place_of(kv, s, (int)min((int64_t)base + i0 + lane, (int64_t)INT32_MAX));
      }
      if (a.page < 0) b.page = -1;
      from[lane] = a;
      to[lane] = b;
      if (lane == 63) last = e;
      if (lane == 0) count = n;
    }
    __syncthreads();
    const int n = count;
    if (piece) move_pieces(store, kv.page_stride * size / 16, kv.token_stride * size / 16, from, to, n);
    else if (scale) move_pieces(scales, v.scale_page_stride, v.scale_token_stride, from, to, n);
    if (n < 64) return;
    __syncthreads();
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
  if (groups * num_reqs >= 1 << 24 || units > INT32_MAX) return fail(LORA_EUNSUPPORTED, "paths too many for one launch");
  hipLaunchKernelGGL(keep_path_kernel, dim3((unsigned)(groups * num_reqs)), dim3(kThreads), 0, stream, view8(kv), seq, base,
                     path, max_path, chunks, size, (int)units, (int)groups);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, "path launch");
}
