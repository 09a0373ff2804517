// Paged KV cache: page copies, page-table rewrites and the append of new tokens'
// rows (lora_kv.h), and the device steps of the sequence bookkeeping.
//
// All of it moves bytes, each read once and written once, in 16-byte units; HBM bounds
// the large calls, the launch the small ones.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "kv_internal.h"
#include "kv_debug.h"

using namespace lora;

namespace {

constexpr int kThreads = 256;
// One unit of 16 bytes per thread.  Two take 204 us for 2048 pages of 256 KiB, one 180 us (5.9 TB/s); loads and
// stores past the caches 170 us there, but 24 us for 1024 pages of 64 KiB, which the last cache holds, and
// these 17.6 us.
constexpr int kSliceBytes = 16 * kThreads;  // of a page, per workgroup
static_assert(kKvMaxPageBytes / kSliceBytes <= UINT32_MAX / kThreads);

// Copies bytes [slice * kSliceBytes, ..) of one page.
__device__ __forceinline__ void copy_slice(char *storage, int64_t page_bytes, int from, int to, int slice) {
  const int64_t at = (int64_t)slice * kSliceBytes;
  const uint4 *s = reinterpret_cast<const uint4 *>(storage + (int64_t)from * page_bytes + at);
  uint4 *d = reinterpret_cast<uint4 *>(storage + (int64_t)to * page_bytes + at);
  if (at + 16 * (int64_t)threadIdx.x < page_bytes) d[threadIdx.x] = s[threadIdx.x];
}

__global__ __launch_bounds__(kThreads) void pages_copy_kernel(char *storage, int64_t page_bytes, int num_pages,
                                                              const int32_t *__restrict__ src,
                                                              const int32_t *__restrict__ dst, int slices) {
  const int i = blockIdx.x / slices, slice = blockIdx.x % slices;
  const int from = src[i], to = dst[i];
  const bool good = (unsigned)from < (unsigned)num_pages && (unsigned)to < (unsigned)num_pages;
  KV_CHECK(good || threadIdx.x != 0, LORA_DEBUG_BAD_PAGE);
  if (good && from != to) copy_slice(storage, page_bytes, from, to, slice);
}

constexpr int kListMoves = 400;
struct MoveList {
  int32_t from[kListMoves], to[kListMoves];
};
__global__ __launch_bounds__(kThreads) void list_copy_kernel(char *storage, int64_t page_bytes, MoveList list, int slices) {
  const int i = blockIdx.x / slices;
  copy_slice(storage, page_bytes, list.from[i], list.to[i], blockIdx.x % slices);
}

constexpr int kListEntries = 256;
struct EntryList {
  int64_t at[kListEntries];
  int32_t page[kListEntries];
};
__global__ __launch_bounds__(kListEntries) void list_entries_kernel(int32_t *table, EntryList list, int n) {
  if ((int)threadIdx.x < n) table[list.at[threadIdx.x]] = list.page[threadIdx.x];
}

__global__ __launch_bounds__(kThreads) void clear_table_kernel(int32_t *table, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) table[i] = -1;
}

__global__ __launch_bounds__(kThreads) void table_remap_kernel(const int32_t *__restrict__ remap, int num_pages,
                                                               const int32_t *in, int32_t *out, int64_t count) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= count) return;
  const int32_t p = in[i];
  out[i] = (unsigned)p < (unsigned)num_pages ? remap[p] : p;
}

// One thread per 16-byte unit of a K row and the V row beside it; units of a token are
// consecutive, so a wave reads and writes whole rows (11902 tokens, 8 heads of 128: 18.2 us, 5.35 TB/s).
__global__ __launch_bounds__(kThreads) void append_kernel(lora_kv_view kv, const uint16_t *__restrict__ k_new,
                                                          const uint16_t *__restrict__ v_new, int64_t token_stride,
                                                          int64_t head_stride, const int32_t *__restrict__ token_seq,
                                                          const int32_t *__restrict__ token_pos, int64_t units) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= units) return;
  const int chunks = kv.head_dim >> 3, per = chunks * kv.kv_heads;
  const int t = (int)(i / per), u = (int)(i % per);
  const int h = u / chunks, c = u % chunks;
  const int s = token_seq[t], p = token_pos[t];
  const bool in = s < kv.num_seqs && p >= 0 && p < kv.max_pages * kv.page_tokens;
  KV_CHECK(in || s < 0, LORA_DEBUG_BAD_TOKEN);
  if (s < 0 || !in) return;
  const int page = kv.page_table[(int64_t)s * kv.max_pages + p / kv.page_tokens];
  KV_CHECK((unsigned)page < (unsigned)kv.num_pages, LORA_DEBUG_BAD_PAGE);
  if ((unsigned)page >= (unsigned)kv.num_pages) return;
  const int64_t from = t * token_stride + h * head_stride + c * 8;
  const int64_t to = page * kv.page_stride + h * kv.head_stride + (p % kv.page_tokens) * kv.token_stride + c * 8;
  const uint4 a = *reinterpret_cast<const uint4 *>(k_new + from);
  const uint4 b = *reinterpret_cast<const uint4 *>(v_new + from);
  *reinterpret_cast<uint4 *>((uint16_t *)kv.k + to) = a;
  *reinterpret_cast<uint4 *>((uint16_t *)kv.v + to) = b;
}

bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

lora_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? ok() : hip_fail(e, what);
}

}  // namespace

// --------------------------------------------------------------- bookkeeping's device steps

lora_status lora::kv_move_pages(void *storage, int64_t page_bytes, const std::vector<std::pair<int32_t, int32_t>> &moves,
                                hipStream_t stream) {
  const int64_t slices = (page_bytes + kSliceBytes - 1) / kSliceBytes;  // lora_kv_create bounds page_bytes
  const size_t most = (size_t)std::min<int64_t>(kListMoves, (int64_t)UINT32_MAX / kThreads / slices);  // of one launch
  for (size_t i0 = 0; i0 < moves.size(); i0 += most) {
    MoveList list{};
    const int n = (int)std::min<size_t>(most, moves.size() - i0);
    for (int i = 0; i < n; ++i) {
      list.from[i] = moves[i0 + (size_t)i].first;
      list.to[i] = moves[i0 + (size_t)i].second;
    }
    hipLaunchKernelGGL(list_copy_kernel, dim3((unsigned)(n * slices)), dim3(kThreads), 0, stream, (char *)storage, page_bytes,
                       list, (int)slices);
  }
  return launched("page move launch");
}

lora_status lora::kv_write_table(int32_t *table, const std::vector<std::pair<int64_t, int32_t>> &entries,
                                 hipStream_t stream) {
  for (size_t i0 = 0; i0 < entries.size(); i0 += kListEntries) {
    EntryList list{};
    const int n = (int)std::min<size_t>(kListEntries, entries.size() - i0);
    for (int i = 0; i < n; ++i) {
      list.at[i] = entries[i0 + (size_t)i].first;
      list.page[i] = entries[i0 + (size_t)i].second;
    }
    hipLaunchKernelGGL(list_entries_kernel, dim3(1), dim3(kListEntries), 0, stream, table, list, n);
  }
  return launched("page-table update launch");
}

lora_status lora::kv_clear_table(int32_t *table, int64_t count) {
  hipLaunchKernelGGL(clear_table_kernel, dim3(256), dim3(kThreads), 0, nullptr, table, count);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess) e = hipStreamSynchronize(nullptr);
  return e == hipSuccess ? LORA_OK : hip_fail(e, "page-table initialisation");
}

namespace {
struct Mark {
  hipEvent_t e = nullptr;
  ~Mark() {
    if (e) (void)hipEventDestroy(e);
  }
};
}  // namespace

lora_status lora::kv_mark(hipStream_t stream, std::shared_ptr<void> *mark) {
  std::shared_ptr<Mark> m = std::make_shared<Mark>();
  hipError_t e = hipEventCreateWithFlags(&m->e, hipEventDisableTiming);
  if (e == hipSuccess) e = hipEventRecord(m->e, stream);
  if (e != hipSuccess) return hip_fail(e, "marking the stream");
  *mark = m;
  return LORA_OK;
}

bool lora::kv_mark_done(const std::shared_ptr<void> &mark, bool wait) {
  const Mark *m = static_cast<const Mark *>(mark.get());
  if (wait) return hipEventSynchronize(m->e) == hipSuccess;
  const hipError_t e = hipEventQuery(m->e);
  if (e != hipSuccess) (void)hipGetLastError();  // "not ready" is no error of the caller's
  return e == hipSuccess;
}

lora_status lora::kv_not_capturing(hipStream_t stream) {
  hipStreamCaptureStatus s = hipStreamCaptureStatusNone;
  const hipError_t e = hipStreamIsCapturing(stream, &s);
  if (e != hipSuccess) return hip_fail(e, "hipStreamIsCapturing");
  if (s != hipStreamCaptureStatusNone)
    return fail(LORA_EINVAL, "sequence bookkeeping cannot be captured into a graph: its effect on the host happens once");
  return LORA_OK;
}

extern "C" lora_status lora_kv_debug_flags(uint32_t *flags, int32_t clear) {
  if (!flags) return fail(LORA_EINVAL, "null flags");
  *flags = 0;
#if LORA_DEBUG
  lora_status st = kv_debug_word(flags, clear);
  if (st == LORA_OK) st = kv_attn_debug(flags, clear);
  return st == LORA_OK ? ok() : st;
#else
  return fail(LORA_EUNSUPPORTED, "library built without LORA_DEBUG (load liblora_sgmv_debug.so)");
#endif
}

// --------------------------------------------------------------- entry points

extern "C" lora_status lora_pages_copy(void *storage, int64_t page_bytes, int32_t num_pages, const int32_t *src,
                                       const int32_t *dst, int32_t n, hipStream_t stream) {
  if (page_bytes <= 0 || page_bytes % 16 || num_pages < 0 || n < 0)
    return fail(LORA_EINVAL, "page copy: %d of %d pages of %lld bytes", n, num_pages, (long long)page_bytes);
  if (n == 0) return ok();
  if (!storage || !src || !dst) return fail(LORA_EINVAL, "null pointer");
  if (!aligned(storage, 16) || !aligned(src, 4) || !aligned(dst, 4))
    return fail(LORA_EINVAL, "page storage must be 16-byte aligned");
  const int64_t slices = (page_bytes + kSliceBytes - 1) / kSliceBytes;
  if (too_many(slices, (int64_t)kThreads * n)) return fail(LORA_EUNSUPPORTED, "page copy too large");
  hipLaunchKernelGGL(pages_copy_kernel, dim3((unsigned)(slices * n)), dim3(kThreads), 0, stream, (char *)storage,
                     page_bytes, num_pages, src, dst, (int)slices);
  return launched("page copy launch");
}

extern "C" lora_status lora_page_table_remap(const int32_t *remap, int32_t num_pages, const int32_t *table_in,
                                             int32_t *table_out, int64_t count, hipStream_t stream) {
  if (num_pages < 0 || count < 0) return fail(LORA_EINVAL, "negative size");
  if (count == 0) return ok();
  if (!table_in || !table_out || (num_pages > 0 && !remap)) return fail(LORA_EINVAL, "null pointer");
  if (!aligned(table_in, 4) || !aligned(table_out, 4) || !aligned(remap, 4))
    return fail(LORA_EINVAL, "page tables must be 4-byte aligned");
  const int64_t blocks = (count + kThreads - 1) / kThreads;
  if (too_many(blocks, kThreads)) return fail(LORA_EUNSUPPORTED, "page table too large");
  hipLaunchKernelGGL(table_remap_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, remap, num_pages, table_in,
                     table_out, count);
  return launched("page-table remap launch");
}

extern "C" lora_status lora_kv_append(const lora_kv_view *kv, const void *k_new, const void *v_new,
                                      int64_t new_token_stride, int64_t new_head_stride, const int32_t *token_seq,
                                      const int32_t *token_pos, int32_t num_tokens, hipStream_t stream) {
  lora_status st = check_view(kv);
  if (st != LORA_OK) return st;
  if (num_tokens < 0) return fail(LORA_EINVAL, "negative token count");
  if (new_token_stride < 0 || new_head_stride < 0 || new_token_stride % 8 || new_head_stride % 8)
    return fail(LORA_EINVAL, "strides of new rows must be multiples of 8 elements, not negative");
  if (num_tokens == 0 || kv->num_pages == 0 || kv->num_seqs == 0 || kv->max_pages == 0) return ok();
  if (!k_new || !v_new || !token_seq || !token_pos) return fail(LORA_EINVAL, "null pointer");
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(token_seq, 4) || !aligned(token_pos, 4))
    return fail(LORA_EINVAL, "new rows must be 16-byte aligned");
  const int64_t units = (int64_t)num_tokens * kv->kv_heads * (kv->head_dim / 8);
  const int64_t blocks = (units + kThreads - 1) / kThreads;
  if (too_many(blocks, kThreads)) return fail(LORA_EUNSUPPORTED, "append too large");
  hipLaunchKernelGGL(append_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, *kv, (const uint16_t *)k_new,
                     (const uint16_t *)v_new, new_token_stride, new_head_stride, token_seq, token_pos, units);
  return launched("append launch");
}
