// Drives the sequence bookkeeping (kv_host.cpp) with marks that cannot be made and waits that fail: no
// page may reach the pool before its readers are known to be done, and none may be lost.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <new>
#include <vector>

#include "kv_internal.h"

extern "C" {
hipError_t hipMemcpyAsync(void *, const void *, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "stub"; }
const char *hipGetErrorName(hipError_t) { return "stub"; }
}

enum Way { kWorks, kFails, kThrows };
static Way g_mark = kWorks;
static bool g_done = false, g_wait_works = true, g_capturing = false;

namespace lora {
lora_status kv_move_pages(void *, int64_t, const std::vector<std::pair<int32_t, int32_t>> &, hipStream_t) { return LORA_OK; }
lora_status kv_write_table(int32_t *table, const std::vector<std::pair<int64_t, int32_t>> &entries, hipStream_t) {
  for (auto &e : entries) table[e.first] = e.second;
  return LORA_OK;
}
lora_status kv_clear_table(int32_t *table, int64_t count) {
  for (int64_t i = 0; i < count; ++i) table[i] = -1;
  return LORA_OK;
}
lora_status kv_mark(hipStream_t stream, std::shared_ptr<void> *mark) {
  if (stream != (hipStream_t)16) abort();
  if (g_mark == kThrows) throw std::bad_alloc();
  if (g_mark == kFails) return fail(LORA_EHIP, "no mark");
  *mark = std::make_shared<int>(0);
  return LORA_OK;
}
bool kv_mark_done(const std::shared_ptr<void> &mark, bool wait) {
  if (!mark) abort();
  return wait ? g_wait_works : g_done;
}
lora_status kv_not_capturing(hipStream_t) { return g_capturing ? fail(LORA_EINVAL, "captured") : LORA_OK; }
void kv_device_wait() {}
}  // namespace lora

#define CHECK(c)                                             \
  do {                                                       \
    if (!(c)) {                                              \
      fprintf(stderr, "%d: %s\n", __LINE__, #c);             \
      exit(1);                                               \
    }                                                        \
  } while (0)

static const int kPages = 12, kSeqs = 3, kMax = 6;  // pages of one position
static uint16_t g_storage[kPages * 16];
static int32_t g_table[kSeqs * kMax];
static const hipStream_t kStream = (hipStream_t)16;

struct Cache {
  lora_pool *pool = nullptr;
  lora_kv *kv = nullptr;
  Cache() {
    g_mark = kWorks;
    g_done = false;
    g_wait_works = true;
    g_capturing = false;
    CHECK(lora_pool_create(kPages, 1, 16, LORA_BF16, LORA_WFMT_PLAIN, g_storage, nullptr, 0, &pool) == LORA_OK);
    CHECK(lora_kv_create(pool, 1, 8, kSeqs, kMax, g_table, 0, &kv) == LORA_OK);
    const int32_t ids[2] = {0, 1}, n[2] = {2, 5};
    CHECK(lora_kv_extend(kv, ids, n, 2, kStream) == LORA_OK);
  }
  int free_pages() {
    int32_t n = 0;
    CHECK(lora_pool_num_free(pool, &n) == LORA_OK);
    return n;
  }
  int spares() {
    lora_kv_stats s;
    CHECK(lora_kv_get_stats(kv, &s) == LORA_OK);
    return s.spare;
  }
  int trim(int wait) {
    int32_t left = -1;
    CHECK(lora_kv_trim(kv, wait, &left) == LORA_OK);
    return left;
  }
  ~Cache() {
    if (kv) lora_kv_destroy(kv);
    lora_pool_destroy(pool);
  }
};

// op 0: free, 1: truncate, 2: compact
static void dropped_pages(int op, Way way) {
  Cache c;
  const int32_t first = 0;
  int spares = 2;
  g_mark = way;
  if (op == 0) {
    CHECK(lora_kv_free(c.kv, &first, 1, kStream) == LORA_OK);
    CHECK(g_table[0] == -1 && g_table[1] == -1);
  } else if (op == 1) {
    CHECK(lora_kv_truncate(c.kv, 1, 3, kStream) == LORA_OK);
    CHECK(g_table[kMax + 2] >= 0 && g_table[kMax + 3] == -1 && g_table[kMax + 4] == -1);
  } else {
    g_mark = kWorks;
    g_done = true;
    CHECK(lora_kv_free(c.kv, &first, 1, kStream) == LORA_OK && c.trim(0) == 0);
    g_done = false;
    g_mark = way;
    int32_t moved = 0;
    CHECK(lora_kv_compact(c.kv, &moved, kStream) == LORA_OK && moved == 2);
  }
  CHECK(c.spares() == spares);
  const int before = c.free_pages();
  CHECK(c.trim(0) == spares && c.trim(1) == spares && c.free_pages() == before);  // no mark: not known to be done
  g_mark = kWorks;
  g_capturing = true;
  CHECK(c.trim(1) == spares);
  g_capturing = false;
  CHECK(c.trim(0) == spares && c.free_pages() == before);  // marked now, and not done
  g_done = true;
  CHECK(c.trim(0) == 0 && c.free_pages() == before + spares);
}

// Spares without a mark are taken again by the cache that dropped them.
static void taken_again() {
  Cache c;
  const int32_t first = 0, n = 2;
  g_mark = kFails;
  CHECK(lora_kv_free(c.kv, &first, 1, kStream) == LORA_OK && c.spares() == 2);
  const int before = c.free_pages();
  CHECK(lora_kv_extend(c.kv, &first, &n, 1, kStream) == LORA_OK && c.spares() == 0 && c.free_pages() == before);
}

// A cache that goes gives back what it knows to be done, and keeps the rest from the pool.
static void destroyed(Way mark, bool wait_works, bool capturing, bool spare) {
  Cache c;
  const int32_t first = 0;
  if (spare) CHECK(lora_kv_free(c.kv, &first, 1, kStream) == LORA_OK);
  const bool works = mark == kWorks && wait_works && !capturing;
  g_mark = mark;
  g_wait_works = wait_works;
  g_capturing = capturing;
  lora_kv_destroy(c.kv);
  c.kv = nullptr;
  // the spares' own mark was made before, and is waited for whatever becomes of the others'
  CHECK(c.free_pages() == (works ? kPages : kPages - 7 + (spare && wait_works ? 2 : 0)));
}

int main() {
  for (bool spare : {false, true}) {
    destroyed(kWorks, true, false, spare);
    destroyed(kFails, true, false, spare);
    destroyed(kThrows, true, false, spare);
    destroyed(kWorks, false, false, spare);
    destroyed(kWorks, true, true, spare);
  }
  for (int op = 0; op < 3; ++op)
    for (Way way : {kFails, kThrows}) dropped_pages(op, way);
  taken_again();
  printf("kv mark driver ok\n");
  return 0;
}
