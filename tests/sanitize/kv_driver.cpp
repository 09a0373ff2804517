// Drives the host half of the paged KV cache (kv_host.cpp, over the pool of
// host.cpp) with random batches under the sanitizers.  Its device steps are
// replaced by host ones that act on host memory, so that moves and page-table
// entries out of range are caught too.
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <memory>
#include <random>
#include <vector>

#include "kv_internal.h"

extern "C" {
hipError_t hipMemcpyAsync(void *dst, const void *src, size_t bytes, hipMemcpyKind, hipStream_t) {
  memcpy(dst, src, bytes);
  return hipSuccess;
}
const char *hipGetErrorString(hipError_t) { return "stub"; }
const char *hipGetErrorName(hipError_t) { return "stub"; }
}

namespace lora {
lora_status kv_move_pages(void *storage, int64_t page_bytes, const std::vector<std::pair<int32_t, int32_t>> &moves,
                          hipStream_t) {
  for (auto &m : moves) memcpy((char *)storage + m.second * page_bytes, (char *)storage + m.first * page_bytes, (size_t)page_bytes);
  return LORA_OK;
}
lora_status kv_write_table(int32_t *table, const std::vector<std::pair<int64_t, int32_t>> &entries, hipStream_t) {
  for (auto &e : entries) table[e.first] = e.second;
  return LORA_OK;
}
lora_status kv_clear_table(int32_t *table, int64_t count) {
  for (int64_t i = 0; i < count; ++i) table[i] = -1;
  return LORA_OK;
}
static int g_queries = 0;
lora_status kv_mark(hipStream_t, std::shared_ptr<void> *mark) {
  *mark = std::make_shared<int>(0);
  return LORA_OK;
}
bool kv_mark_done(const std::shared_ptr<void> &, bool wait) { return wait || ++g_queries % 3 == 0; }
lora_status kv_not_capturing(hipStream_t) { return LORA_OK; }
void kv_device_wait() {}
}  // namespace lora

#define CHECK(c)                                             \
  do {                                                       \
    if (!(c)) {                                              \
      fprintf(stderr, "%d: %s\n", __LINE__, #c);             \
      exit(1);                                               \
    }                                                        \
  } while (0)

static void sequences(std::mt19937 &rng) {
  const int heads = 2, dim = 8, rows = 4, width = 32, pt = rows * width / (2 * heads * dim), pages = 30, seqs = 5, mp = 6;
  std::vector<uint16_t> storage((size_t)pages * rows * width);
  std::vector<int32_t> table((size_t)seqs * mp);
  lora_pool *pool = nullptr;
  alignas(16) static uint16_t dummy;
  (void)dummy;
  CHECK(lora_pool_create(pages, rows, width, LORA_BF16, LORA_WFMT_PLAIN, storage.data(), nullptr, rng(), &pool) == LORA_OK);
  lora_kv *kv = nullptr;
  CHECK(lora_kv_create(pool, heads, dim, seqs, mp, table.data(), 0, &kv) == LORA_OK);
  std::vector<std::vector<uint16_t>> model((size_t)seqs);
  std::vector<bool> live((size_t)seqs, false);
  uint16_t stamp = 0;
  lora_kv_view v;
  CHECK(lora_kv_get_view(kv, &v) == LORA_OK && v.page_tokens == pt);
  for (int step = 0; step < 400; ++step) {
    const int op = (int)(rng() % 10), s = (int)(rng() % seqs);
    if (op < 5) {
      std::vector<int32_t> ids, counts;
      for (int i = 0; i < seqs; ++i)
        if (rng() % 2) {
          ids.push_back(i);
          counts.push_back((int32_t)(rng() % 12));
        }
      const lora_status st = lora_kv_extend(kv, ids.data(), counts.data(), (int32_t)ids.size(), nullptr);
      CHECK(st == LORA_OK || st == LORA_ENOMEM || st == LORA_EINVAL);
      if (st == LORA_OK)
        for (size_t i = 0; i < ids.size(); ++i) {
          live[(size_t)ids[i]] = true;
          auto &m = model[(size_t)ids[i]];
          for (int c = 0; c < counts[i]; ++c) {
            const int p = (int)m.size();
            ((uint16_t *)v.k)[table[(size_t)(ids[i] * mp + p / pt)] * v.page_stride + (p % pt) * v.token_stride] = ++stamp;
            m.push_back(stamp);
          }
        }
    } else if (op == 5) {
      const int d = (int)(rng() % seqs);
      const int32_t dst = d;
      const lora_status st = lora_kv_fork(kv, s, &dst, 1, nullptr);
      CHECK(st == (live[(size_t)s] && !live[(size_t)d] ? LORA_OK : LORA_EINVAL));
      if (st == LORA_OK) {
        model[(size_t)d] = model[(size_t)s];
        live[(size_t)d] = true;
      }
    } else if (op == 6) {
      const int32_t cut = (int32_t)(rng() % (model[(size_t)s].size() + 1));
      CHECK(lora_kv_truncate(kv, s, cut, nullptr) == (live[(size_t)s] ? LORA_OK : LORA_EINVAL));
      if (live[(size_t)s]) model[(size_t)s].resize((size_t)cut);
    } else if (op == 7) {
      const int32_t id = s;
      CHECK(lora_kv_free(kv, &id, 1, nullptr) == (live[(size_t)s] ? LORA_OK : LORA_EINVAL));
      live[(size_t)s] = false;
      model[(size_t)s].clear();
    } else if (op == 8) {
      int32_t moved = 0;
      CHECK(lora_kv_compact(kv, &moved, nullptr) == LORA_OK);
    } else {
      int32_t left = 0;
      CHECK(lora_kv_trim(kv, (int32_t)(rng() % 2), &left) == LORA_OK);
    }
    for (int i = 0; i < seqs; ++i)
      for (size_t p = 0; p < model[(size_t)i].size(); ++p)
        CHECK(((uint16_t *)v.k)[table[(size_t)i * mp + p / pt] * v.page_stride + (int64_t)(p % pt) * v.token_stride] ==
              model[(size_t)i][p]);
  }
  lora_kv_destroy(kv);
  int32_t nf = 0;
  CHECK(lora_pool_num_free(pool, &nf) == LORA_OK && nf == pages);
  lora_pool_destroy(pool);
}

static void plans(std::mt19937 &rng) {
  const int n = (int)(rng() % 12);
  std::vector<int32_t> starts{0}, seq, kv;
  for (int i = 0; i < n; ++i) {
    starts.push_back(starts.back() + (int32_t)(rng() % 3 ? rng() % 3 : rng() % 400));
    seq.push_back((int32_t)(rng() % 20));
    kv.push_back((int32_t)(rng() % 4 ? rng() % 300 : rng() % 100000));
  }
  const int heads = 1 + (int)(rng() % 4), group = 1 + (int)(rng() % 20);
  lora_attn_plan p;
  const int flags = (int)(rng() % 2), window = rng() % 2 ? (int)(rng() % 1000) : 0, parts = (int)(rng() % 65);
  CHECK(lora_kv_attn_plan(starts.data(), seq.data(), kv.data(), n, 20, 100000, heads * group, heads, 64, flags, window, parts, &p,
                          nullptr, 0) == LORA_OK);
  const int total = p.num_row_items + p.num_tile_items + p.num_joins;
  std::vector<lora_attn_item> items((size_t)total);
  CHECK(lora_kv_attn_plan(starts.data(), seq.data(), kv.data(), n, 20, 100000, heads * group, heads, 64, flags, window, parts, &p,
                          items.data(), total) == LORA_OK);
  if (total)
    CHECK(lora_kv_attn_plan(starts.data(), seq.data(), kv.data(), n, 20, 100000, heads * group, heads, 64, flags, window, parts, &p,
                            items.data(), total - 1) == LORA_ENOMEM);
}

int main() {
  std::mt19937 rng(5);
  for (int i = 0; i < 30; ++i) sequences(rng);
  for (int i = 0; i < 300; ++i) plans(rng);
  printf("kv driver ok\n");
  return 0;
}
