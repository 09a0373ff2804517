// Drives what trees, listed pages and 8-bit rows add to the host half of the paged KV cache (kv_host.cpp) under the
// sanitizers: plans of every kind at random sizes, caches of every layout and the places that their views name.
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
lora_status kv_move_pages(void *storage, int64_t page_bytes, const std::vector<std::pair<int32_t, int32_t>> &moves, hipStream_t) {
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
lora_status kv_mark(hipStream_t, std::shared_ptr<void> *mark) {
  *mark = std::make_shared<int>(0);
  return LORA_OK;
}
bool kv_mark_done(const std::shared_ptr<void> &, bool) { return true; }
lora_status kv_not_capturing(hipStream_t) { return LORA_OK; }
}  // namespace lora

#define CHECK(c)                                             \
  do {                                                       \
    if (!(c)) {                                              \
      fprintf(stderr, "%d: %s\n", __LINE__, #c);             \
      exit(1);                                               \
    }                                                        \
  } while (0)

static void plans(std::mt19937 &rng) {
  for (int turn = 0; turn < 400; ++turn) {
    const int kind = (int)(rng() % 3), reqs = (int)(rng() % 40), kv_heads = 1 + (int)(rng() % 8), group = 1 + (int)(rng() % 20);
    std::vector<int32_t> starts = {0}, seq, len;
    for (int r = 0; r < reqs; ++r) {
      starts.push_back(starts.back() + (kind == 2 ? (int)(rng() % 2) : (int)(rng() % (rng() % 3 ? 30 : 400))));
      seq.push_back((int32_t)(rng() % 50));
      len.push_back((int32_t)(rng() % (rng() % 4 ? 3000 : 200000)));
    }
    const int flags = kind == 2 ? LORA_ATTN_BLOCKS : (kind == 1 ? LORA_ATTN_TREE : 0) | (rng() % 2 ? LORA_ATTN_CAUSAL : 0);
    const int window = kind != 2 && rng() % 2 ? 1 + (int)(rng() % 5000) : 0;
    lora_attn_plan p, again;
    auto call = [&](lora_attn_plan *plan, lora_attn_item *items, int32_t room) {
      return lora_kv_attn_plan(starts.data(), seq.data(), len.data(), reqs, 50, 1 << 20, kv_heads * group, kv_heads, 64, flags, window,
                               (int)(rng() % 2) ? 0 : 3, plan, items, room);
    };
    std::mt19937 same = rng;
    CHECK(call(&p, nullptr, 0) == LORA_OK);
    const int n = p.num_row_items + p.num_tile_items + p.num_joins;
    std::vector<lora_attn_item> items((size_t)n);
    rng = same;
    CHECK(call(&again, items.data(), n) == LORA_OK && memcmp(&p, &again, sizeof p) == 0);
    for (int i = 0; i < p.num_row_items + p.num_tile_items; ++i) {
      CHECK(items[i].rows >= 1 && items[i].rows <= (i < p.num_row_items ? LORA_ATTN_ROWS : LORA_ATTN_TILE_ROWS));
      CHECK(0 <= items[i].kv_begin && items[i].kv_begin <= items[i].kv_end && items[i].part >= -1);
      CHECK(items[i].part < 0 || items[i].part + items[i].rows <= p.num_part_rows);
      CHECK(kind != 2 || items[i].row0 + items[i].rows <= group);
    }
  }
}

static void layouts(std::mt19937 &rng) {
  for (int turn = 0; turn < 200; ++turn) {
    const int heads = 1 + (int)(rng() % 4), dim = 16 * (1 + (int)(rng() % 8)), rows = 1 + (int)(rng() % 16), width = 8 * (8 + (int)(rng() % 60));
    const int pages = 9, seqs = 3, mp = 4, flags = (rng() % 2 ? LORA_KV_FP8 : 0) | (rng() % 2 ? LORA_KV_BOUNDS : 0);
    std::vector<char> storage((size_t)pages * rows * width * 2 + 16);
    char *base = storage.data() + (16 - (uintptr_t)storage.data() % 16) % 16;
    std::vector<int32_t> table((size_t)seqs * mp);
    lora_pool *pool = nullptr;
    CHECK(lora_pool_create(pages, rows, width, LORA_BF16, LORA_WFMT_PLAIN, base, nullptr, rng(), &pool) == LORA_OK);
    lora_kv *kv = nullptr;
    const lora_status st = lora_kv_create(pool, heads, dim, seqs, mp, table.data(), flags, &kv);
    if (st != LORA_OK) {
      CHECK(st == LORA_EUNSUPPORTED);
      lora_pool_destroy(pool);
      continue;
    }
    lora_kv8_view v{};
    if (flags & LORA_KV_FP8) {
      CHECK(lora_kv_get_view8(kv, &v) == LORA_OK && lora_kv_get_view(kv, &v.kv) == LORA_EINVAL);
      CHECK(lora_kv_get_view8(kv, &v) == LORA_OK);
    } else {
      CHECK(lora_kv_get_view(kv, &v.kv) == LORA_OK && lora_kv_get_view8(kv, &v) == LORA_EINVAL);
      CHECK(lora_kv_get_view(kv, &v.kv) == LORA_OK);
    }
    CHECK(lora::check_view(&v.kv) == LORA_OK);
    // every place is written once, within the storage
    const int size = flags & LORA_KV_FP8 ? 1 : 2;
    std::vector<char> seen((size_t)pages * rows * width * 2, 0);
    auto mark = [&](const void *at, int64_t bytes) {
      for (int64_t i = 0; i < bytes; ++i) {
        const int64_t o = (const char *)at - base + i;
        CHECK(o >= 0 && o < (int64_t)seen.size() && !seen[(size_t)o]);
        seen[(size_t)o] = 1;
      }
    };
    lora_kv_bounds b{};
    int64_t row = 0;
    CHECK(lora_kv_get_bounds(kv, &b) == (flags & LORA_KV_BOUNDS ? LORA_OK : LORA_EINVAL) && lora_kv_bounds_row_bytes(dim, &row) == LORA_OK);
    for (int g = 0; g < pages; ++g)
      for (int h = 0; h < heads; ++h) {
        for (int p = 0; p < v.kv.page_tokens; ++p) {
          const int64_t at = (g * v.kv.page_stride + h * v.kv.head_stride + p * v.kv.token_stride) * size;
          mark((char *)v.kv.k + at, dim * size);
          mark((char *)v.kv.v + at, dim * size);
          if (size == 1) {
            const int64_t s = g * v.scale_page_stride + h * v.scale_head_stride + p * v.scale_token_stride;
            mark(v.k_scales + s, 1);
            mark(v.v_scales + s, 1);
          }
        }
        if (flags & LORA_KV_BOUNDS) {
          CHECK(((char *)b.rows - base) % 16 == 0 && b.page_stride % 16 == 0 && b.head_stride % 16 == 0);
          mark((char *)b.rows + g * b.page_stride + h * b.head_stride, row);
        }
      }
    const int32_t ids[2] = {0, 2}, grow[2] = {v.kv.page_tokens + 1, 1};
    CHECK(lora_kv_extend(kv, ids, grow, 2, nullptr) == LORA_OK);
    lora_kv_destroy(kv);
    lora_pool_destroy(pool);
  }
}

int main() {
  std::mt19937 rng(7);
  plans(rng);
  layouts(rng);
  printf("kv more driver ok\n");
  return 0;
}
