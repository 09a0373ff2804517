// Host half of the paged KV cache: the attention planner and the bookkeeping of
// sequences over a pool's pages.  Device steps go through kv_internal.h.
#include <algorithm>
#include <exception>
#include <new>
#include <vector>

#include "kv_internal.h"

using namespace lora;

namespace {

// Runs f; memory that the host lacks is an error, not an exception over the C boundary.
template <typename F>
lora_status guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc &) {
    return fail(LORA_ENOMEM, "out of host memory");
  } catch (const std::exception &e) {
    return fail(LORA_ENOMEM, "%s", e.what());
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

lora_status lora::check_view(const lora_kv_view *kv) {
  if (!kv) return fail(LORA_EINVAL, "null view");
  if (kv->dtype != LORA_BF16) return fail(LORA_EUNSUPPORTED, "a KV cache holds bf16 (got dtype %d)", kv->dtype);
  if (kv->head_dim < 8 || kv->head_dim > 256 || kv->head_dim % 8)
    return fail(LORA_EUNSUPPORTED, "head_dim must be a multiple of 8 in 8..256 (got %d)", kv->head_dim);
  if (kv->kv_heads < 1 || kv->page_tokens < 1 || kv->num_pages < 0 || kv->num_seqs < 0 || kv->max_pages < 0)
    return fail(LORA_EINVAL, "KV view sizes: %d heads, %d positions per page, %d pages, %d x %d page table",
                kv->kv_heads, kv->page_tokens, kv->num_pages, kv->num_seqs, kv->max_pages);
  if ((int64_t)kv->max_pages * kv->page_tokens > INT32_MAX)
    return fail(LORA_EUNSUPPORTED, "a sequence of more than 2^31 - 1 positions");
  if (kv->page_stride < 0 || kv->head_stride < 0 || kv->token_stride < 0 || kv->page_stride % 8 ||
      kv->head_stride % 8 || kv->token_stride % 8)
    return fail(LORA_EINVAL, "KV strides must be multiples of 8 elements, not negative");
  // attention reads the page table also where there are no pages for its entries to name
  const bool table = kv->num_seqs > 0 && kv->max_pages > 0, rows = table && kv->num_pages > 0;
  if ((table && !kv->page_table) || (rows && (!kv->k || !kv->v))) return fail(LORA_EINVAL, "null KV pointer");
  if (((uintptr_t)kv->k & 15) || ((uintptr_t)kv->v & 15) || ((uintptr_t)kv->page_table & 3))
    return fail(LORA_EINVAL, "k and v must be 16-byte aligned");
  return LORA_OK;
}

// --------------------------------------------------------------------------
// Attention planner.

namespace {

// Items of one kind aim at this many (item, KV head) units, and at no range of fewer positions than
// kMinRange: below that a range's own start and the join cost more than the
// parallelism gives.  [0] row items, [1] tile items.  Measured, 64 / 8 heads of 128: twice the units, 64 tokens over 512
// positions each 41 us instead of 29.5, a chunk of 512 over 2048 61 instead of 48; half of them, a chunk of 128 over
// 8192 93 instead of 63.  Row items of at least 128 positions, 4 tokens over 300 each: 12.6 us instead of 10.2, of
// at least 512, one token over 2048: 16.1 instead of 13.6.  Tile items of at least 256, a chunk of 16 over 8192: 53
// us instead of 43, of at least 1024, a chunk of 64 over 2048: 39 instead of 33.
constexpr int64_t kAimUnits[2] = {512, 256};
constexpr int64_t kMinRange[2] = {256, 512};
constexpr int64_t kComputeUnits = 256;
constexpr int32_t kTileKv = 64;  // range borders are multiples of this

struct Tile {
  lora_attn_item it;
  int64_t span;
};

}  // namespace

extern "C" lora_status lora_kv_attn_plan(const int32_t *q_starts, const int32_t *seq, const int32_t *kv_len,
                                         int32_t num_reqs, int32_t num_seqs, int64_t max_kv, int32_t q_heads,
                                         int32_t kv_heads, int32_t head_dim, int32_t flags, int32_t window,
                                         int32_t max_parts, lora_attn_plan *plan, lora_attn_item *items,
                                         int32_t capacity) {
  if (!plan) return fail(LORA_EINVAL, "null plan");
  if (num_reqs < 0 || num_seqs < 0 || max_kv < 0 || capacity < 0) return fail(LORA_EINVAL, "negative size");
  if (!q_starts || (num_reqs > 0 && (!seq || !kv_len))) return fail(LORA_EINVAL, "null request arrays");
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads)
    return fail(LORA_EINVAL, "%d query heads over %d KV heads", q_heads, kv_heads);
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(LORA_EUNSUPPORTED, "head_dim must be a multiple of 8 in 8..256 (got %d)", head_dim);
  if (flags & ~LORA_ATTN_CAUSAL) return fail(LORA_EINVAL, "unknown flags 0x%x", flags);
  if (window < 0) return fail(LORA_EINVAL, "negative window");
  if (max_parts < 0 || max_parts > LORA_ATTN_MAX_PARTS)
    return fail(LORA_EINVAL, "max_parts %d outside 0..%d", max_parts, LORA_ATTN_MAX_PARTS);
  if (q_starts[0] != 0) return fail(LORA_EINVAL, "q_starts begins at %d", q_starts[0]);
  const int64_t group = q_heads / kv_heads;
  for (int32_t r = 0; r < num_reqs; ++r) {
    if (q_starts[r + 1] < q_starts[r]) return fail(LORA_EINVAL, "q_starts decreases at %d", r);
    if (seq[r] < 0 || seq[r] >= num_seqs) return fail(LORA_ERANGE, "request %d names sequence %d of %d", r, seq[r], num_seqs);
    if (kv_len[r] < 0 || kv_len[r] > max_kv)
      return fail(LORA_ERANGE, "request %d has %d positions, its sequence holds %lld", r, kv_len[r], (long long)max_kv);
    if ((q_starts[r + 1] - q_starts[r]) * group > INT32_MAX)
      return fail(LORA_EUNSUPPORTED, "request %d has too many rows", r);
  }
  return guarded([&]() -> lora_status {
    std::vector<Tile> tiles[2];  // row items, tile items
    int64_t medium = 0;          // (request, KV head) units whose rows two row items hold
    for (int32_t r = 0; r < num_reqs; ++r) {
      const int64_t rows = (q_starts[r + 1] - q_starts[r]) * group;
      medium += rows > LORA_ATTN_ROWS && rows <= 2 * LORA_ATTN_ROWS ? kv_heads : 0;
    }
    // 17 to 32 rows: one tile item reads K and V once, two row items twice (64 requests of 24 rows over 2048
    // positions, 8 KV heads: 96 us and 184); where units are few the row items' shorter steps count more (4
    // requests: 35 us and 24).  33 rows and more: 64 requests 100 us as tile items, 268 as row items.
    const int64_t tile_min_rows = (medium >= kComputeUnits ? 1 : 2) * LORA_ATTN_ROWS + 1;
    for (int32_t r = 0; r < num_reqs; ++r) {
      const int32_t qn = q_starts[r + 1] - q_starts[r];
      const int64_t rows = qn * group, pos0 = (int64_t)kv_len[r] - qn;
      const int kind = rows >= tile_min_rows;
      const int64_t step = kind ? LORA_ATTN_TILE_ROWS : LORA_ATTN_ROWS;
      for (int64_t row0 = 0; row0 < rows; row0 += step) {
        const int64_t n = std::min(step, rows - row0);
        const int64_t first = pos0 + row0 / group, last = pos0 + (row0 + n - 1) / group;
        const int64_t end = (flags & LORA_ATTN_CAUSAL) ? std::min<int64_t>(kv_len[r], last + 1) : kv_len[r];
        const int64_t begin = window > 0 ? std::max<int64_t>(0, first - window + 1) : 0;
        Tile t{};
        t.it = {q_starts[r], (int32_t)row0, (int32_t)n, seq[r], (int32_t)pos0, (int32_t)begin,
                (int32_t)std::max(begin, end), -1};
        if (end <= begin) t.it.kv_begin = t.it.kv_end = 0;
        t.span = t.it.kv_end - t.it.kv_begin;
        tiles[kind].push_back(t);
      }
    }
    std::vector<lora_attn_item> out[2], joins;
    int64_t part_rows = 0;
    for (int kind = 0; kind < 2; ++kind) {
      int64_t work = 0, widest = 0;
      for (const Tile &t : tiles[kind]) {
        work += t.span * kv_heads;
        widest = std::max(widest, t.span);
      }
      // positions per range: an even share of the work for each unit aimed at
      auto even = [&](int64_t units) { return cdiv(cdiv(work, units), kTileKv) * kTileKv; };
      int64_t share = even(kAimUnits[kind]);
      // Row items of uneven spans aim at twice the units, which the device takes longest first (64 / 8 heads of 128, 64
      // tokens over 256 to 8192 positions: 250 us, else 275).
      if (kind == 0 && widest > share * 3 / 2) share = even(2 * kAimUnits[0]);
      share = std::max(kMinRange[kind], share);
      std::vector<Tile> ranges;
      for (const Tile &t : tiles[kind]) {
        int64_t parts = max_parts == 1 ? 1 : std::max<int64_t>(1, (t.span + share / 2) / share);
        parts = std::min<int64_t>(parts, max_parts ? max_parts : LORA_ATTN_MAX_PARTS);
        if (parts == 1) {
          ranges.push_back(t);
          continue;
        }
        const int64_t base = t.it.kv_begin / kTileKv * kTileKv;
        const int64_t len = cdiv(cdiv(t.it.kv_end - base, parts), kTileKv) * kTileKv;
        parts = cdiv(t.it.kv_end - base, len);
        lora_attn_item j = t.it;
        j.kv_begin = (int32_t)part_rows;
        j.part = (int32_t)parts;
        for (int64_t p = 0; p < parts; ++p) {
          Tile s = t;
          s.it.kv_begin = (int32_t)std::max<int64_t>(t.it.kv_begin, base + p * len);
          s.it.kv_end = (int32_t)std::min<int64_t>(t.it.kv_end, base + (p + 1) * len);
          s.it.part = (int32_t)part_rows;
          s.span = s.it.kv_end - s.it.kv_begin;
          part_rows += t.it.rows;
          if (part_rows > INT32_MAX) return fail(LORA_EUNSUPPORTED, "too many rows of partial results");
          ranges.push_back(s);
        }
        joins.push_back(j);
      }
      std::stable_sort(ranges.begin(), ranges.end(), [](const Tile &a, const Tile &b) { return a.span > b.span; });
      for (const Tile &t : ranges) out[kind].push_back(t.it);
    }
    const size_t total = out[0].size() + out[1].size() + joins.size();
    if (total > (size_t)INT32_MAX || (int64_t)total * kv_heads > INT32_MAX)
      return fail(LORA_EUNSUPPORTED, "plan too large");
    lora_attn_plan p{};
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.flags = flags;
    p.window = window;
    p.num_tokens = q_starts[num_reqs];
    p.num_row_items = (int32_t)out[0].size();
    p.num_tile_items = (int32_t)out[1].size();
    p.num_joins = (int32_t)joins.size();
    p.num_part_rows = (int32_t)part_rows;
    p.workspace_bytes = part_rows * kv_heads * (head_dim + 4) * (int64_t)sizeof(float);
    *plan = p;
    if (!items) return ok();
    if ((int64_t)total > capacity) return fail(LORA_ENOMEM, "plan needs %zu items, capacity %d", total, capacity);
    lora_attn_item *at = items;
    for (const auto *v : {&out[0], &out[1], &joins}) at = std::copy(v->begin(), v->end(), at);
    return ok();
  });
}

// --------------------------------------------------------------------------
// Sequences.

struct Seq {
  int32_t len = -1;  // not in use
  std::vector<int32_t> pages;
};

struct Spare {
  int32_t page;
  bool marked;                 // false: the mark could not be made yet
  std::shared_ptr<void> mark;  // the work that may still read it (null: none, host only)
};

struct lora_kv {
  lora_pool *pool;
  int32_t kv_heads, head_dim, page_tokens, max_pages, flags;
  int32_t *table;
  hipStream_t stream = nullptr;  // of the last call with device steps
  std::vector<Seq> seqs;
  std::vector<int32_t> refs;   // per page of the pool: sequences that hold it
  std::vector<Spare> spares;
  bool host_only() const { return flags & LORA_KV_HOST_ONLY; }
};

namespace {

lora_status check_seq(const lora_kv *kv, int32_t s) {
  if (s < 0 || s >= (int32_t)kv->seqs.size())
    return fail(LORA_ERANGE, "sequence %d outside [0, %zu)", s, kv->seqs.size());
  return LORA_OK;
}

// Checks that the ids are in range and none is listed twice.
lora_status check_ids(const lora_kv *kv, const int32_t *ids, int32_t n) {
  if (n < 0 || (n > 0 && !ids)) return fail(LORA_EINVAL, "bad sequence list");
  std::vector<int32_t> sorted(ids, ids + n);
  for (int32_t s : sorted) {
    lora_status st = check_seq(kv, s);
    if (st != LORA_OK) return st;
  }
  std::sort(sorted.begin(), sorted.end());
  const auto twice = std::adjacent_find(sorted.begin(), sorted.end());
  if (twice != sorted.end()) return fail(LORA_EINVAL, "sequence %d is listed twice", *twice);
  return LORA_OK;
}

lora_status begin_device(lora_kv *kv, hipStream_t stream) {
  if (kv->host_only()) return LORA_OK;
  const lora_status st = kv_not_capturing(stream);
  if (st == LORA_OK) kv->stream = stream;
  return st;
}

// A mark behind everything queued on the cache's stream; false where it cannot be made.
bool try_mark(const lora_kv *kv, std::shared_ptr<void> *mark) {
  try {
    return kv_mark(kv->stream, mark) == LORA_OK;
  } catch (const std::bad_alloc &) {
    return false;
  }
}

// The device steps of one call, in order: page copies, then table entries.
struct Steps {
  std::vector<std::pair<int32_t, int32_t>> moves;
  std::vector<std::pair<int64_t, int32_t>> entries;
};

lora_status run_steps(lora_kv *kv, const Steps &s, hipStream_t stream) {
  if (kv->host_only()) return LORA_OK;
  lora_status st = LORA_OK;
  if (!s.moves.empty())
    st = kv_move_pages(kv->pool->storage, (int64_t)kv->pool->page_rows * (int64_t)kv->pool->row_bytes, s.moves, stream);
  if (st == LORA_OK && !s.entries.empty()) st = kv_write_table(kv->table, s.entries, stream);
  return st;
}

// Pages that nothing holds any more become spares, marked behind everything queued on the stream.  Nothing here
// fails, since the sequences have changed already (the caller has reserved the room): a mark that cannot be made is
// made by a later trim, whose place in the stream is a later one.
void make_spares(lora_kv *kv, const std::vector<int32_t> &dropped) {
  if (dropped.empty()) return;
  std::shared_ptr<void> mark;
  const bool marked = kv->host_only() || try_mark(kv, &mark);
  for (int32_t p : dropped) kv->spares.push_back({p, marked, mark});
}

int64_t entry(const lora_kv *kv, int32_t seq, size_t i) { return (int64_t)seq * kv->max_pages + (int64_t)i; }

void drop(lora_kv *kv, int32_t page, std::vector<int32_t> &dropped) {
  if (--kv->refs[(size_t)page] == 0) dropped.push_back(page);
}

}  // namespace

extern "C" lora_status lora_kv_create(lora_pool *pool, int32_t kv_heads, int32_t head_dim, int32_t max_seqs,
                                      int32_t max_pages, int32_t *device_page_table, int32_t flags, lora_kv **out) {
  if (!pool || !out) return fail(LORA_EINVAL, "null argument");
  if (flags & ~LORA_KV_HOST_ONLY) return fail(LORA_EINVAL, "unknown flags 0x%x", flags);
  if (kv_heads < 1 || max_seqs < 1 || max_pages < 1)
    return fail(LORA_EINVAL, "%d KV heads, %d sequences of %d pages", kv_heads, max_seqs, max_pages);
  if (head_dim < 8 || head_dim > 256 || head_dim % 8)
    return fail(LORA_EUNSUPPORTED, "head_dim must be a multiple of 8 in 8..256 (got %d)", head_dim);
  if (pool->dtype != LORA_BF16 || pool->weight_format != LORA_WFMT_PLAIN)
    return fail(LORA_EUNSUPPORTED, "a KV cache needs a plain bf16 pool");
  const int64_t elems = (int64_t)pool->page_rows * pool->row_width;
  const int64_t tokens = elems / (2 * (int64_t)kv_heads * head_dim);
  if (tokens < 1 || elems % 8)
    return fail(LORA_EUNSUPPORTED, "a page of %lld elements for %d KV heads of %d", (long long)elems, kv_heads, head_dim);
  if (elems > kKvMaxPageBytes / 2) return fail(LORA_EUNSUPPORTED, "a page of %lld elements", (long long)elems);
  if (tokens * max_pages > INT32_MAX) return fail(LORA_EUNSUPPORTED, "a sequence of more than 2^31 - 1 positions");
  const bool host_only = flags & LORA_KV_HOST_ONLY;
  if (!host_only && !device_page_table) return fail(LORA_EINVAL, "null page table");
  if (!host_only && ((uintptr_t)pool->storage & 15)) return fail(LORA_EINVAL, "the pool's storage is not 16-byte aligned");
  return guarded([&]() -> lora_status {
    std::unique_ptr<lora_kv> kv(new lora_kv());
    kv->pool = pool;
    kv->kv_heads = kv_heads;
    kv->head_dim = head_dim;
    kv->page_tokens = (int32_t)tokens;
    kv->max_pages = max_pages;
    kv->flags = flags;
    kv->table = device_page_table;
    kv->seqs.resize((size_t)max_seqs);
    kv->refs.assign((size_t)pool->num_pages, 0);
    if (!host_only) {
      lora_status st = kv_clear_table(device_page_table, (int64_t)max_seqs * max_pages);
      if (st != LORA_OK) return st;
    }
    *out = kv.release();
    return ok();
  });
}

extern "C" lora_status lora_kv_extend(lora_kv *kv, const int32_t *seqs, const int32_t *new_tokens, int32_t n,
                                      hipStream_t stream) {
  if (!kv) return fail(LORA_EINVAL, "null kv");
  if (n > 0 && !new_tokens) return fail(LORA_EINVAL, "null new_tokens");
  return guarded([&]() -> lora_status {
    lora_status st = check_ids(kv, seqs, n);
    if (st != LORA_OK) return st;
    const int64_t pt = kv->page_tokens;
    int64_t need = 0;
    std::vector<int32_t> to_copy;  // sequences whose last page the growth writes into and others hold too
    std::vector<std::pair<int32_t, int32_t>> left;  // (shared page, holders left after the copies before)
    for (int32_t i = 0; i < n; ++i) {
      const Seq &s = kv->seqs[(size_t)seqs[i]];
      const int64_t len = std::max(s.len, 0);
      if (new_tokens[i] < 0) return fail(LORA_EINVAL, "sequence %d grows by %d", seqs[i], new_tokens[i]);
      if (len + new_tokens[i] > pt * kv->max_pages)
        return fail(LORA_EINVAL, "sequence %d of %lld positions does not fit %d pages", seqs[i],
                    (long long)(len + new_tokens[i]), kv->max_pages);
      need += cdiv(len + new_tokens[i], pt) - (int64_t)s.pages.size();
      if (new_tokens[i] > 0 && len % pt && kv->refs[(size_t)s.pages.back()] > 1) {
        const int32_t page = s.pages.back();
        auto it = std::find_if(left.begin(), left.end(), [&](const std::pair<int32_t, int32_t> &q) { return q.first == page; });
        if (it == left.end()) it = left.insert(left.end(), {page, kv->refs[(size_t)page]});
        if (it->second > 1) {  // the last holder keeps the page
          --it->second;
          ++need;
          to_copy.push_back(seqs[i]);
        }
      }
    }
    int32_t free_pages = 0;
    lora_pool_num_free(kv->pool, &free_pages);
    if (need > (int64_t)kv->spares.size() + free_pages)
      return fail(LORA_ENOMEM, "%lld pages needed, the pool has %d and %zu are spare", (long long)need, free_pages,
                  kv->spares.size());
    if ((st = begin_device(kv, stream)) != LORA_OK) return st;
    // the pages, before anything changes: spares first (their readers are on this stream), then the pool's
    std::vector<int32_t> pages((size_t)need);
    const size_t from_spares = std::min((size_t)need, kv->spares.size());
    for (int32_t i = 0; i < n; ++i) {
      Seq &s = kv->seqs[(size_t)seqs[i]];
      s.pages.reserve((size_t)cdiv(std::max(s.len, 0) + (int64_t)new_tokens[i], pt));
    }
    Steps steps;
    steps.moves.reserve(to_copy.size());
    steps.entries.reserve((size_t)need);
    const size_t most = (size_t)(INT32_MAX / kv->pool->page_rows);  // the pool counts in rows
    for (size_t i = from_spares; i < (size_t)need; i += most) {
      st = lora_pool_alloc(kv->pool, (int32_t)std::min(most, (size_t)need - i) * kv->pool->page_rows, pages.data() + i);
      if (st != LORA_OK) return st;  // cannot happen after the count above
    }
    for (size_t i = 0; i < from_spares; ++i) {
      pages[i] = kv->spares.back().page;
      kv->spares.pop_back();
    }
    size_t at = 0;
    for (int32_t id : to_copy) {
      Seq &s = kv->seqs[(size_t)id];
      const int32_t from = s.pages.back(), to = pages[at++];
      steps.moves.push_back({from, to});
      steps.entries.push_back({entry(kv, id, s.pages.size() - 1), to});
      --kv->refs[(size_t)from];  // others hold it still
      kv->refs[(size_t)to] = 1;
      s.pages.back() = to;
    }
    for (int32_t i = 0; i < n; ++i) {
      Seq &s = kv->seqs[(size_t)seqs[i]];
      s.len = std::max(s.len, 0) + new_tokens[i];
      while ((int64_t)s.pages.size() * pt < s.len) {
        const int32_t p = pages[at++];
        kv->refs[(size_t)p] = 1;
        steps.entries.push_back({entry(kv, seqs[i], s.pages.size()), p});
        s.pages.push_back(p);
      }
    }
    if ((st = run_steps(kv, steps, stream)) != LORA_OK) return st;
    return ok();
  });
}

extern "C" lora_status lora_kv_fork(lora_kv *kv, int32_t src, const int32_t *dst, int32_t n, hipStream_t stream) {
  if (!kv) return fail(LORA_EINVAL, "null kv");
  return guarded([&]() -> lora_status {
    lora_status st = check_seq(kv, src);
    if (st == LORA_OK) st = check_ids(kv, dst, n);
    if (st != LORA_OK) return st;
    const Seq &s = kv->seqs[(size_t)src];
    if (s.len < 0) return fail(LORA_EINVAL, "sequence %d is not in use", src);
    for (int32_t i = 0; i < n; ++i)
      if (kv->seqs[(size_t)dst[i]].len >= 0) return fail(LORA_EINVAL, "sequence %d is in use", dst[i]);
    if ((st = begin_device(kv, stream)) != LORA_OK) return st;
    Steps steps;
    steps.entries.reserve((size_t)n * s.pages.size());
    std::vector<std::vector<int32_t>> copies((size_t)n, s.pages);
    for (int32_t i = 0; i < n; ++i) {
      Seq &d = kv->seqs[(size_t)dst[i]];
      d.len = s.len;
      d.pages.swap(copies[(size_t)i]);
      for (size_t p = 0; p < d.pages.size(); ++p) {
        ++kv->refs[(size_t)d.pages[p]];
        steps.entries.push_back({entry(kv, dst[i], p), d.pages[p]});
      }
    }
    if ((st = run_steps(kv, steps, stream)) != LORA_OK) return st;
    return ok();
  });
}

// Cuts each sequence to `keep` pages and sets its length.
static lora_status shorten(lora_kv *kv, const int32_t *seqs, int32_t n, int32_t new_len, hipStream_t stream) {
  lora_status st = begin_device(kv, stream);
  if (st != LORA_OK) return st;
  const size_t keep = (size_t)cdiv(std::max(new_len, 0), kv->page_tokens);
  size_t most = 0;
  for (int32_t i = 0; i < n; ++i) {
    const size_t have = kv->seqs[(size_t)seqs[i]].pages.size();
    most += have > keep ? have - keep : 0;
  }
  Steps steps;
  std::vector<int32_t> dropped;
  steps.entries.reserve(most);
  dropped.reserve(most);
  kv->spares.reserve(kv->spares.size() + most);
  for (int32_t i = 0; i < n; ++i) {
    Seq &s = kv->seqs[(size_t)seqs[i]];
    while (s.pages.size() > keep) {
      drop(kv, s.pages.back(), dropped);
      s.pages.pop_back();
      steps.entries.push_back({entry(kv, seqs[i], s.pages.size()), -1});
    }
    s.len = new_len;
  }
  make_spares(kv, dropped);
  if ((st = run_steps(kv, steps, stream)) != LORA_OK) return st;
  return ok();
}

extern "C" lora_status lora_kv_truncate(lora_kv *kv, int32_t seq, int32_t new_len, hipStream_t stream) {
  if (!kv) return fail(LORA_EINVAL, "null kv");
  return guarded([&]() -> lora_status {
    lora_status st = check_seq(kv, seq);
    if (st != LORA_OK) return st;
    const int32_t len = kv->seqs[(size_t)seq].len;
    if (len < 0) return fail(LORA_EINVAL, "sequence %d is not in use", seq);
    if (new_len < 0 || new_len > len) return fail(LORA_EINVAL, "sequence %d of %d positions cut to %d", seq, len, new_len);
    return shorten(kv, &seq, 1, new_len, stream);
  });
}

extern "C" lora_status lora_kv_free(lora_kv *kv, const int32_t *seqs, int32_t n, hipStream_t stream) {
  if (!kv) return fail(LORA_EINVAL, "null kv");
  return guarded([&]() -> lora_status {
    lora_status st = check_ids(kv, seqs, n);
    if (st != LORA_OK) return st;
    for (int32_t i = 0; i < n; ++i)
      if (kv->seqs[(size_t)seqs[i]].len < 0) return fail(LORA_EINVAL, "sequence %d is not in use", seqs[i]);
    return shorten(kv, seqs, n, -1, stream);
  });
}

extern "C" lora_status lora_kv_compact(lora_kv *kv, int32_t *moved, hipStream_t stream) {
  if (!kv || !moved) return fail(LORA_EINVAL, "null argument");
  *moved = 0;
  return guarded([&]() -> lora_status {
    lora_status st = begin_device(kv, stream);
    if (st != LORA_OK) return st;
    lora_pool *p = kv->pool;
    // lowest ids to move to (the pool's free ones and the spares), highest pages to move
    std::vector<uint8_t> open((size_t)p->num_pages, 0);
    for (size_t i = p->head; i < p->free_list.size(); ++i) open[(size_t)p->free_list[i]] = 1;
    for (const Spare &s : kv->spares) open[(size_t)s.page] = 2;
    std::vector<int32_t> to(kv->refs.size(), -1);
    Steps steps;
    for (int32_t lo = 0, hi = p->num_pages - 1;; ++lo, --hi) {
      while (lo < hi && !open[(size_t)lo]) ++lo;
      while (lo < hi && kv->refs[(size_t)hi] == 0) --hi;
      if (lo >= hi) break;
      steps.moves.push_back({hi, lo});
      to[(size_t)hi] = lo;
    }
    if (steps.moves.empty()) return ok();
    for (size_t s = 0; s < kv->seqs.size(); ++s)
      for (size_t i = 0; i < kv->seqs[s].pages.size(); ++i)
        if (to[(size_t)kv->seqs[s].pages[i]] >= 0)
          steps.entries.push_back({entry(kv, (int32_t)s, i), to[(size_t)kv->seqs[s].pages[i]]});
    std::vector<int32_t> left, dropped;
    left.reserve(p->free_list.size());
    dropped.reserve(steps.moves.size());
    kv->spares.reserve(kv->spares.size() + steps.moves.size());
    // from here on nothing allocates
    std::vector<uint8_t> &used = open;  // 3: now the target of a move
    for (const auto &m : steps.moves) used[(size_t)m.second] = 3;
    for (size_t i = p->head; i < p->free_list.size(); ++i)
      if (used[(size_t)p->free_list[i]] != 3) left.push_back(p->free_list[i]);
    p->free_list.swap(left);
    p->head = 0;
    kv->spares.erase(std::remove_if(kv->spares.begin(), kv->spares.end(), [&](const Spare &s) { return used[(size_t)s.page] == 3; }),
                     kv->spares.end());
    for (const auto &m : steps.moves) {
      p->taken[(size_t)m.second] = 1;
      kv->refs[(size_t)m.second] = kv->refs[(size_t)m.first];
      kv->refs[(size_t)m.first] = 0;
      dropped.push_back(m.first);
    }
    for (Seq &s : kv->seqs)
      for (int32_t &page : s.pages)
        if (to[(size_t)page] >= 0) page = to[(size_t)page];
    st = run_steps(kv, steps, stream);
    make_spares(kv, dropped);
    *moved = (int32_t)steps.moves.size();
    return st != LORA_OK ? st : ok();
  });
}

extern "C" lora_status lora_kv_trim(lora_kv *kv, int32_t wait, int32_t *left) {
  if (!kv) return fail(LORA_EINVAL, "null kv");
  return guarded([&]() -> lora_status {
    std::vector<int32_t> back;
    std::vector<Spare> kept;
    const auto unmarked = [](const Spare &s) { return !s.marked; };
    if (std::any_of(kv->spares.begin(), kv->spares.end(), unmarked)) {
      std::shared_ptr<void> mark;
      if (kv_not_capturing(kv->stream) == LORA_OK && try_mark(kv, &mark))
        for (Spare &s : kv->spares)
          if (!s.marked) s = {s.page, true, mark};
    }
    for (const Spare &s : kv->spares) {
      if (s.marked && (!s.mark || kv_mark_done(s.mark, wait != 0))) back.push_back(s.page);
      else kept.push_back(s);
    }
    lora_status st = lora_pool_free(kv->pool, back.data(), (int32_t)back.size());
    if (st != LORA_OK) return st;
    kv->spares.swap(kept);
    if (left) *left = (int32_t)kv->spares.size();
    return ok();
  });
}

extern "C" lora_status lora_kv_seq(const lora_kv *kv, int32_t seq, int32_t *length, int32_t *page_ids,
                                   int32_t *num_pages) {
  if (!kv) return fail(LORA_EINVAL, "null kv");
  lora_status st = check_seq(kv, seq);
  if (st != LORA_OK) return st;
  const Seq &s = kv->seqs[(size_t)seq];
  if (length) *length = s.len;
  if (num_pages) *num_pages = (int32_t)s.pages.size();
  if (page_ids) std::copy(s.pages.begin(), s.pages.end(), page_ids);
  return ok();
}

extern "C" lora_status lora_kv_get_stats(const lora_kv *kv, lora_kv_stats *out) {
  if (!kv || !out) return fail(LORA_EINVAL, "null argument");
  lora_kv_stats s{};
  s.highest = -1;
  s.page_tokens = kv->page_tokens;
  for (const Seq &q : kv->seqs) s.seqs += q.len >= 0;
  for (size_t p = 0; p < kv->refs.size(); ++p) {
    s.pages += kv->refs[p] > 0;
    s.shared += kv->refs[p] > 1;
    if (kv->refs[p] > 0) s.highest = (int32_t)p;
  }
  for (const Spare &q : kv->spares) s.highest = std::max(s.highest, q.page);
  s.spare = (int32_t)kv->spares.size();
  *out = s;
  return ok();
}

extern "C" lora_status lora_kv_get_view(const lora_kv *kv, lora_kv_view *view) {
  if (!kv || !view) return fail(LORA_EINVAL, "null argument");
  if (kv->host_only()) return fail(LORA_EINVAL, "a host-only cache has no device view");
  lora_kv_view v{};
  v.dtype = LORA_BF16;
  v.head_dim = kv->head_dim;
  v.kv_heads = kv->kv_heads;
  v.page_tokens = kv->page_tokens;
  v.num_pages = kv->pool->num_pages;
  v.num_seqs = (int32_t)kv->seqs.size();
  v.max_pages = kv->max_pages;
  v.k = kv->pool->storage;
  v.v = kv->pool->storage + (int64_t)kv->kv_heads * kv->page_tokens * kv->head_dim * 2;
  v.page_stride = (int64_t)kv->pool->page_rows * kv->pool->row_width;
  v.head_stride = (int64_t)kv->page_tokens * kv->head_dim;
  v.token_stride = kv->head_dim;
  v.page_table = kv->table;
  *view = v;
  return ok();
}

extern "C" void lora_kv_destroy(lora_kv *kv) {
  if (!kv) return;
  try {
    // A page goes back only once its readers are known to be done: behind a mark of the cache's stream for what
    // sequences hold, behind its own for a spare.  Where a wait fails, or memory for it, the page stays taken.
    std::vector<int32_t> back;
    bool any = false;
    for (int32_t r : kv->refs) any = any || r > 0;
    for (const Spare &s : kv->spares) any = any || !s.marked;
    std::shared_ptr<void> mark;
    const bool idle = kv->host_only() || (any && kv_not_capturing(kv->stream) == LORA_OK && try_mark(kv, &mark) &&
                                          kv_mark_done(mark, true));
    for (const Spare &s : kv->spares)
      if (s.marked ? !s.mark || kv_mark_done(s.mark, true) : idle) back.push_back(s.page);
    for (size_t p = 0; p < kv->refs.size(); ++p)
      if (kv->refs[p] > 0 && idle) back.push_back((int32_t)p);
    (void)lora_pool_free(kv->pool, back.data(), (int32_t)back.size());
  } catch (...) {
  }
  delete kv;
}
