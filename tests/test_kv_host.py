"""Host half of the paged KV cache and the argument checks of its device calls and of the 4-bit base
projection, without a GPU: the attention planner's coverage, the sequence bookkeeping against a restated
model, refusals."""
import ctypes
import math

import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B
from segmented_gather_gemm_segments_amd import build as lbuild


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    if not lbuild.up_to_date():
        lbuild.build()
    return B.lib()


def refused(status, call):
    with pytest.raises(B.LoraError) as e:
        call()
    assert e.value.status == status, str(e.value)


# ---------------------------------------------------------------- attention planner
def kept(q_len, kv_len, i, causal, window):
    p = kv_len - q_len + i
    lo = max(0, p - window + 1) if window else 0
    hi = min(p, kv_len - 1) if causal else kv_len - 1
    return lo, hi + 1


@pytest.mark.parametrize("trial", range(60))
def test_plan_covers_every_kept_position_once(trial):
    rng = np.random.default_rng(trial)
    kv_heads, group = int(rng.integers(1, 9)), int(rng.choice([1, 2, 3, 5, 8, 16, 40]))
    n = int(rng.integers(0, 9))
    q_lens = [int(rng.choice([0, 1, 1, 2, 17, 200])) for _ in range(n)]
    kv_lens = [int(rng.choice([0, 1, 63, 64, 65, 700, 3000])) for _ in range(n)]
    causal, window = bool(rng.integers(0, 2)), int(rng.choice([0, 0, 1, 30, 500]))
    max_parts = int(rng.choice([0, 1, 2, 5, 64]))
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    plan = B.lora_kv_attn_plan(starts, range(n), kv_lens, kv_heads * group, kv_heads, 64, causal, window, max_parts)
    d, items = plan.desc, plan.host_items
    assert items.shape == (d.num_row_items + d.num_tile_items + d.num_joins, 8)
    main, joins = items[: d.num_row_items + d.num_tile_items], items[d.num_row_items + d.num_tile_items:]
    seen, final, part_rows, slots = {}, {}, {}, np.zeros(d.num_part_rows, int)
    for k, (qb, row0, rows, seq, pos0, b, e, part) in enumerate(main.tolist()):
        limit = B.LORA_ATTN_ROWS if k < d.num_row_items else B.LORA_ATTN_TILE_ROWS
        assert 1 <= rows <= limit and qb == starts[seq] and pos0 == kv_lens[seq] - q_lens[seq]
        assert 0 <= b <= e <= kv_lens[seq]
        if part >= 0:
            slots[part: part + rows] += 1
            part_rows[(seq, row0, part)] = rows
        for r in range(row0, row0 + rows):
            seen.setdefault((seq, r), []).append((b, e))
            if part < 0:
                final[(seq, r)] = final.get((seq, r), 0) + 1
    assert np.all(slots == 1)  # every slot written by one item
    for qb, row0, rows, seq, pos0, base, _, parts in joins.tolist():
        assert 2 <= parts <= (max_parts or B.LORA_ATTN_MAX_PARTS)
        for p in range(parts):
            assert part_rows.pop((seq, row0, base + p * rows)) == rows
        for r in range(row0, row0 + rows):
            final[(seq, r)] = final.get((seq, r), 0) + 1
    assert not part_rows
    for s in range(n):
        for r in range(q_lens[s] * group):
            assert final[(s, r)] == 1
            lo, hi = kept(q_lens[s], kv_lens[s], r // group, causal, window)
            at = lo  # the ranges, in order, leave no kept position out and none twice
            for b, e in sorted(seen[(s, r)]):
                if hi > lo:
                    assert b <= at or e <= at
                    at = max(at, e)
            assert hi <= lo or at >= hi
            spans = sorted(x for x in seen[(s, r)] if x[0] < x[1])
            assert all(x[1] <= y[0] for x, y in zip(spans, spans[1:]))
    assert len(final) == int(starts[-1]) * group
    assert d.workspace_bytes >= d.num_part_rows * kv_heads * 65 * 4
    if max_parts == 1:
        assert d.num_joins == 0 and d.workspace_bytes == 0
    # heaviest first
    for part in (main[: d.num_row_items], main[d.num_row_items:]):
        assert np.all(np.diff(part[:, 6] - part[:, 5]) <= 0)


def test_plan_long_positions():
    """Lengths near 2^31 neither wrap nor blow the plan up."""
    big = 2**31 - 1
    plan = B.lora_kv_attn_plan([0, 1, 3], [0, 1], [big, 7], 8, 1, 128)
    main = plan.host_items[: plan.desc.num_row_items + plan.desc.num_tile_items]
    assert int(main[:, 6].max()) == big and plan.desc.num_joins == 1
    spans = sorted((int(b), int(e)) for _, _, _, s, _, b, e, _ in main.tolist() if s == 0)
    assert spans[0][0] == 0 and spans[-1][1] == big and all(x[1] == y[0] for x, y in zip(spans, spans[1:]))


def test_plan_refusals():
    ok = dict(q_starts=[0, 1], seqs=[0], kv_lens=[4], q_heads=4, kv_heads=2, head_dim=64)
    B.lora_kv_attn_plan(**ok)
    for status, change in [
            (B.LORA_EINVAL, dict(q_starts=[1, 2])), (B.LORA_EINVAL, dict(q_starts=[0, -1])),
            (B.LORA_EINVAL, dict(q_starts=[0, 1, 2])), (B.LORA_EINVAL, dict(q_starts=[])),
            (B.LORA_EINVAL, dict(q_heads=5)), (B.LORA_EINVAL, dict(kv_heads=0)), (B.LORA_EINVAL, dict(q_heads=0)),
            (B.LORA_EUNSUPPORTED, dict(head_dim=0)), (B.LORA_EUNSUPPORTED, dict(head_dim=12)),
            (B.LORA_EUNSUPPORTED, dict(head_dim=264)), (B.LORA_EINVAL, dict(window=-1)),
            (B.LORA_EINVAL, dict(max_parts=-1)), (B.LORA_EINVAL, dict(max_parts=65)),
            (B.LORA_ERANGE, dict(seqs=[-1])), (B.LORA_ERANGE, dict(seqs=[3], num_seqs=3)),
            (B.LORA_ERANGE, dict(kv_lens=[-1])), (B.LORA_ERANGE, dict(kv_lens=[33], max_kv=32))]:
        refused(status, lambda: B.lora_kv_attn_plan(**{**ok, **change}))
    p = B.lora_attn_plan()
    one = np.zeros(8, np.int32)
    st, sq, kv = (np.array(a, np.int32) for a in ([0, 40], [0], [4]))
    args = (st.ctypes.data, sq.ctypes.data, kv.ctypes.data, 1, 1, 64, 4, 2, 64)
    assert B.lib().lora_kv_attn_plan(*args, 2, 0, 0, ctypes.byref(p), None, 0) == B.LORA_EINVAL  # flags
    assert B.lib().lora_kv_attn_plan(*args, 1, 0, 0, ctypes.byref(p), one.ctypes.data, 0) == B.LORA_ENOMEM
    assert p.num_row_items + p.num_tile_items >= 1
    assert B.lib().lora_kv_attn_plan(*args, 1, 0, 0, None, None, 0) == B.LORA_EINVAL


# ---------------------------------------------------------------- sequences
class HostPool(B.Pool):
    """A pool whose storage is never touched."""

    def __init__(self, pages, rows=16, width=64, seed=0, dtype=B.LORA_BF16, wfmt=B.LORA_WFMT_PLAIN):
        h = ctypes.c_void_p()
        self._keep = (ctypes.c_char * 64)()
        sc = ctypes.addressof(self._keep) if wfmt else None
        assert B.lib().lora_pool_create(pages, rows, width, dtype, wfmt, 4096, sc, seed, ctypes.byref(h)) == B.LORA_OK
        self._h, self.page_rows, self.pages_total = h, rows, pages


def cache(pool, seqs=6, pages=8, heads=2, dim=32):
    return B.KvCache(pool, heads, dim, seqs, pages, host_only=True)


@pytest.mark.parametrize("seed", range(25))
def test_sequences_against_a_model(seed):
    """Random growth, forks, cuts, frees, compactions and trims against sets of pages: shared pages are
    exactly the common whole history, no page is held by strangers, and every page is accounted for."""
    rng = np.random.default_rng(seed)
    pool = HostPool(60, seed=seed)
    other = pool.alloc(16 * 7).tolist()  # adapters in the same pool
    kv, P = cache(pool), 8
    tags = {}     # sequence -> list of tags, one per position (equal tags: written once, shared by a fork)
    data = {}     # page -> list of P tags
    n = 0
    for step in range(150):
        op = rng.random()
        live = sorted(tags)
        if op < 0.45:
            ids = rng.permutation(6)[: int(rng.integers(1, 4))].tolist()
            counts = [int(rng.integers(0, 14)) for _ in ids]
            before = {s: kv.pages(s).tolist() for s in range(6)}
            try:
                kv.extend(ids, counts)
            except B.LoraError as e:
                assert e.status in (B.LORA_ENOMEM, B.LORA_EINVAL)
                if e.status == B.LORA_EINVAL:
                    assert any(len(tags.get(s, [])) + c > 64 for s, c in zip(ids, counts))
                assert {s: kv.pages(s).tolist() for s in range(6)} == before
                continue
            # a copied page carries its contents over
            for s in ids:
                old, new = before[s], kv.pages(s).tolist()
                for a, b in zip(old, new):
                    if a != b:
                        data[b] = list(data[a])
                for p in new[len(old):]:
                    data[p] = [None] * P
            for s, c in zip(ids, counts):
                seq = tags.setdefault(s, [])
                for _ in range(c):
                    n += 1
                    data[int(kv.pages(s)[len(seq) // P])][len(seq) % P] = n
                    seq.append(n)
        elif op < 0.6 and live:
            src = int(rng.choice(live))
            free = [s for s in range(6) if s not in tags][: int(rng.integers(1, 3))]
            if free:
                kv.fork(src, free)
                for s in free:
                    tags[s] = list(tags[src])
        elif op < 0.7 and live:
            s = int(rng.choice(live))
            cut = int(rng.integers(0, len(tags[s]) + 1))
            kv.truncate(s, cut)
            tags[s] = tags[s][:cut]
        elif op < 0.8 and live:
            gone = [int(s) for s in rng.permutation(live)[: int(rng.integers(1, 3))]]
            kv.free(gone)
            for s in gone:
                del tags[s]
        elif op < 0.9:
            before = {s: kv.pages(s).tolist() for s in tags}
            moved = kv.compact()
            pairs = {a: b for s in tags for a, b in zip(before[s], kv.pages(s).tolist()) if a != b}
            assert len(pairs) == moved and not set(pairs) & set(pairs.values())
            assert all(b < a for a, b in pairs.items()) and not set(pairs.values()) & set(other)
            data.update({b: list(data[a]) for a, b in pairs.items()})
            held = {p for s in tags for p in kv.pages(s).tolist()}
            if held:  # nothing lower is left for the highest page
                assert all(p in held or p in other for p in range(max(held)))
        else:
            kv.trim(wait=bool(rng.integers(0, 2)))
            assert kv.stats()["spare"] == 0
        # every sequence reads back what it holds
        holders = {}
        for s in range(6):
            assert kv.length(s) == (len(tags[s]) if s in tags else -1)
            pages = kv.pages(s).tolist()
            assert len(pages) == math.ceil(len(tags.get(s, [])) / P)
            for i, tag in enumerate(tags.get(s, [])):
                assert data[pages[i // P]][i % P] == tag, (step, s, i)
            for p in pages:
                holders.setdefault(p, []).append(s)
        st = kv.stats()
        assert not set(holders) & set(other)
        assert st["pages"] == len(holders) and st["shared"] == sum(len(v) > 1 for v in holders.values())
        assert st["seqs"] == len(tags) and pool.num_free() + st["pages"] + st["spare"] + len(other) == 60
    kv.close()
    assert pool.num_free() == 60 - len(other)
    pool.free(other)  # still the other user's


def test_all_or_nothing_and_last_holder():
    pool = HostPool(4)
    kv = cache(pool)
    kv.extend([0], [12])            # 2 pages, the second half full
    kv.fork(0, [1, 2])
    refused(B.LORA_ENOMEM, lambda: kv.extend([0, 1, 2], [9, 9, 9]))
    assert kv.stats()["pages"] == 2 and pool.num_free() == 2
    kv.extend([0, 1, 2], [1, 1, 1])  # two copies, the last holder writes in place
    assert pool.num_free() == 0 and kv.stats()["shared"] == 1
    assert len({int(kv.pages(s)[1]) for s in range(3)}) == 3
    kv.free([0])
    assert kv.stats()["spare"] == 1 and pool.num_free() == 0
    kv.extend([1], [5])             # takes the spare
    assert kv.stats()["spare"] == 0


def test_a_pool_that_goes_first_takes_its_caches_along():
    pool = HostPool(8)
    kv, gone = cache(pool), cache(pool)
    kv.extend([0], [9])
    gone.extend([0], [3])
    gone.close()
    assert pool.num_free() == 6
    pool.close()
    refused(B.LORA_EINVAL, lambda: kv.extend([0], [1]))
    kv.close()


def test_sequence_refusals():
    pool = HostPool(8)
    for kw, status in [(dict(kv_heads=0), B.LORA_EINVAL), (dict(head_dim=12), B.LORA_EUNSUPPORTED),
                       (dict(head_dim=264), B.LORA_EUNSUPPORTED), (dict(max_seqs=0), B.LORA_EINVAL),
                       (dict(max_pages=0), B.LORA_EINVAL), (dict(kv_heads=17, head_dim=32), B.LORA_EUNSUPPORTED)]:
        args = {**dict(kv_heads=2, head_dim=32, max_seqs=2, max_pages=2), **kw}
        refused(status, lambda: B.KvCache(pool, host_only=True, **args))
    refused(B.LORA_EUNSUPPORTED, lambda: cache(HostPool(8, dtype=B.LORA_F32)))
    refused(B.LORA_EUNSUPPORTED, lambda: cache(HostPool(8, wfmt=B.LORA_WFMT_INT4)))
    refused(B.LORA_EUNSUPPORTED, lambda: B.KvCache(pool, 2, 32, 1, 2**29, host_only=True))
    h = ctypes.c_void_p()
    assert B.lib().lora_kv_create(pool._h, 2, 32, 2, 2, None, 0, ctypes.byref(h)) == B.LORA_EINVAL  # no table
    assert B.lib().lora_kv_create(pool._h, 2, 32, 2, 2, 16, 2, ctypes.byref(h)) == B.LORA_EINVAL    # flags
    kv = cache(pool, seqs=3, pages=3)
    kv.extend([0], [10])
    refused(B.LORA_ERANGE, lambda: kv.extend([3], [1]))
    refused(B.LORA_ERANGE, lambda: kv.extend([-1], [1]))
    refused(B.LORA_EINVAL, lambda: kv.extend([1, 1], [1, 1]))
    refused(B.LORA_EINVAL, lambda: kv.extend([1], [-1]))
    refused(B.LORA_EINVAL, lambda: kv.extend([0], [15]))
    refused(B.LORA_EINVAL, lambda: kv.extend([0], [2**31 - 1]))
    refused(B.LORA_EINVAL, lambda: kv.extend([0, 1], [1]))
    refused(B.LORA_EINVAL, lambda: kv.fork(1, [2]))
    refused(B.LORA_EINVAL, lambda: kv.fork(0, [0]))
    refused(B.LORA_EINVAL, lambda: kv.fork(0, [1, 1]))
    refused(B.LORA_ERANGE, lambda: kv.fork(0, [7]))
    refused(B.LORA_EINVAL, lambda: kv.truncate(0, 11))
    refused(B.LORA_EINVAL, lambda: kv.truncate(0, -1))
    refused(B.LORA_EINVAL, lambda: kv.truncate(1, 0))
    refused(B.LORA_EINVAL, lambda: kv.free([1]))
    refused(B.LORA_EINVAL, lambda: kv.free([0, 0]))
    refused(B.LORA_ERANGE, lambda: kv.length(5))
    assert kv.length(0) == 10 and kv.stats()["pages"] == 2 and pool.num_free() == 6
    v = B.lora_kv_view()
    assert B.lib().lora_kv_get_view(kv._h, ctypes.byref(v)) == B.LORA_EINVAL


# ---------------------------------------------------------------- refusals of the device calls (nothing is launched)
def view(**kw):
    d = dict(dtype=B.LORA_BF16, head_dim=64, kv_heads=2, page_tokens=16, num_pages=4, num_seqs=1, max_pages=4, reserved=0,
             k=4096, v=8192, page_stride=4096, head_stride=1024, token_stride=64, page_table=64)
    d.update(kw)
    return B.lora_kv_view(**d)


BAD_VIEWS = [(dict(dtype=B.LORA_F32), B.LORA_EUNSUPPORTED), (dict(head_dim=0), B.LORA_EUNSUPPORTED),
             (dict(head_dim=60), B.LORA_EUNSUPPORTED), (dict(head_dim=512), B.LORA_EUNSUPPORTED),
             (dict(kv_heads=0), B.LORA_EINVAL), (dict(page_tokens=0), B.LORA_EINVAL), (dict(num_pages=-1), B.LORA_EINVAL),
             (dict(k=None), B.LORA_EINVAL), (dict(v=None), B.LORA_EINVAL), (dict(page_table=None), B.LORA_EINVAL),
             (dict(k=4100), B.LORA_EINVAL), (dict(page_stride=4), B.LORA_EINVAL), (dict(token_stride=-8), B.LORA_EINVAL),
             (dict(max_pages=2**28), B.LORA_EUNSUPPORTED)]


def test_append_refusals():
    def call(v, k=16, vv=16, ts=128, hs=64, seq=16, pos=16, n=1):
        return B.lib().lora_kv_append(ctypes.byref(v) if v is not None else None, k, vv, ts, hs, seq, pos, n, None)
    for kw, status in BAD_VIEWS:
        assert call(view(**kw)) == status, kw
    assert call(None) == B.LORA_EINVAL
    for kw in (dict(k=None), dict(vv=None), dict(seq=None), dict(pos=None), dict(k=8), dict(seq=2), dict(ts=4),
               dict(hs=-8), dict(n=-1)):
        assert call(view(), **kw) == B.LORA_EINVAL, kw
    assert call(view(), n=0) == B.LORA_OK
    assert call(view(num_pages=0)) == B.LORA_OK


def test_attention_refusals():
    plan = B.lora_kv_attn_plan([0, 1], [0], [4], 4, 2, 64).desc
    split = B.lora_kv_attn_plan([0, 1], [0], [9000], 4, 2, 64).desc
    assert split.workspace_bytes > 0

    def call(v, p, items=16, q=16, qt=256, qh=64, o=16, ot=256, oh=64, lse=None, scale=0.1, ws=None, wb=0):
        return B.lib().lora_kv_attn(ctypes.byref(v) if v is not None else None, ctypes.byref(p) if p is not None else None,
                                    items, q, qt, qh, o, ot, oh, lse, scale, ws, wb, None)
    for kw, status in BAD_VIEWS:
        assert call(view(**kw), plan) == status, kw
    assert call(None, plan) == B.LORA_EINVAL and call(view(), None) == B.LORA_EINVAL
    assert call(view(kv_heads=1), plan) == B.LORA_EINVAL and call(view(head_dim=128), plan) == B.LORA_EINVAL
    for kw in (dict(items=None), dict(q=None), dict(o=None), dict(q=8), dict(o=8), dict(items=8), dict(lse=2),
               dict(qt=4), dict(oh=-8), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(view(), plan, **kw) == B.LORA_EINVAL, kw
    for kw in (dict(), dict(ws=16, wb=split.workspace_bytes - 4), dict(ws=8, wb=1 << 30), dict(wb=1 << 30)):
        assert call(view(), split, **kw) == B.LORA_EINVAL, kw
    for field, value in (("q_heads", 0), ("q_heads", 3), ("num_row_items", -1), ("num_joins", 2**30), ("window", -1),
                         ("flags", 6), ("num_part_rows", -1)):
        bad = B.lora_attn_plan()
        ctypes.memmove(ctypes.byref(bad), ctypes.byref(plan), ctypes.sizeof(plan))
        setattr(bad, field, value)
        assert call(view(), bad) == B.LORA_EINVAL, field
    empty = B.lora_kv_attn_plan([0], [], [], 4, 2, 64).desc
    assert call(view(), empty, items=None, q=None, o=None) == B.LORA_OK


def test_page_refusals():
    f = B.lib().lora_pages_copy
    assert f(16, 32, 4, 16, 16, 0, None) == B.LORA_OK
    for args in ((None, 32, 4, 16, 16, 1), (16, 0, 4, 16, 16, 1), (16, 24, 4, 16, 16, 1), (16, 32, -1, 16, 16, 1),
                 (16, 32, 4, None, 16, 1), (16, 32, 4, 16, None, 1), (16, 32, 4, 16, 16, -1), (8, 32, 4, 16, 16, 1)):
        assert f(*args, None) == B.LORA_EINVAL, args
    assert f(16, 2**40, 4, 16, 16, 64, None) == B.LORA_EUNSUPPORTED
    g = B.lib().lora_page_table_remap
    assert g(None, 0, None, None, 0, None) == B.LORA_OK
    for args in ((None, 4, 16, 16, 1), (16, 4, None, 16, 1), (16, 4, 16, None, 1), (16, -1, 16, 16, 1), (16, 4, 16, 16, -1),
                 (16, 4, 18, 16, 1)):
        assert g(*args, None) == B.LORA_EINVAL, args


def test_w4_refusals():
    def call(m=1, n=16, k=128, group=128, sd=B.LORA_BF16, codes=16, scales=16, zeros=None, x=16, xs=128, y=16, ys=16,
             dtype=B.LORA_BF16):
        w = B.lora_w4_weights(n, k, group, sd, codes, scales, zeros)
        return B.lib().lora_base_w4(dtype, m, ctypes.byref(w), x, xs, y, ys, None)
    assert call(m=0) == B.LORA_OK
    for kw in (dict(m=-1), dict(n=0), dict(k=0), dict(codes=None), dict(scales=None), dict(x=None), dict(y=None),
               dict(codes=8), dict(scales=8), dict(zeros=8), dict(x=8), dict(y=8), dict(xs=120), dict(ys=8), dict(xs=132),
               dict(ys=20)):
        assert call(**kw) == B.LORA_EINVAL, kw
    for kw in (dict(dtype=B.LORA_F32), dict(n=12, ys=16), dict(group=16), dict(group=256, k=256, xs=256),
               dict(k=96, group=64), dict(sd=2)):
        assert call(**kw) == B.LORA_EUNSUPPORTED, kw
    assert B.lib().lora_base_w4(B.LORA_BF16, 1, None, 16, 8, 16, 8, None) == B.LORA_EINVAL
    assert B.lora_w4_bytes(17, 129) == 4 * 1024
    refused(B.LORA_EINVAL, lambda: B.lora_w4_bytes(0, 128))
    f = B.lib().lora_w4_pack
    for args, status in (((8, 32, 0, None, 16), B.LORA_EINVAL), ((8, 32, 2, 16, 16), B.LORA_EINVAL),
                         ((8, 32, 0, 16, 8), B.LORA_EINVAL), ((12, 32, 0, 16, 16), B.LORA_EUNSUPPORTED),
                         ((8, 48, 0, 16, 16), B.LORA_EUNSUPPORTED), ((8, 0, 0, 16, 16), B.LORA_EINVAL)):
        assert f(*args, None) == status, args


def test_binding_refuses_tensors_it_cannot_pass_on():
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    codes = torch.zeros((1, 1, 64, 16), dtype=torch.uint8)
    refused(B.LORA_EINVAL, lambda: B.W4Weights(16, 128, 128, codes, torch.ones((1, 16), dtype=torch.float16)))
    refused(B.LORA_EINVAL, lambda: B.W4Weights(16, 128, 128, codes, torch.ones((1, 8))))
    refused(B.LORA_EINVAL, lambda: B.W4Weights(32, 128, 128, codes, torch.ones((1, 32))))
    refused(B.LORA_EINVAL, lambda: B.W4Weights(16, 128, 128, codes, torch.ones((1, 16)), torch.ones((1, 16), dtype=bf)))
    w = B.W4Weights(16, 128, 128, codes, torch.ones((1, 16)))
    refused(B.LORA_EINVAL, lambda: B.lora_base_w4(torch.zeros((1, 64), dtype=bf), w, torch.zeros((1, 16), dtype=bf)))
    refused(B.LORA_EINVAL, lambda: B.lora_base_w4(torch.zeros((1, 128)), w, torch.zeros((1, 16), dtype=bf)))
    # host tensors are not device tensors
    refused(B.LORA_EINVAL, lambda: B.lora_base_w4(torch.zeros((1, 128), dtype=bf), w, torch.zeros((1, 16), dtype=bf)))
    k = torch.zeros((4, 2, 16, 64), dtype=bf)
    table = torch.zeros((1, 4), dtype=i32)
    refused(B.LORA_EINVAL, lambda: B.KvView(k, k.float(), table))
    refused(B.LORA_EINVAL, lambda: B.KvView(k, k.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), table))
    refused(B.LORA_EINVAL, lambda: B.KvView(k, k, table.long()))
    refused(B.LORA_EINVAL, lambda: B.KvView(k[..., ::2], k[..., ::2], table))
    v = B.KvView(k, k, table)
    plan = B.lora_kv_attn_plan([0, 1], [0], [4], 4, 2, 64)
    q = torch.zeros((1, 4, 64), dtype=bf)
    refused(B.LORA_EINVAL, lambda: B.lora_kv_attn(v, plan, q, q.clone()))  # not uploaded
    plan.to("cpu")
    for bad_q, lse in ((q[:, :2], None), (q.float(), None), (q[:0], None), (q, torch.zeros((1, 3))), (q, torch.zeros((0, 4)))):
        refused(B.LORA_EINVAL, lambda: B.lora_kv_attn(v, plan, bad_q, bad_q.clone(), lse=lse))
    refused(B.LORA_EINVAL, lambda: B.lora_kv_attn(v, plan, q, q.clone()))  # on the host
    new = torch.zeros((3, 2, 64), dtype=bf)
    ids = torch.zeros(3, dtype=i32)
    for a in ((new[:, :1], new, ids, ids), (new, new[:2], ids, ids), (new, new, ids[:2], ids), (new, new, ids, ids.long()),
              (new, new, ids, ids)):
        refused(B.LORA_EINVAL, lambda: B.lora_kv_append(v, *a))
    refused(B.LORA_EINVAL, lambda: B.lora_pages_copy(k, ids, ids[:2]))
    refused(B.LORA_EINVAL, lambda: B.lora_page_table_remap(ids, table, ids))


def test_a_plan_past_the_view_is_refused():
    torch = pytest.importorskip("torch")
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    v = B.KvView(k, k, torch.zeros((2, 3), dtype=torch.int32))  # 2 sequences of up to 48 positions
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    for seqs, lens, parts, status in (([0, 1], [48, 0], 0, B.LORA_EINVAL),  # fits: refused as a host tensor only
                                      ([0, 2], [4, 4], 0, B.LORA_ERANGE), ([0, 1], [4, 49], 0, B.LORA_ERANGE),
                                      ([0, 1], [4, 9000], 5, B.LORA_ERANGE), ([5, 0], [0, 4], 0, B.LORA_ERANGE)):
        plan = B.lora_kv_attn_plan([0, 1, 2], seqs, lens, 4, 2, 64, max_parts=parts).to("cpu")
        refused(status, lambda: B.lora_kv_attn(v, plan, q, q.clone()))


def test_a_view_without_pages_still_needs_its_table():
    """Attention looks positions up in the page table before it knows that no page exists."""
    plan = B.lora_kv_attn_plan([0, 1], [0], [4], 4, 2, 64).desc
    for v in (view(num_pages=0, page_table=None), view(num_pages=0, page_table=None, k=None, v=None)):
        assert B.lib().lora_kv_attn(ctypes.byref(v), ctypes.byref(plan), 16, 16, 256, 64, 16, 256, 64, None, 0.1, None, 0,
                                    None) == B.LORA_EINVAL
        assert B.lib().lora_kv_append(ctypes.byref(v), 16, 16, 128, 64, 16, 16, 1, None) == B.LORA_EINVAL
    for change in (dict(num_seqs=0), dict(max_pages=0)):  # nothing to look up
        v = view(page_table=None, k=None, v=None, **change)
        assert B.lib().lora_kv_append(ctypes.byref(v), 16, 16, 128, 64, 16, 16, 1, None) == B.LORA_OK


def test_calls_too_large_for_a_launch():
    """A launch has fewer than 2^32 threads: what needs more is refused before it fails on the device."""
    f, g = B.lib().lora_pages_copy, B.lib().lora_page_table_remap
    for args in ((16, 16, 4, 16, 16, 2**24), (16, 2**20, 4, 16, 16, 2**16), (16, 2**36, 4, 16, 16, 1)):
        assert f(*args, None) == B.LORA_EUNSUPPORTED, args
    assert g(16, 4, 16, 16, 2**32, None) == B.LORA_EUNSUPPORTED
    v = view()  # 16 units of 16 bytes a token
    assert B.lib().lora_kv_append(ctypes.byref(v), 16, 16, 128, 64, 16, 16, 2**28, None) == B.LORA_EUNSUPPORTED
    # a page that no launch could copy when a shared one is written
    refused(B.LORA_EUNSUPPORTED, lambda: B.KvCache(HostPool(2, rows=2**20, width=2**15), 256, 256, 1, 1, host_only=True))
    B.KvCache(HostPool(2, rows=2**20, width=2**14), 256, 256, 1, 1, host_only=True).close()
    plan = B.lora_kv_attn_plan([0, 1], [0], [4], 4, 2, 64).desc
    for field, n in (("num_row_items", 2**23), ("num_tile_items", 2**23), ("num_joins", 2**21)):
        bad = B.lora_attn_plan()
        ctypes.memmove(ctypes.byref(bad), ctypes.byref(plan), ctypes.sizeof(plan))
        setattr(bad, field, n)
        assert B.lib().lora_kv_attn(ctypes.byref(v), ctypes.byref(bad), 16, 16, 256, 64, 16, 256, 64, None, 0.1, None, 0,
                                    None) == B.LORA_EUNSUPPORTED, field


def test_w4_sizes_that_the_kernels_cannot_count():
    """Row and column counts near 2^31 would wrap in the kernels' 32-bit indexes."""
    def base(n, k, group=32):
        w = B.lora_w4_weights(n, k, group, B.LORA_BF16, 16, 16, None)
        return B.lib().lora_base_w4(B.LORA_BF16, 1, ctypes.byref(w), 16, k, 16, n, None)
    for n, k in ((2**31 - 8, 32), (2**26 + 8, 32), (8, 2**31 - 32), (8, 2**24 + 32)):
        assert base(n, k) == B.LORA_EUNSUPPORTED, (n, k)
        assert B.lib().lora_w4_pack(n, k, 0, 16, 16, None) == B.LORA_EUNSUPPORTED, (n, k)
    assert B.lib().lora_w4_pack(2**26, 512, 0, 16, 16, None) == B.LORA_EUNSUPPORTED  # codes of 2^32 words


def test_objects_left_at_the_interpreters_end(monkeypatch):
    """By then a module's names may be None: what is left of its objects goes without an error."""
    pool = HostPool(8)
    kv = cache(pool)
    for name in ("_close_later", "LoraError", "_capturing", "_kv_destroy"):
        with monkeypatch.context() as m:
            m.setattr(B, name, None)
            kv.__del__()
            pool.__del__()
    kv.close()
