"""A step, draft or accepted path that is refused leaves the serving block's cache as it was, without a GPU: limits that are known
before are met before a sequence grows, and what raises after that takes the growth back."""
import ctypes

import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B
from segmented_gather_gemm_segments_amd import build as lbuild

torch = pytest.importorskip("torch")
HEADS, DIM, WIDTH = 2, 32, 128


@pytest.fixture(scope="module", autouse=True)
def library():
    if not lbuild.up_to_date():
        lbuild.build()
    return B.lib()


class HostPool:
    def __init__(self, pages, page_rows=16):
        self._h, self._kv_handles, self.storage = ctypes.c_void_p(), [], np.zeros((pages, page_rows, WIDTH), np.uint16)
        B._check(B.lib().lora_pool_create(pages, page_rows, WIDTH, B.LORA_BF16, B.LORA_WFMT_PLAIN, self.storage.ctypes.data, None, 0,
                                          ctypes.byref(self._h)))


class Block:
    """A serving block over a cache that only keeps its books; the device calls are recorded."""

    def __new__(cls, monkeypatch, max_pages=8, bounds=True, pool_pages=24):
        from segmented_gather_gemm_segments_amd import runner as R
        b = object.__new__(R.ServingBlock)
        b.device, b.d_model, b.head_dim, b.q_heads, b.kv_heads = torch.device("cpu"), WIDTH, DIM, 4, HEADS
        b._drafts = {}
        b.kv = B.KvCache(HostPool(pool_pages), HEADS, DIM, 4, max_pages, host_only=True, bounds=bounds)
        tokens = b.kv.stats()["page_tokens"]
        k = torch.zeros((pool_pages, HEADS, tokens, DIM), dtype=torch.bfloat16)
        b.kv.view = B.KvView(k, k.clone(), torch.zeros((4, max_pages), dtype=torch.int32))
        if bounds:
            b.kv.bounds = B.KvBounds(b.kv.view, torch.zeros((pool_pages, HEADS, B.lora_kv_bounds_row_bytes(DIM)), dtype=torch.uint8))
        b.page, b.calls, b.fails = tokens, [], None
        for name in ("lora_kv_keep_path", "lora_kv_bounds_update"):
            monkeypatch.setattr(B, name, lambda *args, _name=name, **kw: b.calls.append((_name, args)))

        def run(hidden, seq, pos, ids, ranges, attend):
            b.calls.append(("run", (seq, pos, ranges)))
            if b.fails:
                raise b.fails
            return hidden
        b._run = run
        monkeypatch.setattr(B, "_On", lambda *args: __import__("contextlib").nullcontext())
        return b


def state(b):
    return [b.kv.length(s) for s in range(4)], [b.kv.pages(s).tolist() for s in range(4)], dict(b._drafts), b.kv.stats()["pages"]


def rows(t):
    return torch.zeros((t, WIDTH), dtype=torch.bfloat16)


def ids(t):
    return torch.zeros(t, dtype=torch.int32)


def grow(b, seqs, new):
    return b.step(rows(sum(new)), seqs, new, ids(sum(new)))


def refused(b, status, call, *args, **kw):
    before, calls = state(b), len(b.calls)
    with pytest.raises(B.LoraError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    assert state(b) == before and len(b.calls) == calls


def test_more_pages_than_a_selection_takes(monkeypatch):
    b = Block(monkeypatch, max_pages=B.LORA_BLOCKS_MAX_PAGES + 1)
    grow(b, [0, 1], [b.page + 3, 2])
    b.draft(rows(2), [1], [[-1, 0]], ids(2))
    for seqs, new in (([0], [1]), ([0, 1], [2, 3]), ([2], [4])):
        refused(b, B.LORA_EUNSUPPORTED, b.step, rows(sum(new)), seqs, new, ids(sum(new)), pages=4)
    b.accept([1], [[0]])
    assert b.kv.length(1) == 3


def test_more_tokens_than_a_selection_takes(monkeypatch):
    """2^22 lists of a wide table (the count alone: a view of so many heads is never run)."""
    b = Block(monkeypatch, max_pages=3000)
    b.kv.view.desc.kv_heads = 1 << 21
    b.kv.bounds.heads = (1 << 21, DIM)
    refused(b, B.LORA_EUNSUPPORTED, b.step, rows(2), [0], [2], ids(2), pages=4)


def test_more_bounds_than_a_launch_takes(monkeypatch):
    b = Block(monkeypatch)
    b.kv.view.desc.kv_heads = 1 << 23
    refused(b, B.LORA_EUNSUPPORTED, grow, b, [0, 1], [1, 1])
    refused(b, B.LORA_EUNSUPPORTED, b.draft, rows(2), [0, 1], [[-1], [-1]], ids(2))


def test_more_positions_than_a_sequence_holds(monkeypatch):
    b = Block(monkeypatch, max_pages=2)
    grow(b, [0], [2 * b.page - 1])
    refused(b, B.LORA_EINVAL, grow, b, [0], [2])
    refused(b, B.LORA_EINVAL, b.draft, rows(2), [0], [[-1, 0]], ids(2))
    refused(b, B.LORA_EINVAL, b.step, rows(2), [0], [2], ids(2), pages=4)
    refused(b, B.LORA_EINVAL, grow, b, [1, 1], [1, 1])
    refused(b, B.LORA_ERANGE, grow, b, [4], [1])
    b = Block(monkeypatch, pool_pages=3)
    grow(b, [0, 1], [b.page + 1, 1])
    refused(b, B.LORA_ENOMEM, grow, b, [1, 2], [1, 1])


@pytest.mark.parametrize("error", [B.LoraError(B.LORA_EUNSUPPORTED, "too large"), torch.OutOfMemoryError("no memory"), KeyboardInterrupt()])
@pytest.mark.parametrize("how", ["step", "pages", "draft"])
def test_what_raises_later_takes_the_growth_back(monkeypatch, error, how):
    b = Block(monkeypatch)
    grow(b, [0, 1, 2], [b.page + 3, 2, b.page])
    b.draft(rows(3), [1], [[-1, 0, 0]], ids(3))
    b.kv.fork(0, [3])
    before = state(b)[::2]
    b.fails, b.calls[:] = error, []
    new = [1, b.page + 1, 2, 0]
    with pytest.raises(type(error)):
        if how == "draft":
            b.draft(rows(sum(new)), [0, 1, 2, 3], [[-1] * n for n in new], ids(sum(new)))
        else:
            b.step(rows(sum(new)), [0, 1, 2, 3], new, ids(sum(new)), pages=4 if how == "pages" else None)
    assert state(b)[::2] == before
    # the bounds of the pages that growth began on are those of the rows that are left; the fork's shared page is not touched
    assert [name for name, _ in b.calls] == ["run", "lora_kv_bounds_update"]
    seq, begin, end = (x.tolist() for x in b.calls[1][1][2:5])
    assert (seq, begin, end) == ([0, 1], [b.page + 2, 4], [b.page + 3, 5])
    b.fails = None
    b.accept([1], [[0, 2]])
    assert b.kv.length(1) == 4


def test_a_sequence_that_was_not_in_use_is_not_afterwards(monkeypatch):
    b = Block(monkeypatch)
    b.fails = B.LoraError(B.LORA_EUNSUPPORTED, "too large")
    with pytest.raises(B.LoraError):
        grow(b, [0, 2], [3, 0])
    assert state(b) == ([-1] * 4, [[]] * 4, {}, 0)


@pytest.mark.parametrize("paths", [[[0, 1], [1]], [[], [0]], [[], []]])
def test_siblings_accepted_at_a_page_border(monkeypatch, paths):
    """Forks whose context ends with a page share it: no two ranges of bounds touch it, and none has to."""
    b = Block(monkeypatch)
    grow(b, [0], [2 * b.page])
    b.kv.fork(0, [1, 2])
    grow(b, [2], [3])  # and one that ends within a page
    b.draft(rows(6), [0, 1, 2], [[-1, 0], [-1, -1], [-1, -1]], ids(6))
    shared, b.calls[:] = b.kv.pages(0)[:2].tolist(), []
    b.accept([0, 1, 2], [*paths, []])
    written = []
    for name, args in b.calls:
        if name == "lora_kv_bounds_update":
            for s, begin, end in zip(*(x.tolist() for x in args[2:5])):
                if s >= 0:
                    written += b.kv.pages(s)[begin // b.page: -(-end // b.page)].tolist()
    assert len(written) == len(set(written)) and not set(written) & set(shared)
    assert set(written) == {int(b.kv.pages(s)[2]) for s, p in ((0, paths[0]), (1, paths[1]), (2, [0])) if p}


@pytest.mark.parametrize("seqs,begins,lens", [([0, 1, 2], [0, 5, 7], [700, 1, 0]), ([0, 1], [3, 9], [1, 1]), ([0, 1, 2], [15, 40, 0], [300, 300, 300]),
                                              ([1], [3], [500]), ([2, 0], [4, 8], [0, 0])])
def test_ranges_cover_the_pages_once(monkeypatch, seqs, begins, lens):
    """Cut ranges name every page of the whole ones once, with the same last position, and none is longer than said."""
    b = Block(monkeypatch, max_pages=100)
    ends = [x + n for x, n in zip(begins, lens)]
    *cut, most = b._ranges(seqs, begins, ends)
    got = {}
    for s, begin, end in zip(*(x.tolist() for x in cut)):
        assert 0 <= begin < end and end - begin <= most
        for j in range(begin // b.page, -(-end // b.page)):
            assert (s, j) not in got
            got[s, j] = min(end, (j + 1) * b.page)
    assert got == {(s, j): min(e, (j + 1) * b.page) for s, x, e in zip(seqs, begins, ends) if x < e for j in range(x // b.page, -(-e // b.page))}


def test_a_long_prompt_beside_many_tokens(monkeypatch):
    """128Ki positions in pages of 16 beside 255 single tokens, 8 KV heads: 2^24 workgroups as whole ranges, and no reason to refuse
    the step that a block without bounds takes."""
    b = Block(monkeypatch)
    for field, value in (("kv_heads", 8), ("page_tokens", 16), ("max_pages", 8192)):
        setattr(b.kv.view.desc, field, value)
    *cut, most = b._ranges(list(range(256)), [0] + [77] * 255, [1 << 17] + [78] * 255)
    workgroups = ((most + 14) // 16 + 1) * 8 * len(cut[0])
    assert workgroups < 4 * 8 * (8192 + 255)  # of its pages and heads, a small multiple
    *cut, most = b._ranges([0, 1, 2], [5, 9, 30], [6, 10, 31])
    assert (cut[0].tolist(), most) == ([0, 1, 2], 1)
