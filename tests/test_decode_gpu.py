"""The serving block with 8-bit rows, drafted trees and selected pages, as a server runs them one after the other: what each
attention gets and gives is checked against a plain 64-bit form over the rows that the cache holds (kv_plain.py, which
derives the bounds); what moves in the cache is checked bit for bit."""
import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")
from kv_plain import attention, compare  # noqa: E402

pytestmark = pytest.mark.gpu
D_MODEL, HEADS, KV_HEADS, DIM = 512, 8, 2, 64


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


class Watched:
    """A block whose attention's inputs and outputs are kept."""

    def __init__(self, monkeypatch, fp8, bounds=True, **kw):
        from segmented_gather_gemm_segments_amd import runner as R
        self.block = R.ServingBlock(D_MODEL, HEADS, KV_HEADS, DIM, 4, 16, max_seqs=6, max_pages=12, pool_pages=64, seed=3, fp8=fp8,
                                    bounds=bounds, **kw)
        self.page = self.block.kv.stats()["page_tokens"]
        self.gen = torch.Generator(device="cuda").manual_seed(9)
        self.seen = []
        for name, q_at in (("lora_kv_attn", 2), ("lora_kv_attn_tree", 3), ("lora_kv_attn_blocks", 4)):
            monkeypatch.setattr(B, name, self.spy(getattr(B, name), q_at))

    def spy(self, call, q_at):
        def inner(*args, **kw):
            if "lse" not in kw and len(args) == q_at + 2 and "_call" not in kw:
                lse = torch.empty(args[q_at].shape[:2], device="cuda")
                self.seen.append((args, args[q_at], args[q_at + 1], lse))
                return call(*args, lse=lse, **kw)
            return call(*args, **kw)
        return inner

    def hidden(self, t):
        return torch.randn((t, D_MODEL), generator=self.gen, device="cuda").bfloat16(), torch.arange(t, dtype=torch.int32, device="cuda") % 5 - 1

    def rows(self, s, n=None):
        n = self.block.kv.length(s) if n is None else n
        k, v = (torch.empty((n, KV_HEADS, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        B.lora_kv_read(self.block.kv.view, torch.full((n,), s, dtype=torch.int32, device="cuda"),
                       torch.arange(n, dtype=torch.int32, device="cuda"), k, v)
        return k.cpu(), v.cpu()

    def check(self, seqs, new, keep_of):
        """The last attention against the plain form; keep_of(i, s, new, length) -> mask of request i."""
        args, q, out, lse = self.seen[-1]
        assert bool(torch.isfinite(out).all())
        at = 0
        for i, (s, n) in enumerate(zip(seqs, new)):
            k, v = self.rows(s)
            want = attention(q[at: at + n].cpu(), k.double(), v.double(), keep_of(i, s, n, k.shape[0], at), DIM ** -0.5)
            compare(out[at: at + n], lse[at: at + n], *want, DIM, (i, s))
            at += n

    def check_bounds(self, seqs):
        """Bounds enclose every key, and are those of the rows that a page has where no drafted node was dropped."""
        rows = self.block.kv.bounds.rows.cpu()
        f = rows[..., -16:-12].contiguous().view(torch.int32)[..., 0].double()
        codes = rows.view(torch.int8)
        for s in seqs:
            k = self.rows(s)[0].double()
            for j, g in enumerate(self.block.kv.pages(s)):
                part = k[j * self.page: (j + 1) * self.page]
                unit = torch.exp2(f[int(g)])[:, None]
                assert bool((codes[int(g), :, :DIM] * unit >= part.amax(0)).all()) and bool((codes[int(g), :, DIM: 2 * DIM] * unit <= part.amin(0)).all())


def causal(i, s, n, length, at):
    return torch.arange(length)[None] <= torch.arange(length - n, length)[:, None]


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_drafts_and_selected_pages(monkeypatch, fp8):
    w = Watched(monkeypatch, fp8)
    block, rng = w.block, np.random.default_rng(1)

    def step(seqs, new, **kw):
        print(f"[case] step fp8={fp8} {seqs} {new} {kw}", flush=True)
        h, ids = w.hidden(sum(new))
        y = block.step(h, seqs, new, ids, **kw)
        assert bool(torch.isfinite(y).all())

    def listed(i, s, n, length, at):
        keep = torch.zeros((n, KV_HEADS, length))
        blocks, pos = w.seen[-1][0][2].cpu(), w.seen[-1][0][3].cpu()
        for t in range(n):
            p = length - n + t
            assert int(pos[at + t]) == p
            for h in range(KV_HEADS):
                pages = [b for b in blocks[at + t, h].tolist() if b >= 0]
                assert pages == sorted(set(pages)) and pages[0] == 0 and pages[-1] == p // w.page and len(pages) <= blocks.shape[2]
                for b in pages:
                    keep[t, h, b * w.page: min((b + 1) * w.page, p + 1)] = 1
        return keep

    step([0, 1, 2], [5 * w.page + 3, 40, 1])
    w.check([0, 1, 2], [5 * w.page + 3, 40, 1], causal)
    w.check_bounds([0, 1, 2])
    step([0, 1, 2], [1, 1, 1], pages=4)
    w.check([0, 1, 2], [1, 1, 1], listed)
    step([2, 0], [2 * w.page + 5, 3], pages=3)
    w.check([2, 0], [2 * w.page + 5, 3], listed)
    block.kv.fork(0, [3, 4])
    before = {s: w.rows(s) for s in (0, 1, 3, 4)}
    base = {s: block.kv.length(s) for s in (0, 1, 3)}
    # trees of sequences of which two share all their pages
    parents = {0: [-1, 0, 0, 1, 2, 4, -1, 6], 1: [-1] + [int(rng.integers(-1, i)) for i in range(1, 40)], 3: [-1]}
    h, ids = w.hidden(49)
    y = block.draft(h, [0, 1, 3], [parents[0], parents[1], parents[3]], ids)
    assert bool(torch.isfinite(y).all())

    def nodes(i, s, n, length, at):
        keep = torch.zeros((n, length), dtype=torch.bool)
        for j in range(n):
            keep[j, : length - n] = True
            a = j
            while a >= 0:
                keep[j, length - n + a] = True
                a = parents[s][a]
        return keep
    w.check([0, 1, 3], [8, 40, 1], nodes)
    path1 = [39]
    while parents[1][path1[0]] >= 0:
        path1.insert(0, parents[1][path1[0]])
    paths = {0: [0, 2, 4, 5], 1: path1, 3: []}
    drafted = {s: w.rows(s) for s in (0, 1, 3)}
    block.accept([0, 1, 3], [paths[s] for s in (0, 1, 3)])
    for s in (0, 1, 3):
        assert block.kv.length(s) == base[s] + len(paths[s])
        for now, then, old in zip(w.rows(s), drafted[s], before[s]):
            assert torch.equal(now[: base[s]], old) and torch.equal(now[base[s]:], then[[base[s] + n for n in paths[s]]])
    for now, old in zip(w.rows(4), before[4]):  # the fork that drafted nothing
        assert torch.equal(now, old)
    w.check_bounds([0, 1, 2, 3, 4])
    step([0, 1, 3, 4], [1, 2, 1, 1], pages=5)
    w.check([0, 1, 3, 4], [1, 2, 1, 1], listed)
    block.kv.free([2])
    assert block.kv.compact() >= 0
    step([0, 1, 3, 4], [1, 1, 30, 1])
    w.check([0, 1, 3, 4], [1, 1, 30, 1], causal)
    w.check_bounds([0, 1, 3, 4])
    step([0, 1, 3, 4], [1, 1, 1, 1], pages=3)
    w.check([0, 1, 3, 4], [1, 1, 1, 1], listed)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_chain_is_what_decoding_it_is(monkeypatch, fp8):
    """A tree without branches, accepted whole, leaves the cache that a chunk of its tokens leaves, and gives its output."""
    w = Watched(monkeypatch, fp8, bounds=False)
    h, ids = w.hidden(30)
    w.block.step(h, [0], [30], ids)
    w.block.kv.fork(0, [1])
    h, ids = w.hidden(20)
    y = w.block.draft(h, [0], [list(range(-1, 19))], ids)
    w.check([0], [20], causal)
    w.block.accept([0], [list(range(20))])
    z = w.block.step(h, [1], [20], ids)
    w.check([1], [20], causal)
    assert all(torch.equal(a, b) for a, b in zip(w.rows(0), w.rows(1)))
    assert y.shape == z.shape


def test_what_accept_and_draft_refuse(monkeypatch):
    w = Watched(monkeypatch, False)
    h, ids = w.hidden(30)
    w.block.step(h, [0, 1], [20, 10], ids)
    call = lambda n, *args: w.block.draft(*w.hidden(n)[:1], *args, w.hidden(n)[1])
    before = [w.block.kv.length(s) for s in (0, 1)]
    for n, seqs, parents in ((2, [0], [[-1, 1]]), (2, [0], [[-1, -2]]), (3, [0], [[-1, 0]]), (1, [0, 1], [[-1]])):
        with pytest.raises(B.LoraError):
            call(n, seqs, parents)
    refused = lambda seqs, paths: pytest.raises(B.LoraError, w.block.accept, seqs, paths)
    refused([0], [[0]])                      # no draft
    assert [w.block.kv.length(s) for s in (0, 1)] == before
    call(5, [0, 1], [[-1, 0, 1], [-1, -1]])
    store = w.block.pool.storage.clone()
    for seqs, paths in (([0], [[1, 0]]), ([0], [[0, 3]]), ([0], [[-1]]), ([0, 0], [[0], [0]]), ([0], [[0], [1]]), ([2], [[0]])):
        refused(seqs, paths)
    for path in ([1, 2], [0, 2], [2]):       # nodes whose ancestors would go
        refused([0], [path])
    w.block.kv.fork(0, [2])
    refused([0], [[1, 2]])                   # a fork holds the draft's pages
    refused([0], [[0, 1, 2]])
    assert torch.equal(w.block.pool.storage.view(torch.int16), store.view(torch.int16)) and w.block.kv.length(0) == 23
    w.block.accept([1], [[1]])
    refused([1], [[0]])                      # over already
    w.block.kv.free([2])
    w.block.step(*[w.hidden(1)[0], [0], [1], w.hidden(1)[1]])
    refused([0], [[0]])                      # the sequence went on
    plain = Watched(monkeypatch, False, bounds=False)
    with pytest.raises(B.LoraError):
        plain.block.step(*[plain.hidden(1)[0], [0], [1], plain.hidden(1)[1]], pages=3)
    with pytest.raises(B.LoraError):
        w.block.step(*[w.hidden(1)[0], [0], [1], w.hidden(1)[1]], pages=2, sink=1, recent=2)


def test_drafts_dropped_and_replaced(monkeypatch):
    """A draft accepted with no node of it, over a context that has none either; one that a step or a second draft follows."""
    w = Watched(monkeypatch, False)
    run = lambda call, n, *args: call(w.hidden(n)[0], *args, w.hidden(n)[1])
    run(w.block.draft, 3, [0], [[-1, 0, 0]])
    w.block.accept([0], [[]])
    assert w.block.kv.length(0) == 0
    run(w.block.step, 9, [0, 1], [9, 0])
    run(w.block.draft, 3, [0, 1], [[-1, 0, 0], []])
    run(w.block.draft, 2, [0], [[-1, 0]])    # the first draft's nodes are context now
    with pytest.raises(B.LoraError):
        w.block.accept([0], [[0, 2]])
    w.block.accept([0], [[0]])
    assert w.block.kv.length(0) == 13
    run(w.block.draft, 3, [0], [[-1, 0, 0]])
    w.block.kv.free([0])
    run(w.block.step, 16, [0], [16])         # as long as the draft was
    with pytest.raises(B.LoraError):
        w.block.accept([0], [[0]])
    assert w.block.kv.length(0) == 16


def test_debug_build_reports_bad_places():
    """The debug build names bad pages, tokens and items of the calls around 8-bit rows, trees and listed pages."""
    B.select_library(True)
    try:
        B.lora_kv_debug_flags(clear=True)
        i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
        store = torch.zeros((4, 2, 1, 8, 64), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.full((4, 2, 1, 8), 127, dtype=torch.uint8, device="cuda")
        bf = torch.zeros((4, 2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
        table = torch.tensor([[0, 1, 3, 0], [2, 9, -1, 2]], dtype=torch.int32, device="cuda")  # sequence 1: pages 1 and 2 are absent
        views = [B.KvView(store[:, 0], store[:, 1], table, scales[:, 0], scales[:, 1]), B.KvView(bf[:, 0], bf[:, 1], table)]
        new = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
        q = torch.ones((40, 2, 64), dtype=torch.bfloat16, device="cuda")
        PAGE, TOKEN, ITEM = B.LORA_DEBUG_BAD_PAGE, B.LORA_DEBUG_BAD_TOKEN, B.LORA_DEBUG_BAD_ITEM

        def flags_of(call, *args, **kw):
            call(*args, **kw)
            return B.lora_kv_debug_flags(clear=True)
        for view in views:
            out = torch.empty_like(q)
            for call, rows in ((B.lora_kv_append, lambda s, p: (view, new, new.clone(), i(s), i(p))), (B.lora_kv_read, lambda s, p: (view, i(s), i(p), new, new.clone()))):
                for (s, p), want in (((0, 9), 0), ((-1, 9), 0), ((1, 9), PAGE), ((0, 32), TOKEN), ((2, 0), TOKEN), ((0, -1), TOKEN)):
                    assert flags_of(call, *rows(s, p)) == want, (call, s, p)
            for n in (1, 40):  # row items and tile items
                plan = lambda s, kv, **kw: B.lora_kv_attn_plan([0, n], [s], [kv], 2, 1, 64, **kw).to("cuda")
                tree = B.Tree(n, n, "cuda")
                assert flags_of(B.lora_tree_mask, i(0, n), i(*range(-1, n - 1)), tree) == 0
                for s, kv, want in ((0, 24, 0), (1, 24, PAGE), (0, 60, ITEM)):
                    assert flags_of(B.lora_kv_attn, view, plan(s, kv, causal=False), q, out) == want, (n, s, kv)
                    assert flags_of(B.lora_kv_attn_tree, view, plan(s, kv, tree=True, causal=False), tree, q, out) == want, (n, s, kv)
            lists = torch.tensor([[[0, 2, -1, -1]]], dtype=torch.int32, device="cuda")
            one = lambda s: B.lora_kv_attn_plan([0, 1], [s], [32], 2, 1, 64, blocks=True).to("cuda")
            for s, pos, count, want in ((0, 30, 4, 0), (1, 30, 4, PAGE), (1, 5, 4, 0), (0, 30, 3, ITEM)):
                assert flags_of(B.lora_kv_attn_blocks, view, one(s), lists[..., :count].contiguous(), i(pos), q[:1], out[:1]) == want, (s, pos, count)
            assert flags_of(B.lora_kv_keep_path, view, i(0), i(2), i(1, 3, -1)[None]) == 0
            assert flags_of(B.lora_kv_keep_path, view, i(0), i(2), i(1, 3, 3)[None]) == TOKEN
            assert flags_of(B.lora_kv_keep_path, view, i(0), i(30), i(1, 3)[None]) == TOKEN
            assert flags_of(B.lora_kv_keep_path, view, i(2), i(0), i(1)[None]) == TOKEN
            assert flags_of(B.lora_kv_keep_path, view, i(1), i(7), i(2)[None]) == PAGE
            bounds = B.KvBounds(view, torch.zeros((4, 1, 144), dtype=torch.uint8, device="cuda"))
            for (s, b, e, most), want in (((0, 0, 32, 32), 0), ((1, 0, 8, 8), 0), ((1, 0, 9, 9), PAGE), ((0, 0, 33, 40), TOKEN), ((0, 4, 4, 4), TOKEN),
                                          ((2, 0, 1, 1), TOKEN), ((-1, 0, 99, 8), 0), ((0, 0, 32, 16), TOKEN)):
                assert flags_of(B.lora_kv_bounds_update, view, bounds, i(s), i(b), i(e), most) == want, (s, b, e, most)
            blocks = torch.empty((1, 1, 2), dtype=torch.int32, device="cuda")
            for (s, p), want in (((0, 31), 0), ((-1, 31), 0), ((1, 31), PAGE), ((1, 15), 0), ((0, 32), TOKEN), ((2, 0), TOKEN)):
                assert flags_of(B.lora_kv_block_select, view, bounds, i(s), i(p), q[:1], blocks, sink=1, recent=1) == want, (s, p)
        tree = B.Tree(3, 64, "cuda")
        assert flags_of(B.lora_tree_mask, i(0, 3), i(-1, 1, 0), tree) == TOKEN and flags_of(B.lora_tree_mask, i(0, 4), i(-1, -1, 0), tree) == TOKEN
    finally:
        B.select_library(False)
