"""Attention over selected pages on the GPU (lora_blocks.h): bounds, lists and attention over bf16 and 8-bit caches, against
plain 64-bit forms (kv_plain.py, which derives attention's bounds).  Bounds and lists are exact: they are whole numbers
times powers of two, and orders of them."""
import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")
from kv_plain import Cache, attention, compare, replayed  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


def say(msg):
    print(f"[case] {msg}", flush=True)


def dev(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def step_of(m):
    """The least f of -50 .. 50 with m <= 127 2^f."""
    f = -50
    while f < 50 and m > 127 * 2.0 ** f:
        f += 1
    return f


def plain_bounds(k):
    """H, L and f of a page and head from its keys [positions, dim] in 64 bits."""
    x = k.numpy()
    ok = np.isfinite(x)
    hi, lo = np.where(ok, x, -np.inf).max(0), np.where(ok, x, np.inf).min(0)
    none = ~ok.any(0)
    hi[none] = lo[none] = 0
    f = step_of(max(np.abs(hi).max(), np.abs(lo).max()))
    return np.clip(np.ceil(hi / 2.0 ** f), -127, 127), np.clip(np.floor(lo / 2.0 ** f), -127, 127), f


def new_bounds(c):
    shape = (c.view.desc.num_pages, c.heads, B.lora_kv_bounds_row_bytes(c.dim))
    return B.KvBounds(c.view, torch.full(shape, 0x55, dtype=torch.uint8, device="cuda"))


def unpack(rows, dim):
    """H, L, padding and f of rows [..., bytes]."""
    rows = rows.cpu()
    codes, f = rows[..., :-16].view(torch.int8), rows[..., -16:-12].contiguous().view(torch.int32)[..., 0]
    return codes[..., :dim].numpy(), codes[..., dim: 2 * dim].numpy(), codes[..., 2 * dim:].numpy(), f.numpy()


def filled(c, bounds):
    """Bounds of everything that the sequences hold."""
    n = len(c.kv_lens)
    B.lora_kv_bounds_update(c.view, bounds, dev(range(n)), dev([0] * n), dev(c.kv_lens), max(c.kv_lens))
    return bounds


# ---------------------------------------------------------------- bounds
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("page,layout", [(1, "page"), (8, "token"), (24, "apart"), (300, "page")])
def test_bounds(fp8, dim, page, layout):
    c = Cache([70, 25, 1], 3, dim, page, fp8, seed=dim + page, layout=layout)
    say(f"bounds fp8={fp8} dim={dim} page={page} {layout}")
    bounds = new_bounds(c)
    ranges = [(0, 30, 70), (1, 0, 25), (2, 0, 1)]
    B.lora_kv_bounds_update(c.view, bounds, *(dev(x) for x in zip(*ranges)), 40)
    hi, lo, pad, f = unpack(bounds.rows, dim)
    touched = set()
    for s, begin, end in ranges:
        for j in range(begin // page, -(-end // page)):
            g = int(c.table[s, j])
            touched.add(g)
            for h in range(3):
                want = plain_bounds(c.k[s][j * page: min(end, (j + 1) * page), h])
                assert (hi[g, h] == want[0]).all() and (lo[g, h] == want[1]).all() and f[g, h] == want[2] and (pad[g, h] == 0).all(), (s, j, h)
    rest = [g for g in range(c.view.desc.num_pages) if g not in touched]
    assert bool((bounds.rows[rest] == 0x55).all())
    assert bool((bounds.rows[..., -12:] == 0x55).all())


@pytest.mark.parametrize("dim", [8, 24, 40])
def test_bounds_of_heads_that_only_bf16_has(dim):
    c = Cache([37], 2, dim, 16, False, seed=dim)
    hi, lo, pad, f = unpack(filled(c, new_bounds(c)).rows, dim)
    for j in range(3):
        g = int(c.table[0, j])
        for h in range(2):
            want = plain_bounds(c.k[0][16 * j: min(37, 16 * j + 16), h])
            assert (hi[g, h] == want[0]).all() and (lo[g, h] == want[1]).all() and f[g, h] == want[2] and (pad[g, h] == 0).all()


def test_bounds_of_keys_that_are_not_finite_or_of_any_size():
    c = Cache([64], 1, 16, 8, False, seed=1)
    nan, inf = float("nan"), float("inf")
    for j, values in enumerate(([nan] * 8, [inf, -inf, 1.0, nan, -2.0, 0.5, inf, 0.0], [0.0] * 8, [1e38] * 8, [-1e-30] * 8,
                                [127.0, 0, 0, 0, 0, 0, 0, 127.0], [127.5, -1, 0, 0, 0, 0, 0, 0.001], [2.0 ** 56 * 1.5, -2.0 ** 57, 0, 0, 0, 0, 0, 1])):
        rows = torch.tensor(values).bfloat16()[:, None].repeat(1, 16)
        c.rows(0)[int(c.table[0, j]), 0] = rows.cuda()
        c.k[0][8 * j: 8 * j + 8, 0] = rows.double()
    hi, lo, _, f = unpack(filled(c, new_bounds(c)).rows, 16)
    for j in range(8):
        g = int(c.table[0, j])
        want = plain_bounds(c.k[0][8 * j: 8 * j + 8, 0])
        assert (hi[g, 0] == want[0]).all() and (lo[g, 0] == want[1]).all() and f[g, 0] == want[2], j


def test_ranges_without_a_place_change_nothing():
    c = Cache([40, 10], 2, 64, 8, False, seed=1, max_pages=6)
    bounds = new_bounds(c)
    before = bounds.rows.clone()
    B.lora_kv_bounds_update(c.view, bounds, dev([-1, 2, 0, 0, 0, 1]), dev([0, 0, 5, -1, 40, 30]), dev([8, 8, 5, 4, 49, 40]), 8)
    assert torch.equal(bounds.rows, before)
    B.lora_kv_bounds_update(c.view, bounds, dev([0]), dev([0]), dev([40]), 0)
    B.lora_kv_bounds_update(c.view, bounds, dev([]), dev([]), dev([]), 8)
    assert torch.equal(bounds.rows, before)
    B.lora_kv_bounds_update(c.view, bounds, dev([0]), dev([3]), dev([40]), 10)  # positions 3 .. 12: two pages
    changed = (bounds.rows != before).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert sorted(changed) == sorted(c.table[0, :2].tolist())


# ---------------------------------------------------------------- selection
def plain_select(c, bounds, q, seq, pos, count, sink, recent, table=None):
    hi, lo, _, f = unpack(bounds.rows, c.dim)
    table = c.table if table is None else table
    t, heads, dim = q.shape
    group = heads // c.heads
    out = np.full((t, c.heads, count), -1, np.int32)
    x = q.double().numpy()
    x = np.where(np.isfinite(x), x, 0)
    for i in range(t):
        if not (0 <= seq[i] < table.shape[0] and 0 <= pos[i] < table.shape[1] * c.page):
            continue
        n = pos[i] // c.page + 1
        for h in range(c.heads):
            if n <= count:
                out[i, h, :n] = np.arange(n)
                continue
            ids = table[seq[i], :n].numpy()
            there = (ids >= 0) & (ids < c.view.desc.num_pages)
            ids = np.where(there, ids, 0)
            H, L = hi[ids, h].astype(np.float64), lo[ids, h].astype(np.float64)
            score = np.full(n, -np.inf)
            for g in range(group):
                row = x[i, h * group + g]
                s = step_of(np.abs(row).max())
                w = np.clip(np.rint(row / 2.0 ** s), -127, 127)
                score = np.maximum(score, np.maximum(w * H, w * L).sum(1) * 2.0 ** s)
            score = np.where(there, score * 2.0 ** np.clip(f[ids, h], -50, 50), -np.inf)
            score[:sink] = np.inf
            score[n - recent:] = np.inf
            out[i, h] = np.sort(np.argsort(-score, kind="stable")[:count])
    return torch.from_numpy(out)


def check_select(c, heads, tokens, count, sink=1, recent=1, bounds=None, table=None, q=None, label=""):
    say(f"select {label} heads={heads}/{c.heads} dim={c.dim} page={c.page} fp8={c.fp8} tokens={tokens[:6]} count={count} sink={sink} recent={recent}")
    bounds = filled(c, new_bounds(c)) if bounds is None else bounds
    seq, pos = [s for s, _ in tokens], [p for _, p in tokens]
    if q is None:
        q = torch.randn((len(tokens), heads, c.dim), generator=torch.Generator().manual_seed(count)).bfloat16()
    blocks = torch.full((len(tokens) + 1, c.heads, count), 77, dtype=torch.int32, device="cuda")
    view = c.view if table is None else c.view_of(table)
    B.lora_kv_block_select(view, bounds, dev(seq), dev(pos), q.cuda(), blocks, sink=sink, recent=recent)
    want = plain_select(c, bounds, q, seq, pos, count, sink, recent, table)
    got = blocks.cpu()
    assert bool((got[-1] == 77).all()) and torch.equal(got[:-1], want), (label, (got[:-1] != want).nonzero()[:4].tolist())
    return bounds, blocks[:-1]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
def test_select(fp8, dim):
    c = Cache([700, 90], 2, dim, 8, fp8, seed=dim)
    tokens = [(0, 699), (0, 350), (1, 89), (0, 7), (0, 0), (1, 40), (0, 63), (0, 64), (0, 71), (0, 72)]
    check_select(c, 8, tokens, 9)
    check_select(c, 8, tokens, 9, sink=0, recent=1)
    check_select(c, 2, tokens, 30, sink=4, recent=5)
    check_select(c, 8, tokens, 2)
    check_select(c, 8, tokens, 1, sink=0)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 1), (16, 1), (17, 1), (40, 1), (24, 8)])
def test_select_head_layouts(heads, kv_heads):
    c = Cache([500], kv_heads, 64, 8, False, seed=heads)
    check_select(c, heads, [(0, 499), (0, 300)], 7)


@pytest.mark.parametrize("n,max_pages", [(2048, None), (2100, None), (9000, None), (600, 32768)])
def test_select_over_many_pages(n, max_pages):
    """Pages of one position: as many as the kernels' variants hold."""
    c = Cache([n], 1, 16, 1, False, seed=n, max_pages=max_pages)
    check_select(c, 4, [(0, n - 1), (0, n // 2), (0, 40)], 64)
    check_select(c, 4, [(0, n - 1)], 1500 if n > 2000 else 300, sink=3, recent=17)


def test_select_ties_go_to_the_lower_page():
    c = Cache([320], 2, 64, 8, False, seed=3)
    bounds = filled(c, new_bounds(c))
    rows = bounds.rows[c.table[0, 5].item()].clone()
    for j in (2, 5, 8, 9, 20, 30, 33):  # seven pages of the same bounds
        bounds.rows[c.table[0, j].item()] = rows
    for count in (3, 4, 6, 8, 12):
        check_select(c, 4, [(0, 319), (0, 250)], count, bounds=bounds, label="ties")
    bounds.rows[c.table[0].long().cuda()] = rows  # all of them
    check_select(c, 4, [(0, 319)], 11, bounds=bounds, label="all tie")
    check_select(c, 4, [(0, 319)], 11, bounds=bounds, q=torch.zeros((1, 4, 64)).bfloat16(), label="no query")


def test_select_for_queries_of_any_size_and_padding():
    c = Cache([400, 90], 1, 64, 8, False, seed=4, max_pages=60)
    q = torch.randn((8, 2, 64), generator=torch.Generator().manual_seed(1))
    q = (q * torch.tensor([1, 1e30, 1e-30, 1e-5, 300, 1, 1, 1])[:, None, None]).bfloat16()
    q[5, 0, ::2], q[6, 1, 3], q[7] = float("nan"), float("inf"), -float("inf")
    check_select(c, 2, [(0, 399)] * 8, 5, q=q, label="sizes")
    check_select(c, 2, [(-1, 10), (2, 10), (0, -1), (0, 480), (1, 89), (0, 2 ** 31 - 1)], 5, label="padding")


def test_absent_pages_come_last():
    c = Cache([400], 2, 64, 8, False, seed=5)
    table = c.table.clone()
    table[0, [0, 3, 10, 49]] = torch.tensor([-1, 1 << 30, -9, 500], dtype=torch.int32)
    check_select(c, 4, [(0, 399), (0, 200)], 6, table=table)
    table[0, 1:] = -1
    check_select(c, 4, [(0, 399)], 6, table=table)


# ---------------------------------------------------------------- attention
def listed_keep(blocks, pos, n, page, max_pages):
    """[t, kv_heads, n]: how often each position counts."""
    t, h, count = blocks.shape
    keep = torch.zeros((t, h, n))
    for i in range(t):
        for j in range(h):
            for b in blocks[i, j].tolist():
                if 0 <= b < max_pages:
                    keep[i, j, b * page: max(b * page, min((b + 1) * page, pos[i] + 1, n))] += 1
    return keep


def check_attention(c, heads, tokens, blocks, max_parts=0, label="", kv_lens=None):
    """blocks [t, kv_heads, count] host lists of (sequence, position) tokens."""
    t, _, count = blocks.shape
    say(f"listed attention {label} heads={heads}/{c.heads} dim={c.dim} page={c.page} fp8={c.fp8} tokens={t} count={count} parts={max_parts}")
    seq, pos = [s for s, _ in tokens], [p for _, p in tokens]
    q = (torch.randn((t, heads, c.dim), generator=torch.Generator().manual_seed(t)) * 1.5).bfloat16()
    plan = B.lora_kv_attn_plan(list(range(t + 1)), seq, [count * c.page] * t if kv_lens is None else kv_lens, heads, c.heads, c.dim,
                               blocks=True, max_parts=max_parts).to("cuda")
    if plan.workspace is not None:
        plan.workspace.fill_(float("nan"))
    qd = torch.cat([q, torch.full((2, heads, c.dim), float("nan"), dtype=torch.bfloat16)]).cuda()
    out = torch.full(qd.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(qd.shape[:2], 9.0, device="cuda")
    B.lora_kv_attn_blocks(c.view, plan, blocks.cuda(), dev(pos), qd, out, lse=lse)
    assert bool((out[t:] == 9).all()) and bool((lse[t:] == 9).all()), "rows behind the last token were written"
    for i, s in enumerate(seq):
        n = c.kv_lens[s]
        keep = listed_keep(blocks[i: i + 1], pos[i: i + 1], n, c.page, c.table.shape[1])
        want = attention(q[i: i + 1], c.k[s], c.v[s], keep, c.dim ** -0.5)
        compare(out[i: i + 1], lse[i: i + 1], *want, c.dim, (label, i))
    return plan, qd, out, lse


def some_lists(c, tokens, count, seed):
    """Distinct pages up to each token's, in any order, with -1 among them."""
    rng = np.random.default_rng(seed)
    out = np.full((len(tokens), c.heads, count), -1, np.int32)
    for i, (s, p) in enumerate(tokens):
        n = p // c.page + 1
        for h in range(c.heads):
            pick = rng.permutation(n)[:count]
            out[i, h, np.sort(rng.permutation(count)[: len(pick)])] = pick
    return torch.from_numpy(out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 192, 256])
def test_attention_head_dims(fp8, dim):
    c = Cache([300, 77], 2, dim, 16, fp8, seed=dim)
    tokens = [(0, 299), (1, 76), (0, 150), (0, 0), (1, 15), (1, 16)]
    check_attention(c, 8, tokens, some_lists(c, tokens, 6, dim))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,page", [(1, 1, 1), (3, 1, 7), (16, 1, 64), (24, 8, 33), (40, 1, 16), (14, 2, 24)])
def test_attention_head_layouts_and_pages(fp8, heads, kv_heads, page):
    c = Cache([200, 65], kv_heads, 64, page, fp8, seed=page)
    tokens = [(0, 199), (1, 64), (0, 100), (1, 0)]
    check_attention(c, heads, tokens, some_lists(c, tokens, 5, page))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_parts", [1, 2, 64, 0])
def test_long_lists_and_ranges_joined(fp8, max_parts):
    """Lists longer than the 64 entries that a wave holds at a time."""
    c = Cache([1900, 500], 2, 64, 8, fp8, seed=8)
    tokens = [(0, 1899), (1, 499), (0, 1000)]
    check_attention(c, 8, tokens, some_lists(c, tokens, 150, 1), max_parts=max_parts)
    c = Cache([300], 2, 64, 1, fp8, seed=9)
    check_attention(c, 4, [(0, 299)], some_lists(c, [(0, 299)], 200, 2), max_parts=max_parts, label="pages of one")


def test_many_tokens():
    c = Cache([400] * 3, 8, 128, 16, False, seed=2)
    tokens = [(i % 3, 399 - 5 * i) for i in range(40)]
    check_attention(c, 16, tokens, some_lists(c, tokens, 7, 3), label="many")


def test_lists_as_they_come():
    """Pages twice, out of range, behind the token's own; lists that name nothing; a plan for fewer pages than the list has."""
    c = Cache([100, 30], 2, 64, 16, False, seed=5)
    tokens = [(0, 99), (0, 40), (1, 29), (0, -1), (0, 10)]
    blocks = torch.tensor([[3, 3, 0, 6], [-1, 7, 1 << 30, -5], [2, 1, 5, 6], [0, 1, 2, 3], [1, 2, 3, 4]], dtype=torch.int32)[:, None].repeat(1, 2, 1)
    blocks[0, 1] = torch.tensor([1, -1, 1, 1])
    check_attention(c, 4, tokens, blocks)
    cut = blocks.clone()
    cut[:, :, 2:] = -1
    plan, q, out, lse = check_attention(c, 4, tokens, cut)
    few = B.lora_kv_attn_plan(list(range(6)), [s for s, _ in tokens], [32] * 5, 4, 2, 64, blocks=True).to("cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    B.lora_kv_attn_blocks(c.view, few, blocks.cuda(), dev([p for _, p in tokens]), q, o2, lse=l2)
    assert torch.equal(o2[:5], out[:5]) and torch.equal(l2[:5], lse[:5])


@pytest.mark.parametrize("fp8", [False, True])
def test_positions_behind_the_token_never_reach_it(fp8):
    c = Cache([100], 2, 64, 16, fp8, seed=6)
    blocks = torch.tensor([0, 2, 3, -1], dtype=torch.int32).repeat(1, 2, 1)
    plan, q, out, lse = check_attention(c, 4, [(0, 50)], blocks)
    page, _ = c.place(0, 51)
    for which in (0, 1):  # position 51 and on of the token's own page, and a page that is not listed
        for g, slots in ((page, slice(3, None)), (int(c.table[0, 1]), slice(None))):
            c.rows(which)[g, :, slots] = 0x7f if fp8 else float("nan")
            if fp8:
                c.row_scales(which)[g, :, slots] = 255
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    B.lora_kv_attn_blocks(c.view, plan, blocks.cuda(), dev([50]), q, o2, lse=l2)
    assert torch.equal(o2[:1], out[:1]) and torch.equal(l2[:1], lse[:1])


@pytest.mark.parametrize("fp8", [False, True])
def test_all_pages_selected_is_attention_over_everything(fp8):
    c = Cache([300, 90], 2, 128, 16, fp8, seed=7)
    tokens = [(0, 299), (1, 89)]
    _, blocks = check_select(c, 8, tokens, 20)
    check_attention(c, 8, tokens, blocks.cpu())
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    out, lse, o2, l2 = torch.empty_like(q), torch.empty((2, 8), device="cuda"), torch.empty_like(q), torch.empty((2, 8), device="cuda")
    B.lora_kv_attn(c.view, B.lora_kv_attn_plan([0, 1, 2], [0, 1], [300, 90], 8, 2, 128, max_parts=1).to("cuda"), q, out, lse=lse)
    plan = B.lora_kv_attn_plan([0, 1, 2], [0, 1], [320, 320], 8, 2, 128, blocks=True, max_parts=1).to("cuda")
    B.lora_kv_attn_blocks(c.view, plan, blocks, dev([299, 89]), q, o2, lse=l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_step_in_a_graph(fp8):
    """Append, bounds, selection and attention captured once; the positions, which are device data, move on between replays."""
    c = Cache([60, 300, 9], 2, 64, 8, fp8, seed=9, max_pages=60, spare=8)
    free = [g for g in range(c.view.desc.num_pages) if g not in c.table.flatten().tolist()]
    table = c.table.clone()
    table[0, 8], table[1, 38], table[2, 2] = free[0], free[1], free[2]  # the pages that the next tokens grow into
    table[0, 7], table[1, 37], table[2, 1] = c.table[0, 7], c.table[1, 37], c.table[2, 1]
    view = c.view_of(table)
    bounds = filled(c, new_bounds(c))
    bounds = B.KvBounds(view, bounds.rows)
    plan = B.lora_kv_attn_plan([0, 1, 2, 3], [0, 1, 2], [48] * 3, 4, 2, 64, blocks=True).to("cuda")
    seq, pos, end = dev([0, 1, 2]), dev([60, 300, 9]), dev([61, 301, 10])
    gen = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((3, h, 64), generator=gen).bfloat16().cuda() for h in (4, 2, 2))
    blocks = torch.empty((3, 2, 6), dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")

    def step():
        B.lora_kv_append(view, k, v, seq, pos)
        B.lora_kv_bounds_update(view, bounds, seq, pos, end, 1)
        B.lora_kv_block_select(view, bounds, seq, pos, q, blocks, sink=1, recent=2)
        B.lora_kv_attn_blocks(view, plan, blocks, pos, q, out, lse=lse)

    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step()
    store, scales, rows = c.store.clone(), c.scales.clone(), bounds.rows.clone()
    got = []
    for eager in (False, True):
        c.store.copy_(store), c.scales.copy_(scales), bounds.rows.copy_(rows)
        pos.copy_(dev([60, 300, 9])), end.copy_(dev([61, 301, 10]))
        for i in range(4):
            q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)).bfloat16())
            torch.cuda.synchronize()
            step() if eager else graph.replay()
            torch.cuda.synchronize()
            got.append([x.clone() for x in (blocks, out, lse, bounds.rows)])
            pos.add_(1), end.add_(1)
    for a, b in zip(got[:4], got[4:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_bounds_and_lists_are_replayed():
    c = Cache([500, 90], 2, 64, 8, False, seed=10)
    bounds = new_bounds(c)
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    blocks = torch.empty((2, 2, 9), dtype=torch.int32, device="cuda")
    seq, begin, end, pos = dev([0, 1]), dev([0, 0]), dev([500, 90]), dev([499, 89])

    def run():
        B.lora_kv_bounds_update(c.view, bounds, seq, begin, end, 500)
        B.lora_kv_block_select(c.view, bounds, seq, pos, q, blocks)
    replayed(run, run, [blocks], lambda: (bounds.rows.zero_(), q.float().sum()))
