"""Trees of drafted tokens on the GPU (lora_tree.h): masks and depths, attention over bf16 and 8-bit caches, accepted paths
moved, against plain 64-bit forms (kv_plain.py, which derives attention's bounds).  Masks, depths and moved rows
are exact."""
import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")
from kv_plain import Cache, attention, compare, replayed, starts_of  # noqa: E402

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


def random_parents(n, rng, back=6):
    return [int(rng.integers(max(-1, i - back), i)) if i else -1 for i in range(n)]


def ancestors(parents, window=0):
    """Per node: the nodes that it keeps, and its depth."""
    kept, depth = [], []
    for i, p in enumerate(parents):
        up = (lines[p] if p >= 0 else []) + [i] if i else [i]
        if i == 0:
            lines = {}
        lines[i] = up
        depth.append(len(up) - 1)
        kept.append(up[-window:] if window else up)
    return kept, depth


def words_of(kept, words):
    rows = np.zeros((len(kept), words), np.uint64)
    for i, nodes in enumerate(kept):
        for a in nodes:
            rows[i, a // 64] |= np.uint64(1) << np.uint64(a % 64)
    return torch.from_numpy(rows.view(np.int64))


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("sizes,most", [([1], 1), ([2, 0, 5], 5), ([63, 64, 65], 65), ([26] * 40, 26), ([130, 1, 200], 256), ([700], 1000)])
@pytest.mark.parametrize("window", [0, 1, 3, 70])
def test_masks_and_depths(sizes, most, window):
    rng = np.random.default_rng(sum(sizes) + window)
    say(f"tree mask {sizes} window={window}")
    parents = [random_parents(n, rng) for n in sizes]
    tree = B.Tree(sum(sizes), most, "cuda")
    tree.mask.fill_(-1), tree.depth.fill_(-1)
    B.lora_tree_mask(dev(starts_of(sizes)), dev(sum(parents, [])), tree, window=window)
    want = [ancestors(p, window) for p in parents]
    assert torch.equal(tree.depth.cpu(), torch.tensor(sum((d for _, d in want), []), dtype=torch.int32))
    assert torch.equal(tree.mask.cpu(), torch.cat([words_of(k, tree.desc.words) for k, _ in want]))


@pytest.mark.parametrize("window", [0, 100])
def test_the_longest_chain(window):
    n = 4096
    tree = B.Tree(n, n, "cuda")
    B.lora_tree_mask(dev([0, n]), dev(range(-1, n - 1)), tree, window=window)
    kept, depth = list(range(n)), list(range(n))
    assert tree.depth.tolist() == depth
    assert torch.equal(tree.mask.cpu(), words_of([range(max(0, i - window + 1) if window else 0, i + 1) for i in kept], 64))


def test_parents_out_of_range_count_as_the_context():
    parents = [5, 0, 2, -7, 3, 1 << 30]
    tree = B.Tree(6, 6, "cuda")
    B.lora_tree_mask(dev([0, 6]), dev(parents), tree)
    kept, depth = ancestors([-1, 0, -1, -1, 3, -1])
    assert tree.depth.tolist() == depth and torch.equal(tree.mask.cpu(), words_of(kept, 1))


def test_requests_that_do_not_fit_are_skipped():
    tree = B.Tree(140, 64, "cuda")
    for starts, kept in (([0, 65, 70], range(0, 65)), ([-1, 5, 5], range(0, 5)), ([0, 10, 141], range(10, 140)), ([20, 10, 12], range(0, 10))):
        tree.mask.fill_(-3), tree.depth.fill_(-3)
        B.lora_tree_mask(dev(starts), dev([-1] * 140), tree)
        assert bool((tree.mask[list(kept)] == -3).all()) and bool((tree.depth[list(kept)] == -3).all()), starts
    assert tree.depth[10].item() == 0 and tree.mask[11, 0].item() == 2
    B.lora_tree_mask(dev([0]), dev([-1] * 140), tree)
    empty = B.Tree(0, 0, "cuda")
    B.lora_tree_mask(dev([0, 0]), dev([]), empty)


# ---------------------------------------------------------------- attention
def tree_keep(kept, depth, kv_len, window, causal):
    """[nodes, positions] of one request."""
    n = len(kept)
    base = kv_len - n
    keep = torch.zeros((n, kv_len), dtype=torch.bool)
    for i in range(n):
        low = base + min(max(depth[i], 0), i) - window + 1 if window else 0
        keep[i, max(low, 0): max(base, 0)] = True
        for a in kept[i]:
            if 0 <= base + a < kv_len and not (causal and a > i):
                keep[i, base + a] = True
    return keep


def check(c, sizes, heads, window=0, causal=True, max_parts=0, seqs=None, kv_lens=None, seed=0, masks=None, label=""):
    """masks: (kept, depth) of each request given by hand, else of random trees through lora_tree_mask."""
    seqs = list(range(len(sizes))) if seqs is None else seqs
    kv_lens = [c.kv_lens[s] for s in seqs] if kv_lens is None else kv_lens
    say(f"tree attention {label} nodes={sizes} kv={kv_lens} heads={heads}/{c.heads} dim={c.dim} page={c.page} fp8={c.fp8} "
        f"window={window} causal={causal}")
    rng = np.random.default_rng(seed + sum(sizes))
    starts, t = starts_of(sizes), sum(sizes)
    tree = B.Tree(t, max(sizes + [1]), "cuda")
    if masks is None:
        parents = [random_parents(n, rng) for n in sizes]
        B.lora_tree_mask(dev(starts), dev(sum(parents, [])), tree, window=window)
        masks = [ancestors(p, window) for p in parents]
    else:
        tree.mask.copy_(torch.cat([words_of(k, tree.desc.words) for k, _ in masks]))
        tree.depth.copy_(torch.tensor(sum((d for _, d in masks), []), dtype=torch.int32))
    q = (torch.randn((t, heads, c.dim), generator=torch.Generator().manual_seed(seed)) * 1.5).bfloat16()
    plan = B.lora_kv_attn_plan(starts, seqs, kv_lens, heads, c.heads, c.dim, window=window, causal=causal, max_parts=max_parts, tree=True).to("cuda")
    if plan.workspace is not None:
        plan.workspace.fill_(float("nan"))
    qd = torch.cat([q, torch.full((2, heads, c.dim), float("nan"), dtype=torch.bfloat16)]).cuda()
    out = torch.full(qd.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(qd.shape[:2], 9.0, device="cuda")
    B.lora_kv_attn_tree(c.view, plan, tree, qd, out, lse=lse)
    assert bool((out[t:] == 9).all()) and bool((lse[t:] == 9).all()), "rows behind the last token were written"
    for r, s in enumerate(seqs):
        a, b, n = int(starts[r]), int(starts[r + 1]), kv_lens[r]
        want = attention(q[a:b], c.k[s][:n], c.v[s][:n], tree_keep(*masks[r], n, window, causal), c.dim ** -0.5)
        compare(out[a:b], lse[a:b], *want, c.dim, (label, r))
    return plan, tree, qd, out, lse


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 192, 256])
def test_head_dims(fp8, dim):
    c = Cache([120, 77, 300, 33], 2, dim, 16, fp8, seed=dim)
    check(c, [2, 1, 3, 2], 8, label="few")
    check(c, [20, 70, 40, 33], 8, label="many")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 1, 4, 50, 1000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_count_along_the_path(fp8, window, causal):
    c = Cache([300, 64, 65, 40], 2, 64, 24, fp8, seed=window)
    check(c, [90, 64, 2, 1], 4, window, causal)
    check(c, [3, 4, 2, 1], 4, window, causal)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,kv_heads,page", [(1, 1, 1), (3, 1, 7), (16, 1, 64), (24, 8, 33), (40, 1, 16)])
def test_head_layouts_and_pages(fp8, heads, kv_heads, page):
    c = Cache([130, 200], kv_heads, 64, page, fp8, seed=page)
    check(c, [26, 61], heads)
    check(c, [1, 1], heads)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_requests(fp8, dim):
    kv_lens = [30 + (37 * i) % 190 for i in range(36)]
    c = Cache(kv_lens, 8, dim, 16, fp8, seed=dim)
    check(c, [1 + i % 27 for i in range(36)], 8, label="many")
    check(c, [1 + i % 2 for i in range(36)], 8, window=20, label="many, windowed")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("max_parts", [1, 3, 64, 0])
def test_ranges_joined(fp8, max_parts):
    c = Cache([1500, 700], 2, 128, 16, fp8, seed=8)
    check(c, [26, 130], 8, max_parts=max_parts)
    check(c, [2, 3], 8, max_parts=max_parts, window=500)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [6, 70])
def test_any_mask_is_taken_as_it_is(fp8, n):
    """Rows without a node, nodes that are not ancestors, bits behind the request's nodes, depths out of range."""
    rng = np.random.default_rng(n)
    for context in (0, 1, 130):
        c = Cache([context + n, 50], 2, 64, 16, fp8, seed=n + context)
        kept = [sorted(rng.choice(n, rng.integers(0, n), replace=False).tolist()) for _ in range(n)]
        kept[0] = kept[n - 1] = []
        kept[1] = kept[1] + [n, n + 2]
        depth = [int(x) for x in rng.integers(-5, 2 * n, n)]
        for causal in (True, False):
            for window in (0, 9):
                check(c, [n, 1], 4, window, causal, masks=[(kept, depth), ([[0]], [0])], label=f"context {context}")


@pytest.mark.parametrize("fp8", [False, True])
def test_trees_longer_than_their_sequence(fp8):
    """Nodes before position 0 are in no cache."""
    c = Cache([10, 5, 90], 2, 64, 8, fp8, seed=4)
    check(c, [13, 9, 80], 4, kv_lens=[10, 0, 70])
    check(c, [13, 9, 80], 4, window=7, kv_lens=[10, 5, 80])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [4, 70])
def test_nodes_that_are_not_kept_never_reach_a_node(fp8, n):
    """Siblings' rows that are not finite."""
    c = Cache([100 + n], 2, 64, 16, fp8, seed=n)
    star = ([[i] for i in range(n)], [0] * n)  # every node hangs below the context
    plan, tree, q, out, lse = check(c, [n], 4, masks=[star])
    page, slot = c.place(0, 100 + n - 2)  # node n - 2
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[n - 2] = False
    for which in (0, 1):
        c.rows(which)[page, :, slot] = 0x7f if fp8 else float("inf")
        if fp8:
            c.row_scales(which)[page, :, slot] = 255
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        B.lora_kv_attn_tree(c.view, plan, tree, q, o2, lse=l2)
        assert torch.equal(o2[:n][others], out[:n][others]) and torch.equal(l2[:n][others], lse[:n][others])
        assert not bool(torch.isfinite(o2[n - 2]).any())


# ---------------------------------------------------------------- paths
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["page", "token", "apart"])
@pytest.mark.parametrize("dim,page", [(16, 1), (64, 5), (256, 16)])
def test_paths_are_moved(fp8, layout, dim, page):
    kv_lens = [60, 33, 90, 41, 20]
    c = Cache(kv_lens, 3, dim, page, fp8, seed=dim, layout=layout)
    base = [20, 0, 30, 41, 5]
    path = [[0, 1, 2, 3, 9, 10, 11, 12, 13, 20, 21, 39], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 31, 32], [59] + [-1] * 11,
            [-1] * 12, [3, 5, 5, 6] + [8] * 8]
    say(f"path fp8={fp8} {layout} dim={dim} page={page}")
    store, scales = c.store.cpu().clone(), c.scales.cpu().clone()
    for r in range(5):
        before = -1
        for i, e in enumerate(path[r]):
            if e <= before:
                break
            before = e
            (pa, sa), (pb, sb) = c.place(r, base[r] + e), c.place(r, base[r] + i)
            for which in (0, 1):
                rows = c._pick(store, which)[..., :dim]
                rows[pb, :, sb] = rows[pa, :, sa].clone()
                if fp8:
                    c._pick(scales, which)[pb, :, sb] = c._pick(scales, which)[pa, :, sa].clone()
    B.lora_kv_keep_path(c.view, dev(range(5)), dev(base), dev(path))
    bits = torch.uint8 if fp8 else torch.int16
    assert torch.equal(c.store.cpu().view(bits), store.view(bits)) and torch.equal(c.scales.cpu(), scales)


def test_paths_without_a_place_change_nothing():
    for fp8 in (False, True):
        c = Cache([40, 10], 2, 64, 8, fp8, seed=1, max_pages=6)
        bits = torch.uint8 if fp8 else torch.int16
        store, scales = c.store.clone(), c.scales.clone()
        call = lambda seq, base, path: B.lora_kv_keep_path(c.view, dev(seq), dev(base), dev(path))
        call([-1, 2, 0, 1], [0, 0, -3, 2 ** 31 - 1], [[1], [1], [1], [1]])
        call([0], [44], [[4]])    # past the last page
        call([0], [4], [[2 ** 31 - 1]])
        call([1], [12], [[5]])    # from and to a place behind the sequence's pages
        call([0], [4], [[0, 1, 2, 3]])  # where they are already
        B.lora_kv_keep_path(c.view, dev([]), dev([]), torch.empty((0, 4), dtype=torch.int32, device="cuda"))
        B.lora_kv_keep_path(c.view, dev([0]), dev([0]), torch.empty((1, 0), dtype=torch.int32, device="cuda"))
        assert torch.equal(c.store.view(bits), store.view(bits)) and torch.equal(c.scales, scales)


@pytest.mark.parametrize("fp8", [False, True])
def test_mask_attention_and_path_in_a_graph(fp8):
    c = Cache([900, 130], 2, 128, 16, fp8, seed=9)
    sizes = [26, 61]
    plan, tree, q, out, lse = check(c, sizes, 8)
    rng = np.random.default_rng(5)
    starts, parents = dev(starts_of(sizes)), dev(sum((random_parents(n, rng) for n in sizes), []))
    seq, base, path = dev([0, 1]), dev([900 - 26, 130 - 61]), dev([[4, 7, 20, -1], [9, 30, 40, 60]])
    # nodes that the path's rows go to are among none of those it reads, so that every replay moves the same rows

    def run():
        B.lora_tree_mask(starts, parents, tree)
        B.lora_kv_attn_tree(c.view, plan, tree, q, out, lse=lse)
    replayed(run, run, [tree.mask, tree.depth, out[:87], lse[:87]], lambda: q.float().sum())

    def move():
        B.lora_kv_keep_path(c.view, seq, base, path)
    move()
    want = c.store.clone()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        move()
    bits = torch.uint8 if fp8 else torch.int16
    for _ in range(3):
        for s in (0, 1):
            page, slot = c.place(s, int(base[s]))
            c.rows(0)[page, :, slot] = 0
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.store.view(bits), want.view(bits))
