"""Kernels that the calls around the KV cache choose by numbers of lists, tokens and pages, each compared with a plain form: the
selection's (kv_blocks.hip: 256 and 128 threads, 1024 with scores of their own, the launch that only scores, each for three sizes of
a row of bounds), and the row items' with half the waves (kv_attn.h), which large batches take."""
import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")
from kv_plain import Cache, attention, compare  # noqa: E402
from test_blocks_gpu import dev, filled, listed_keep, new_bounds, say, some_lists, step_of, unpack  # noqa: E402
from test_tree_gpu import tree_keep  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


# ---------------------------------------------------------------- selection
def whole_queries(q):
    """Query rows in whole numbers, and the exponents of their steps."""
    x = q.double().numpy()
    s = np.vectorize(step_of)(np.abs(x).max(-1))
    return np.clip(np.rint(x / 2.0 ** s[..., None]), -127, 127), s


def selected(c, bounds, q, seq, pos, count, sink, recent):
    """kv_plain's tables, scores of a list's pages at once: whole numbers times powers of two, exact in 64 bits."""
    hi, lo, _, f = unpack(bounds.rows, c.dim)
    w, s = whole_queries(q)
    up, down = np.maximum(w, 0), np.minimum(w, 0)
    t, heads, _ = q.shape
    group = heads // c.heads
    out = np.full((t, c.heads, count), -1, np.int32)
    for i in range(t):
        n = pos[i] // c.page + 1
        ids = c.table[seq[i], :n].numpy()
        for h in range(c.heads):
            if n <= count:
                out[i, h, :n] = np.arange(n)
                continue
            g = slice(h * group, (h + 1) * group)
            sums = up[i, g] @ hi[ids, h].astype(np.float64).T + down[i, g] @ lo[ids, h].astype(np.float64).T
            score = (sums * 2.0 ** s[i, g, None]).max(0) * 2.0 ** f[ids, h]
            score[:sink] = score[n - recent:] = np.inf
            out[i, h] = np.sort(np.argsort(-score, kind="stable")[:count])
    return torch.from_numpy(out)


def check_lists(c, heads, tokens, count, sink=1, recent=2, workspace="own"):
    """workspace: the binding's own, or "none": the C call without one."""
    say(f"select {len(tokens)} tokens, {c.heads} heads of {c.dim}, {c.table.shape[1]} pages, count={count} workspace={workspace}")
    bounds = filled(c, new_bounds(c))
    seq, pos = [s for s, _ in tokens], [p for _, p in tokens]
    q = torch.randn((len(tokens), heads, c.dim), generator=torch.Generator().manual_seed(count)).bfloat16()
    blocks = torch.full((len(tokens) + 1, c.heads, count), 77, dtype=torch.int32, device="cuda")
    args = dev(seq), dev(pos), q.cuda()
    if workspace == "own":
        B.lora_kv_block_select(c.view, bounds, *args, blocks, sink=sink, recent=recent)
    else:
        stream = torch.cuda.current_stream().cuda_stream
        B._check(B.lib().lora_kv_block_select(c.view.ref, bounds.ref, args[0].data_ptr(), args[1].data_ptr(), len(tokens), args[2].data_ptr(),
                                              heads * c.dim, c.dim, heads, count, sink, recent, blocks.data_ptr(), None, 0, stream))
    got = blocks.cpu()
    want = selected(c, bounds, q, seq, pos, count, sink, recent)
    assert bool((got[-1] == 77).all()) and torch.equal(got[:-1], want), (got[:-1] != want).nonzero()[:4].tolist()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("t,kv_heads", [(100, 3), (700, 2)])
def test_many_lists(t, kv_heads, dim, fp8):
    """300 lists take workgroups of 256 threads, 1400 of 128; rows of bounds of one, two, four and eight products of 64."""
    c = Cache([930, 500], kv_heads, dim, 8, fp8, seed=dim + t)
    tokens = [(i % 2, (930 if i % 2 == 0 else 500) - 1 - (7 * i) % 480) for i in range(t)]
    check_lists(c, 4 * kv_heads if t < 200 else kv_heads, tokens, 16)
    check_lists(c, kv_heads, tokens, 40, sink=3, recent=9)


@pytest.mark.parametrize("dim", [32, 128, 256])
@pytest.mark.parametrize("n,max_pages", [(2500, None), (9000, None), (300, 3000), (500, 20000)])
@pytest.mark.parametrize("t,workspace", [(33, "own"), (2, "none")])
def test_wide_tables_scored_where_they_are_listed(n, max_pages, dim, t, workspace):
    """More than 2048 pages, and more than 8192, in a table: 1024 threads, which score for themselves where lists are more than 64
    or there is no workspace."""
    c = Cache([n], 2, dim, 1, False, seed=n, max_pages=max_pages)
    assert B.lora_kv_block_select_workspace(c.view, 33) == 0 and B.lora_kv_block_select_workspace(c.view, 2) > 0
    tokens = [(0, n - 1 - (11 * i) % (n // 2)) for i in range(t)]
    check_lists(c, 6, tokens, 64, workspace=workspace)
    check_lists(c, 34 if t == 2 else 2, tokens, min(n // 2, 1500), sink=5, recent=20, workspace=workspace)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [32, 64, 128, 256])
@pytest.mark.parametrize("n", [513, 700, 1900])
def test_few_lists_scored_by_a_launch_of_their_own(n, dim, fp8):
    c = Cache([n], 2, dim, 1, fp8, seed=n + dim)
    assert B.lora_kv_block_select_workspace(c.view, 9) == 9 * 2 * n * 4
    tokens = [(0, n - 1), (0, n // 2), (0, 255), (0, 256), (0, 257), (0, 511), (0, 512), (0, 40), (0, 3)]
    check_lists(c, 8, tokens, 30)
    check_lists(c, 40, tokens, 200, sink=0, recent=1)


# ---------------------------------------------------------------- row items of half the waves
def sampled(t, n=40):
    """Some of t requests, the first and last among them."""
    return sorted(set(np.linspace(0, t - 1, n).astype(int).tolist()))


def lengths(t, most):
    return [1 + (37 * i) % most for i in range(t)]


@pytest.mark.parametrize("dim", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("window", [0, 20])
def test_many_tokens_over_8_bit_rows(dim, window):
    """1280 units of a request and KV head and more."""
    t, kv_heads, heads = 165, 8, 24
    kv_lens = lengths(t, 150)
    c = Cache(kv_lens, kv_heads, dim, 24, True, seed=dim)
    plan = B.lora_kv_attn_plan(list(range(t + 1)), list(range(t)), kv_lens, heads, kv_heads, dim, window=window).to("cuda")
    assert plan.desc.num_row_items * kv_heads >= 1280 and plan.desc.num_tile_items == 0
    say(f"half the waves, 8-bit, dim={dim} window={window}: {plan.desc.num_row_items * kv_heads} workgroups")
    q = (torch.randn((t, heads, dim), generator=torch.Generator().manual_seed(1)) * 1.5).bfloat16()
    out, lse = torch.full((t + 1, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((t + 1, heads), 9.0, device="cuda")
    B.lora_kv_attn(c.view, plan, torch.cat([q, q[:1]]).cuda(), out, lse=lse)
    assert bool((out[t] == 9).all()) and bool((lse[t] == 9).all())
    for i in sampled(t):
        n = kv_lens[i]
        keep = torch.ones((1, n), dtype=torch.bool)
        if window:
            keep[0, : max(0, n - window)] = False
        compare(out[i: i + 1], lse[i: i + 1], *attention(q[i: i + 1], c.k[i], c.v[i], keep, dim ** -0.5), dim, i)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("window", [0, 20])
def test_many_small_trees(dim, fp8, window):
    """One or two nodes each."""
    r, kv_heads, heads = 165, 8, 24
    sizes = [1 + i % 2 for i in range(r)]
    kv_lens = [n + s for n, s in zip(lengths(r, 150), sizes)]
    starts = np.concatenate([[0], np.cumsum(sizes)])
    t = int(starts[-1])
    c = Cache(kv_lens, kv_heads, dim, 24, fp8, seed=dim)
    plan = B.lora_kv_attn_plan(starts, list(range(r)), kv_lens, heads, kv_heads, dim, window=window, tree=True).to("cuda")
    assert plan.desc.num_row_items * kv_heads >= 1280 and plan.desc.num_tile_items == 0
    say(f"half the waves, trees, dim={dim} fp8={fp8} window={window}: {plan.desc.num_row_items * kv_heads} workgroups")
    parents = [[-1] if n == 1 else [-1, i // 2 % 2 - 1] for i, n in enumerate(sizes)]
    tree = B.Tree(t, 2, "cuda")
    B.lora_tree_mask(dev(starts), dev(sum(parents, [])), tree, window=window)
    q = (torch.randn((t, heads, dim), generator=torch.Generator().manual_seed(2)) * 1.5).bfloat16()
    out, lse = torch.full((t + 1, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((t + 1, heads), 9.0, device="cuda")
    B.lora_kv_attn_tree(c.view, plan, tree, torch.cat([q, q[:1]]).cuda(), out, lse=lse)
    assert bool((out[t] == 9).all()) and bool((lse[t] == 9).all())
    for i in sampled(r):
        a, b = int(starts[i]), int(starts[i + 1])
        kept = [[0]] if b - a == 1 else [[0], [0, 1] if parents[i][1] == 0 else [1]]
        keep = tree_keep(kept, [len(x) - 1 for x in kept], kv_lens[i], window, True)
        compare(out[a:b], lse[a:b], *attention(q[a:b], c.k[i], c.v[i], keep, dim ** -0.5), dim, i)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("page,count", [(16, 7), (128, 8), (40, 26)])
def test_many_lists_attended_to(dim, fp8, page, count):
    """1024 lists and more, of up to 112, 1024 and 1040 positions: 8-bit lists above 1024 keep all their waves."""
    t, kv_heads, heads = 130, 8, 16
    c = Cache([1100, 300, 1], kv_heads, dim, page, fp8, seed=dim)
    tokens = [(i % 3, (1099, 299, 0)[i % 3] - (0 if i % 3 == 2 else 2 * i)) for i in range(t)]
    blocks = some_lists(c, tokens, count, dim)
    plan = B.lora_kv_attn_plan(list(range(t + 1)), [s for s, _ in tokens], [count * page] * t, heads, kv_heads, dim, blocks=True).to("cuda")
    assert plan.desc.num_row_items * kv_heads >= 1024
    say(f"half the waves, lists, dim={dim} fp8={fp8} of {count} pages of {page}: {plan.desc.num_row_items * kv_heads} workgroups")
    q = (torch.randn((t, heads, dim), generator=torch.Generator().manual_seed(3)) * 1.5).bfloat16()
    out, lse = torch.full((t + 1, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda"), torch.full((t + 1, heads), 9.0, device="cuda")
    B.lora_kv_attn_blocks(c.view, plan, blocks.cuda(), dev([p for _, p in tokens]), torch.cat([q, q[:1]]).cuda(), out, lse=lse)
    assert bool((out[t] == 9).all()) and bool((lse[t] == 9).all())
    for i in sampled(t, 25):
        s, p = tokens[i]
        keep = listed_keep(blocks[i: i + 1], [p], c.kv_lens[s], page, c.table.shape[1])
        compare(out[i: i + 1], lse[i: i + 1], *attention(q[i: i + 1], c.k[s], c.v[s], keep, dim ** -0.5), dim, i)
