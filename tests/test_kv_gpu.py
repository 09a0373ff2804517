"""The paged KV cache on the GPU (lora_kv.h): page copies and table rewrites, append, attention of new
tokens, and the sequence bookkeeping's device steps, against plain 64-bit forms.

Attention's bounds.  out: its own rounding and that of the softmax weights to bf16 are at most 2^-8 each,
of |out| and of sum p |v|; a score of head_dim products summed in fp32 is off by at most
2^-24 head_dim sum |q k| scale, which moves every weight by twice that, and exp2 and the running
rescales add a few 2^-22 each, taken as 2^-14 together.  lse: the score's error, plus 2^-24 per added
term (below 2^-12 for these lengths) of 1.  With q = 0 every kept position weighs the same and lse is the
logarithm of their number, which tells exactly which mask was applied."""
import math

import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


def say(msg):
    print(f"[case] {msg}", flush=True)


# ---------------------------------------------------------------- a paged cache and its plain attention
class Paged:
    """Sequences of kv_lens positions in shuffled pages; everything outside them is NaN."""

    def __init__(self, kv_lens, kv_heads, dim, page, seed=0, layout="page", spare=3):
        gen = torch.Generator().manual_seed(seed)
        self.kv_lens, self.page, self.dim = list(kv_lens), page, dim
        need = [-(-n // page) for n in kv_lens]
        total = sum(need) + spare
        ids = torch.randperm(total, generator=gen).int()
        self.table = torch.full((len(need), max(need + [1])), -1, dtype=torch.int32)
        self.k = [torch.randn((n, kv_heads, dim), generator=gen).bfloat16() for n in kv_lens]
        self.v = [torch.randn((n, kv_heads, dim), generator=gen).bfloat16() for n in kv_lens]
        shape = {"page": (total, 2, kv_heads, page, dim), "token": (total, page, 2, kv_heads, dim),
                 "apart": (2, kv_heads, total, page, dim + 8)}[layout]
        store = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        if layout == "page":
            pick = lambda s, i: s[:, i]
        elif layout == "token":
            pick = lambda s, i: s[:, :, i].permute(0, 2, 1, 3)
        else:
            pick = lambda s, i: s[i].permute(1, 0, 2, 3)[..., :dim]
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at: at + n]
            at += n
        for which, rows in ((0, self.k), (1, self.v)):
            part = pick(store, which)
            for i, n in enumerate(kv_lens):
                for j in range(n):
                    part[int(self.table[i, j // page]), :, j % page] = rows[i][j]
        self.store = store.cuda()
        self.view = B.KvView(pick(self.store, 0), pick(self.store, 1), self.table.cuda())


def plain(q, k, v, q_len, kv_len, causal, window, scale):
    """64-bit attention of one request: out, lse, sum p |v|, the largest sum |q k|."""
    t, heads, dim = q.shape
    group = heads // k.shape[1]
    pos = torch.arange(kv_len - q_len, kv_len)[:, None]
    j = torch.arange(kv_len)[None]
    keep = torch.ones((q_len, kv_len), dtype=torch.bool)
    if causal:
        keep &= j <= pos
    if window:
        keep &= j > pos - window
    out = torch.zeros((t, heads, dim), dtype=torch.float64)
    mass = torch.zeros_like(out)
    lse = torch.full((t, heads), -math.inf, dtype=torch.float64)
    worst = 0.0
    for h in range(heads):
        kk, vv, qq = k[:, h // group].double(), v[:, h // group].double(), q[:, h].double()
        for i in range(q_len):
            idx = keep[i].nonzero()[:, 0]
            if idx.numel() == 0:
                continue
            s = (kk[idx] @ qq[i]) * scale
            worst = max(worst, float((kk[idx].abs() @ qq[i].abs()).max()) * abs(scale))
            lse[i, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[i, h])
            out[i, h] = p @ vv[idx]
            mass[i, h] = p @ vv[idx].abs()
    return out, lse, mass, worst


def check_attention(c: Paged, q_lens, heads, causal=True, window=0, max_parts=0, seqs=None, scale=None, q_scale=1.5,
                    label="", kv_lens=None):
    seqs = list(range(len(q_lens))) if seqs is None else seqs
    kv_lens = [c.kv_lens[s] for s in seqs] if kv_lens is None else kv_lens
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    t = int(starts[-1])
    kv_heads = c.view.desc.kv_heads
    say(f"attention {label} q={q_lens} kv={kv_lens} heads={heads}/{kv_heads} dim={c.dim} page={c.page} causal={causal} "
        f"window={window} parts={max_parts}")
    gen = torch.Generator().manual_seed(t + heads)
    q = (torch.randn((t, heads, c.dim), generator=gen) * q_scale).bfloat16()
    plan = B.lora_kv_attn_plan(starts, seqs, kv_lens, heads, kv_heads, c.dim, causal=causal, window=window,
                               max_parts=max_parts, num_seqs=c.table.shape[0], max_kv=c.table.shape[1] * c.page).to("cuda")
    if plan.workspace is not None:
        plan.workspace.fill_(float("nan"))
    out = torch.full((t + 2, heads, c.dim), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((t + 2, heads), 9.0, dtype=torch.float32, device="cuda")
    qd = torch.cat([q, torch.full((2, heads, c.dim), float("nan"), dtype=torch.bfloat16)]).cuda()
    B.lora_kv_attn(c.view, plan, qd, out, lse=lse, scale=scale)
    torch.cuda.synchronize()
    got, got_lse = out.cpu().double(), lse.cpu().double()
    assert bool((got[t:] == 9).all()) and bool((got_lse[t:] == 9).all()), "rows behind the last token were written"
    sc = c.dim ** -0.5 if scale is None else scale
    for r, s in enumerate(seqs):
        a, b = int(starts[r]), int(starts[r + 1])
        want, wl, mass, worst = plain(q[a:b], c.k[s][:kv_lens[r]], c.v[s][:kv_lens[r]], b - a, kv_lens[r], causal, window, sc)
        ds = 2.0 ** -24 * c.dim * worst
        tol = 2.0 ** -8 * (want.abs() + mass) + (2 * ds + 2.0 ** -14) * mass + 1e-30
        assert bool(((got[a:b] - want).abs() <= tol).all()), (
            label, r, float(((got[a:b] - want).abs() - tol).max()))
        none = wl == -math.inf
        assert bool((got_lse[a:b][none] == -math.inf).all()) and bool((got[a:b][none] == 0).all())
        diff = (got_lse[a:b] - wl)[~none].abs()
        assert bool((diff <= ds + 2.0 ** -12 + 2.0 ** -22 * wl[~none].abs()).all()), (label, r, float(diff.max()))
    return plan, qd, out, lse


def check_masks(c: Paged, q_lens, heads, causal, window, max_parts=0, kv_lens=None, seqs=None):
    """q = 0: exp(lse) is the number of kept positions."""
    seqs = list(range(len(q_lens))) if seqs is None else seqs
    kv_lens = [c.kv_lens[s] for s in seqs] if kv_lens is None else kv_lens
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    t = int(starts[-1])
    say(f"masks q={q_lens} kv={kv_lens} causal={causal} window={window}")
    plan = B.lora_kv_attn_plan(starts, seqs, kv_lens, heads, c.view.desc.kv_heads, c.dim, causal=causal, window=window,
                               max_parts=max_parts).to("cuda")
    q = torch.zeros((t, heads, c.dim), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((t, heads), device="cuda")
    B.lora_kv_attn(c.view, plan, q, out, lse=lse)
    n = lse.double().exp().cpu()
    for r in range(len(q_lens)):
        for i in range(q_lens[r]):
            p = kv_lens[r] - q_lens[r] + i
            lo = max(0, p - window + 1) if window else 0
            hi = min(p, kv_lens[r] - 1) if causal else kv_lens[r] - 1
            want = max(0, hi - lo + 1)
            got = n[int(starts[r]) + i]
            assert bool(((got - want).abs() <= 1e-4 * want).all()), (r, i, want, got)


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dim", [8, 40, 64, 80, 96, 128, 168, 256])
def test_decode_head_dims(dim):
    c = Paged([1, 77, 300, 33], 2, dim, 16, seed=dim)
    check_attention(c, [1, 1, 1, 1], 8, label="decode")


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (4, 4), (8, 1), (16, 1), (24, 8), (40, 1), (14, 2)])
def test_head_layouts(heads, kv_heads):
    c = Paged([130, 20], kv_heads, 64, 16, seed=heads)
    check_attention(c, [1, 1], heads, label="decode heads")
    check_attention(c, [9, 20], heads, label="chunk heads")


@pytest.mark.parametrize("page", [1, 3, 8, 24, 33, 64, 128])
def test_page_sizes(page):
    c = Paged([200, 65, 1], 2, 64, page, seed=page)
    check_attention(c, [1, 5, 1], 4, label="pages")
    check_attention(c, [70, 65, 1], 4, label="pages chunk")


@pytest.mark.parametrize("layout", ["page", "token", "apart"])
def test_strides(layout):
    c = Paged([100, 40], 4, 64, 16, seed=3, layout=layout)
    check_attention(c, [1, 1], 8, label=layout)
    check_attention(c, [33, 7], 8, label=layout)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 5, 64, 1000])
def test_masks(causal, window):
    c = Paged([300, 64, 65, 1], 2, 64, 24, seed=1)
    check_attention(c, [90, 64, 2, 1], 4, causal, window, label="masked")
    check_masks(c, [90, 64, 2, 1], 4, causal, window)
    check_masks(c, [1, 1, 1, 1], 4, causal, window)
    check_masks(c, [300, 33, 65, 1], 2, causal, window)


@pytest.mark.parametrize("dim", [40, 64, 80, 128, 256])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("q_len", [1, 40])
def test_many_requests(dim, page, q_len):
    """More requests times KV heads than the card has compute units: other variants than few of them take."""
    kv_lens = [1 + (37 * i) % 190 for i in range(36)]
    c = Paged(kv_lens, 8, dim, page, seed=dim + page)
    q_lens = [min(q_len, n) for n in kv_lens]
    check_attention(c, q_lens, 8 if q_len > 1 else 24, label="many")
    check_attention(c, q_lens, 8, window=50, label="many, windowed")
    check_masks(c, q_lens, 8, True, 50)
    check_masks(c, [q_len] * 36, 8, True, 0)
    check_masks(c, q_lens, 8, False, 0)


@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_len", [3, 70])
def test_many_requests_with_bad_places(dim, bad, q_len):
    """As above, with a position that is not finite and a page that is absent."""
    n, at, many = 150, 150 - q_len + 1, 34
    c = Paged([n], 8, dim, 16, seed=dim)
    plan, q, out, lse = check_attention(c, [q_len] * many, 8, seqs=[0] * many, label="many, clean")
    t = q_len * many
    first = torch.arange(0, t, q_len, device="cuda")
    page, slot = int(c.table[0, at // 16]), at % 16
    for which in (0, 1):
        keep = c.store[page, which, :, slot].clone()
        c.store[page, which, :, slot] = bad
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        B.lora_kv_attn(c.view, plan, q, o2, lse=l2)
        assert torch.equal(o2[first], out[first]) and torch.equal(l2[first], lse[first])
        if which == 1:
            reached = torch.ones(t, dtype=torch.bool, device="cuda")
            reached[first] = False
            assert not bool(torch.isfinite(o2[:t][reached]).any())
        c.store[page, which, :, slot] = keep
    table = c.table.clone()
    table[0, [0, 2]] = torch.tensor([-1, 1 << 30], dtype=torch.int32)
    q0, o2, l2 = torch.zeros_like(q), torch.empty_like(out), torch.empty_like(lse)
    B.lora_kv_attn(B.KvView(c.view.k, c.view.v, table.cuda()), plan, q0, o2, lse=l2)
    want = (torch.arange(q_len) + (n - q_len + 1 - 32)).double().repeat(many)[:, None]
    assert bool(((l2[:t].double().exp().cpu() - want).abs() <= 1e-4 * want).all()) and bool(torch.isfinite(o2[:t]).all())


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_keep_nothing(causal):
    """Chunks longer than their sequence, and sequences without positions."""
    c = Paged([10, 5, 40], 2, 64, 8, seed=4)
    check_masks(c, [13, 3, 1], 4, causal, 0, kv_lens=[10, 0, 40])
    check_masks(c, [30, 9, 50], 4, causal, 7, kv_lens=[3, 5, 40])
    check_attention(c, [13, 3, 1], 4, causal, 0, kv_lens=[10, 0, 40], label="nothing kept")


@pytest.mark.parametrize("max_parts", [1, 2, 7, 64, 0])
def test_ranges_joined(max_parts):
    c = Paged([1500, 700, 2], 2, 128, 16, seed=8)
    check_attention(c, [1, 1, 1], 8, max_parts=max_parts, label="joined")
    check_attention(c, [40, 3, 2], 8, max_parts=max_parts, label="joined chunk")
    check_attention(c, [40, 3, 2], 8, window=300, max_parts=max_parts, label="joined window")


def test_same_sequence_twice_and_scales():
    c = Paged([90, 50], 2, 64, 16, seed=2)
    check_attention(c, [1, 4, 2], 4, seqs=[1, 0, 0], kv_lens=[50, 90, 60], label="twice")
    for scale in (0.0, -0.25, 3.0):
        check_attention(c, [3, 1], 4, scale=scale, label=f"scale {scale}")
    check_attention(c, [3, 1], 4, q_scale=60.0, label="one position takes all")


def test_empty_calls():
    c = Paged([4], 1, 64, 4)
    for q_lens in ([], [0], [0, 0]):
        starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        plan = B.lora_kv_attn_plan(starts, [0] * len(q_lens), [4] * len(q_lens), 2, 1, 64).to("cuda")
        q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
        B.lora_kv_attn(c.view, plan, q, q.clone())
    check_attention(c, [0, 2, 0], 2, seqs=[0, 0, 0], label="requests without tokens")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q_len", [3, 70])
def test_values_behind_the_mask(bad, q_len):
    """A position's K and V reach the tokens that keep it and no others, also where they are not finite."""
    n, at = 150, 150 - q_len + 1  # a position that the chunk's first token does not keep
    c = Paged([n], 2, 64, 16, seed=6)
    plan, q, out, lse = check_attention(c, [q_len], 4, label="clean")
    page, slot = int(c.table[0, at // 16]), at % 16
    for which in (0, 1):
        keep = c.store[page, which, :, slot].clone()
        c.store[page, which, :, slot] = bad
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        B.lora_kv_attn(c.view, plan, q, o2, lse=l2)
        assert torch.equal(o2[:1], out[:1]) and torch.equal(l2[:1], lse[:1])
        if which == 1:
            assert not bool(torch.isfinite(o2[1:q_len]).any())
        c.store[page, which, :, slot] = keep


def test_absent_pages_are_not_seen():
    """A page id out of range hides its positions and nothing else."""
    c = Paged([100], 2, 64, 16, seed=5)
    plan = B.lora_kv_attn_plan([0, 1], [0], [100], 4, 2, 64).to("cuda")
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, 4), device="cuda")
    for gone, want in (([1], 84), ([1, 6], 80), ([0, 1, 2, 3, 4, 5, 6], 0)):
        table = c.table.clone()
        table[0, gone] = torch.tensor([-1, 1 << 30, -7, 99, 99, 99, 99], dtype=torch.int32)[: len(gone)]
        B.lora_kv_attn(B.KvView(c.view.k, c.view.v, table.cuda()), plan, q, out, lse=lse)
        n = lse.double().exp()
        assert bool(((n - want).abs() <= 1e-4 * max(want, 1)).all())
        assert bool(torch.isfinite(out).all())


def test_strided_q_and_out():
    """q as a block of a wider projection, out head-major, lse absent."""
    c = Paged([60, 9], 2, 64, 16, seed=7)
    heads, t = 4, 12
    plan = B.lora_kv_attn_plan([0, 10, 12], [0, 1], [60, 9], heads, 2, 64).to("cuda")
    wide = torch.randn((t, heads * 64 + 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q = wide[:, 64:64 + heads * 64].view(t, heads, 64)
    want = torch.empty((t, heads, 64), dtype=torch.bfloat16, device="cuda")
    B.lora_kv_attn(c.view, plan, q.contiguous(), want)
    got = torch.full((heads, t, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    B.lora_kv_attn(c.view, plan, q, got.permute(1, 0, 2)[..., :64])
    assert torch.equal(got[..., :64].permute(1, 0, 2), want) and bool((got[..., 64:] == 3).all())


def test_attention_repeats_and_graph():
    c = Paged([900, 30, 400], 2, 128, 16, seed=9)
    q_lens = [1, 30, 20]
    plan, q, out, lse = check_attention(c, q_lens, 8, label="repeat")
    t = sum(q_lens)
    st = torch.cuda.Stream()
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        B.lora_kv_attn(c.view, plan, q, o2, lse=l2)
    for _ in range(3):
        o2.zero_()
        l2.zero_()
        plan.workspace is not None and plan.workspace.fill_(float("nan"))
        B.lora_kv_attn(c.view, plan, q, out, lse=lse)  # eager, same workspace, before the replay
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2[:t], out[:t]) and torch.equal(l2[:t], lse[:t])


@pytest.mark.parametrize("reqs", [3, 36])
@pytest.mark.parametrize("q_len", [17, 32])
def test_medium_chunks(reqs, q_len):
    """17 to 32 rows of a request: row items where requests are few, tile items where they are many."""
    c = Paged([40 + 3 * i for i in range(reqs)], 8, 64, 16, seed=reqs)
    plan = check_attention(c, [q_len] * reqs, 8, label="medium")[0]
    assert (plan.desc.num_tile_items > 0) == (reqs * 8 >= 256)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_len", [2, 40])
@pytest.mark.parametrize("max_parts", [2, 64])
def test_bad_places_in_joined_ranges(bad, q_len, max_parts):
    """A value that is not finite reaches the joined rows that keep it and leaves the others bit for bit."""
    n = 3900
    c = Paged([n], 2, 64, 16, seed=12)
    plan, q, out, lse = check_attention(c, [q_len], 4, max_parts=max_parts, label="joined, clean")
    assert plan.desc.num_joins > 0
    at = n - q_len + 1  # not kept by the first token
    page, slot = int(c.table[0, at // 16]), at % 16
    for which in (0, 1):
        keep = c.store[page, which, :, slot].clone()
        c.store[page, which, :, slot] = bad
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        B.lora_kv_attn(c.view, plan, q, o2, lse=l2)
        assert torch.equal(o2[:1], out[:1]) and torch.equal(l2[:1], lse[:1])
        if which == 1 or math.isnan(bad):
            assert not bool(torch.isfinite(o2[1:q_len]).any())
        c.store[page, which, :, slot] = keep


def test_plan_stays_where_it_is():
    plan = B.lora_kv_attn_plan([0, 1], [0], [5000], 2, 1, 64).to("cuda")
    at = plan.items.data_ptr(), plan.workspace.data_ptr()
    assert plan.to("cuda") is plan and plan.to(plan.items.device) is plan
    assert (plan.items.data_ptr(), plan.workspace.data_ptr()) == at


def test_bad_items_are_skipped():
    c = Paged([64], 1, 64, 16)
    plan = B.lora_kv_attn_plan([0, 1], [0], [64], 2, 1, 64).to("cuda")
    q = torch.ones((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    for col, value in ((0, 5), (0, -1), (1, 4), (1, -3), (2, 0), (2, 4000), (3, 1), (3, -1), (5, -2), (6, 1 << 20), (7, 3)):
        say(f"bad item field {col} = {value}")
        bad = plan.items.clone()
        bad[0, col] = value
        p = B.AttnPlan(plan.desc, plan.host_items)
        p.items, p.workspace = bad, None
        out = torch.full((1, 2, 64), 4.0, dtype=torch.bfloat16, device="cuda")
        B.lora_kv_attn(c.view, p, q, out)
        torch.cuda.synchronize()
        assert bool((out == 4).all())


@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("seq,kv_len", [(0, 3000), (3, 900)])
def test_joins_past_the_view_are_skipped(q_len, seq, kv_len):
    """Ranges that reach past the view are skipped, and so is what joins them: out and lse keep what they hold, whatever
    the workspace does."""
    c = Paged([900], 1, 64, 16, seed=2)
    plan = B.lora_kv_attn_plan([0, q_len], [seq], [kv_len], 2, 1, 64, max_parts=4).to("cuda")
    assert plan.desc.num_joins > 0
    plan.workspace.fill_(1.0)
    q = torch.ones((q_len, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 4.0), torch.full((q_len, 2), 4.0, device="cuda")
    with pytest.raises(B.LoraError) as e:
        B.lora_kv_attn(c.view, plan, q, out, lse=lse)
    assert e.value.status == B.LORA_ERANGE
    # the library itself, which learns of it on the device
    strides = q.stride(0), q.stride(1)
    status = B.lib().lora_kv_attn(c.view.ref, plan.ref, plan.items.data_ptr(), q.data_ptr(), *strides, out.data_ptr(), *strides,
                                  lse.data_ptr(), 0.125, plan.workspace.data_ptr(), plan.workspace.nbytes,
                                  torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert status == B.LORA_OK
    assert bool((out == 4).all()) and bool((lse == 4).all())


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dim,page,heads", [(64, 16, 2), (8, 1, 1), (128, 24, 8), (256, 33, 3), (80, 8, 5)])
@pytest.mark.parametrize("layout", ["page", "token"])
def test_append(dim, page, heads, layout):
    say(f"append dim={dim} page={page} heads={heads} {layout}")
    lens = [page * 2 + 1, 1, page * 3]
    c = Paged(lens, heads, dim, page, seed=dim, layout=layout)
    rng = np.random.default_rng(dim)
    places = [(s, p) for s, n in enumerate(lens) for p in range(n)]
    chosen = [places[i] for i in rng.permutation(len(places))[: max(1, len(places) // 2)]]
    # padding and out-of-range tokens among them are skipped
    rows = chosen + [(-1, 0), (-5, 3), (len(lens), 0), (0, -1), (1, c.table.shape[1] * page), (1, page)]
    seq = torch.tensor([s for s, _ in rows], dtype=torch.int32).cuda()
    pos = torch.tensor([p for _, p in rows], dtype=torch.int32).cuda()
    wide = torch.randn((len(rows), 2, heads, dim), generator=torch.Generator().manual_seed(1)).bfloat16()
    want = c.store.clone()
    view = B.KvView(*((want[:, 0], want[:, 1]) if layout == "page" else
                      (want[:, :, 0].permute(0, 2, 1, 3), want[:, :, 1].permute(0, 2, 1, 3))), c.view.page_table)
    for i, (s, p) in enumerate(chosen):
        g = int(c.table[s, p // page])
        view.k[g, :, p % page] = wide[i, 0].cuda()
        view.v[g, :, p % page] = wide[i, 1].cuda()
    dev = wide.cuda()
    B.lora_kv_append(c.view, dev[:, 0], dev[:, 1], seq, pos)
    assert torch.equal(c.store.view(torch.int16), want.view(torch.int16))


def test_append_nothing():
    c = Paged([4], 1, 64, 4)
    before = c.store.clone()
    e = torch.empty((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    i = torch.empty((0,), dtype=torch.int32, device="cuda")
    B.lora_kv_append(c.view, e, e, i, i)
    assert torch.equal(before.view(torch.int16), c.store.view(torch.int16))


# ---------------------------------------------------------------- pages
@pytest.mark.parametrize("shape", [(9, 8), (40, 1000), (64, 16, 512), (5, 131072), (700, 24)])
def test_pages_copy(shape):
    say(f"pages copy {shape}")
    n = shape[0]
    store = torch.randint(-2**15, 2**15, shape, dtype=torch.int16, device="cuda")
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(n)).int()
    h = n // 2
    src = torch.cat([perm[:h], torch.tensor([-1, n, int(perm[h]), 0], dtype=torch.int32)]).cuda()
    dst = torch.cat([perm[h:2 * h], torch.tensor([0, 0, n, -2], dtype=torch.int32)]).cuda()
    same = torch.tensor([int(perm[0])], dtype=torch.int32).cuda()
    want = store.clone()
    want[dst[:h].long()] = store[src[:h].long()]
    B.lora_pages_copy(store, src, dst)
    B.lora_pages_copy(store, same, same)
    B.lora_pages_copy(store, src[:0], dst[:0])
    assert torch.equal(store, want)


def test_page_table_remap():
    n = 1000
    remap = torch.randperm(n, generator=torch.Generator().manual_seed(1)).int().cuda()
    table = torch.randint(-3, n + 3, (37, 61), dtype=torch.int32, device="cuda")
    inside = (table >= 0) & (table < n)
    want = torch.where(inside, remap[table.clamp(0, n - 1).long()], table)
    out = torch.empty_like(table)
    B.lora_page_table_remap(remap, table, out)
    assert torch.equal(out, want)
    B.lora_page_table_remap(remap, table, table)  # in place
    assert torch.equal(table, want)


# ---------------------------------------------------------------- sequences on the device
def test_sequences_fork_copy_compact():
    """Sequences grow, fork, diverge, shrink and are compacted; after each step the cache holds, position by
    position, what a plain list of rows holds."""
    heads, dim, rows, width = 2, 32, 16, 64  # 8 positions per page
    pool = B.Pool(torch.zeros((40, rows, width), dtype=torch.bfloat16, device="cuda"), rows, shuffle_seed=3)
    adapter_pages = pool.alloc(rows * 5)  # the pool's other user
    pool.storage[torch.from_numpy(adapter_pages).long().cuda()] = 5.0
    kv = B.KvCache(pool, heads, dim, max_seqs=6, max_pages=8)
    assert kv.stats()["page_tokens"] == 8
    model, rng, stamp = {}, np.random.default_rng(11), [0]

    def write(seqs):
        """New tokens of each sequence, appended in one call."""
        ids, pos, vals = [], [], []
        for s, n in seqs:
            for p in range(len(model[s]), len(model[s]) + n):
                stamp[0] += 1
                ids.append(s)
                pos.append(p)
                vals.append(stamp[0] % 251)
            model[s] = model[s] + vals[len(vals) - n:] if n else model[s]
        t = torch.tensor(vals, dtype=torch.bfloat16, device="cuda")[:, None, None].expand(-1, heads, dim)
        B.lora_kv_append(kv.view, t.contiguous(), (t + 0).contiguous().neg(),
                         torch.tensor(ids, dtype=torch.int32, device="cuda"),
                         torch.tensor(pos, dtype=torch.int32, device="cuda"))

    def check():
        table = kv.page_table.cpu().numpy()
        k, v = kv.view.k.float().cpu().numpy(), kv.view.v.float().cpu().numpy()
        for s in range(6):
            pages = kv.pages(s)
            assert kv.length(s) == (len(model[s]) if s in model else -1)
            assert table[s, : pages.size].tolist() == pages.tolist() and np.all(table[s, pages.size:] == -1)
            for p, val in enumerate(model.get(s, [])):
                assert np.all(k[pages[p // 8], :, p % 8] == val) and np.all(v[pages[p // 8], :, p % 8] == -val), (s, p)
        assert bool((pool.storage[torch.from_numpy(adapter_pages).long().cuda()] == 5.0).all())

    def grow(seqs):
        kv.extend([s for s, _ in seqs], [n for _, n in seqs])
        for s, _ in seqs:
            model.setdefault(s, [])
        write(seqs)
        check()

    grow([(0, 13), (1, 5)])
    kv.fork(0, [2, 3, 4])
    for s in (2, 3, 4):
        model[s] = list(model[0])
    check()
    assert kv.stats()["shared"] == 2
    grow([(0, 1), (2, 1), (3, 4), (4, 2)])  # each copies the shared half-full page, the last keeps it
    assert kv.stats()["shared"] == 1
    kv.truncate(3, 3)
    model[3] = model[3][:3]
    check()
    grow([(3, 6), (1, 20)])
    kv.free([0, 4])
    del model[0], model[4]
    check()
    moved = kv.compact()
    check()
    held = sorted({int(p) for s in model for p in kv.pages(s)})
    assert moved > 0 and held[-1] <= len(held) + 5 + kv.stats()["spare"]
    for _ in range(30):
        s = int(rng.integers(0, 6))
        if s not in model:
            grow([(s, int(rng.integers(0, 12)))])
        elif rng.random() < 0.3:
            kv.free([s])
            del model[s]
        elif len(model[s]) < 40:
            grow([(s, int(rng.integers(1, 12)))])
        if rng.random() < 0.2:
            kv.compact()
        if rng.random() < 0.3:
            kv.trim()
        check()
    kv.free(sorted(model))
    model.clear()
    assert kv.trim(wait=True) == 0 and pool.num_free() == 40 - 5
    kv.close()
    pool.free(adapter_pages)


def test_bookkeeping_is_refused_under_capture():
    pool = B.Pool(torch.zeros((8, 16, 64), dtype=torch.bfloat16, device="cuda"), 16)
    kv = B.KvCache(pool, 2, 32, 2, 4)
    kv.extend([0], [3])
    torch.cuda.synchronize()
    g, x = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
    with torch.cuda.graph(g):
        x.add_(1)
        for call in (lambda: kv.extend([0], [30]), lambda: kv.fork(0, [1]), lambda: kv.free([0]),
                     lambda: kv.truncate(0, 1), lambda: kv.compact()):
            with pytest.raises(B.LoraError) as e:
                call()
            assert e.value.status == B.LORA_EINVAL
    g.replay()
    torch.cuda.synchronize()
    assert kv.length(0) == 3 and float(x[0]) == 1


@pytest.mark.parametrize("side", [False, True])
def test_a_new_cache_waits_for_the_memory_of_its_table(side):
    """The page table may be a block that work queued on the current stream still writes: it holds -1 all the same."""
    pool = B.Pool(torch.zeros((8, 16, 64), dtype=torch.bfloat16, device="cuda"), 16)
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    big = torch.zeros(1 << 28, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        old = torch.empty((40, 3000), dtype=torch.int32, device="cuda")
        at = old.data_ptr()
        for _ in range(20):  # about 10 ms of work before the write
            big.add_(1)
        old.fill_(7)
        del old
        kv = B.KvCache(pool, 2, 32, 40, 3000)
        assert kv.page_table.data_ptr() == at, "the allocator gave other memory: the case is not the one meant"
    torch.cuda.synchronize()
    assert bool((kv.page_table == -1).all())
    kv.extend([3], [20])
    assert kv.page_table[3, :3].tolist() == kv.pages(3).tolist()


def test_a_cache_is_not_made_under_capture():
    pool = B.Pool(torch.zeros((8, 16, 64), dtype=torch.bfloat16, device="cuda"), 16)
    g, x = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        x.add_(1)
        with pytest.raises(B.LoraError) as e:
            B.KvCache(pool, 2, 32, 2, 4)
        assert e.value.status == B.LORA_EINVAL
    g.replay()
    torch.cuda.synchronize()
    assert float(x[0]) == 1 and pool.num_free() == 8


def test_caches_that_go_during_a_capture():
    """A KvCache (and a pool with one) collected while a graph is captured leaves the capture whole and gives its pages
    back at the next call; closing one there is refused."""
    storage = torch.zeros((8, 16, 64), dtype=torch.bfloat16, device="cuda")
    pool, lost = B.Pool(storage, 16), B.Pool(storage.clone(), 16)
    kept, gone, orphan = B.KvCache(pool, 2, 32, 2, 4), B.KvCache(pool, 2, 32, 2, 4), B.KvCache(lost, 2, 32, 2, 4)
    kept.extend([0], [3])
    gone.extend([0, 1], [9, 3])
    gone.free([1])
    orphan.extend([0], [1])
    torch.cuda.synchronize()
    g, x = torch.cuda.CUDAGraph(), torch.zeros(4, device="cuda")
    with torch.cuda.graph(g):
        x.add_(1)
        for call in (kept.close, kept.trim, pool.close):
            with pytest.raises(B.LoraError) as e:
                call()
            assert e.value.status == B.LORA_EINVAL
        del gone, orphan, lost
        x.add_(1)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert float(x[0]) == 4 and kept.length(0) == 3
    assert pool.num_free() == 8 - 1 - 2 - 1
    kept.extend([0], [1])
    assert pool.num_free() == 8 - 1 and not B._waiting
    kept.close()
    assert pool.num_free() == 8
    pool.close()


# ---------------------------------------------------------------- head dims between the usual ones
@pytest.mark.parametrize("dim", [40, 80, 96, 104, 120, 136, 160, 192, 200, 248])
def test_chunks_of_other_head_dims(dim):
    """Heads that fill none of the kernels' widths, or 96 and 192 whole: few requests and many, single tokens and chunks."""
    c = Paged([150, 64, 65, 1], 2, dim, 24, seed=dim)
    check_attention(c, [70, 64, 2, 1], 4, label="few")
    check_attention(c, [70, 33, 40, 1], 2, False, 30, label="few, windowed", kv_lens=[150, 64, 65, 1])
    check_masks(c, [70, 33, 65, 1], 4, True, 5)
    kv_lens = [1 + (37 * i) % 90 for i in range(36)]
    c = Paged(kv_lens, 8, dim, 16, seed=dim + 1)
    q_lens = [min(40, n) for n in kv_lens]
    check_attention(c, q_lens, 8, label="many")
    check_attention(c, [1] * 36, 24, window=50, label="many, single tokens")
    check_masks(c, q_lens, 8, True, 50)


@pytest.mark.parametrize("dim", [40, 96, 104, 192, 248, 256])
@pytest.mark.parametrize("reqs", [1, 34])
@pytest.mark.parametrize("q_len", [3, 70])
def test_bad_places_with_other_head_dims(dim, reqs, q_len):
    """A position that is not finite reaches the tokens that keep it and no others."""
    n, at = 150, 150 - q_len + 1  # not kept by a chunk's first token
    c = Paged([n], 8, dim, 16, seed=dim)
    plan, q, out, lse = check_attention(c, [q_len] * reqs, 8, seqs=[0] * reqs, label="clean")
    t = q_len * reqs
    first = torch.arange(0, t, q_len, device="cuda")
    others = torch.ones(t, dtype=torch.bool, device="cuda")
    others[first] = False
    page, slot = int(c.table[0, at // 16]), at % 16
    for which, bad in ((0, float("nan")), (0, float("inf")), (1, float("nan")), (1, -float("inf"))):
        keep = c.store[page, which, :, slot].clone()
        c.store[page, which, :, slot] = bad
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        B.lora_kv_attn(c.view, plan, q, o2, lse=l2)
        assert torch.equal(o2[first], out[first]) and torch.equal(l2[first], lse[first])
        if which == 1 or math.isnan(bad):
            assert not bool(torch.isfinite(o2[:t][others]).any())
        c.store[page, which, :, slot] = keep


@pytest.mark.parametrize("dim,max_parts", [(104, 3), (192, 5), (248, 2)])
@pytest.mark.parametrize("q_len", [1, 40])
def test_joined_ranges_of_other_head_dims(dim, max_parts, q_len):
    c = Paged([1300], 2, dim, 16, seed=dim)
    plan = check_attention(c, [q_len], 8, max_parts=max_parts, label="joined")[0]
    assert plan.desc.num_joins > 0


# ---------------------------------------------------------------- a cache above 4 GiB
def test_offsets_past_32_bits():
    """Pages whose byte and element offsets pass 2^32 and 2^31: attention, append and copies reach them."""
    total, heads, page, dim = 20000, 8, 64, 128  # 256 KiB a page, 4.9 GiB
    small = Paged([300, 130], heads, dim, page, seed=31)
    far = torch.tensor([19999, 16383, 16384, 3, 18001, 8191, 8192, 17000, 19000, 12345, 12346], dtype=torch.int32)
    far = far[: small.store.shape[0]]
    assert far.numel() == small.store.shape[0] and total * 2 * heads * page * dim > 2**31
    store = torch.full((total, 2, heads, page, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    store[far.long().cuda()] = small.store
    small.table = torch.where(small.table < 0, small.table, far[small.table.clamp(min=0).long()])
    small.store = store
    small.view = B.KvView(store[:, 0], store[:, 1], small.table.cuda())
    check_attention(small, [1, 1], 64, label="far pages")
    check_attention(small, [70, 40], 16, label="far pages, chunks")
    new = torch.randn((2, 2, heads, dim), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    B.lora_kv_append(small.view, new[:, 0], new[:, 1], torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                     torch.tensor([299, 129], dtype=torch.int32, device="cuda"))
    for i, (s, p) in enumerate(((0, 299), (1, 129))):
        assert torch.equal(store[int(small.table[s, p // page]), :, :, p % page], new[i])
    ids = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    B.lora_pages_copy(store, ids(19999, 5), ids(19998, 16385))
    same = lambda a, b: torch.equal(store[a].view(torch.int16), store[b].view(torch.int16))
    assert same(19998, 19999) and same(16385, 5)
