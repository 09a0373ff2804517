"""The 8-bit KV cache on the GPU (lora_kv8_view in lora_kv.h): rows quantised by append, read back, and attended to,
against plain 64-bit forms (kv_plain.py, which derives attention's bounds).  Codes, exponents and rows read back are
exact: every product on the way is with a power of two and every rounding the one that the format defines."""
import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")
from kv_plain import Cache, attention, causal_keep, compare, dequantise, quantise, replayed, starts_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


def say(msg):
    print(f"[case] {msg}", flush=True)


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- append and read
def rows_of_every_kind(n, heads, dim, seed):
    """bf16 rows: random ones of many magnitudes, and those whose exponent or codes are special."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((n, heads, dim), generator=gen) * torch.exp2(torch.randint(-40, 40, (n, heads, 1), generator=gen).float())
    x = x.bfloat16()
    kinds = [torch.zeros(dim), torch.full((dim,), float("nan")), torch.full((dim,), 1e-40), torch.full((dim,), 3.3e38),
             torch.full((dim,), -float("inf")), torch.linspace(-448, 448, dim), torch.linspace(0, 1.75, dim),
             torch.linspace(0, 1.7578125, dim), torch.linspace(-2 ** -9, 2 ** -9, dim), -torch.zeros(dim), torch.full((dim,), 2.0 ** -126)]
    for i, row in enumerate(kinds):
        x[i % n, i // n % heads] = row.bfloat16()
    x[-1, -1, 0], x[-1, -1, dim // 2] = float("nan"), float("inf")
    return x


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 176, 256])
@pytest.mark.parametrize("layout", ["page", "token", "apart"])
def test_append_quantises(dim, layout):
    c = Cache([40, 3, 17], 3, dim, 8, True, seed=dim, layout=layout)
    say(f"append8 dim={dim} {layout}")
    seq = [0] * 30 + [1, 2, 2]
    pos = list(range(10, 40)) + [2, 0, 16]
    k, v = rows_of_every_kind(33, 3, dim, 1), rows_of_every_kind(33, 3, dim, 2)
    store, scales = c.store.clone(), c.scales.clone()
    B.lora_kv_append(c.view, k.cuda(), v.cuda(), i32(*seq), i32(*pos))
    got = c.store.cpu(), c.scales.cpu()
    c.store.copy_(store), c.scales.copy_(scales)  # the plain form writes into the same places
    for which, x in ((0, k), (1, v)):
        codes, e = quantise(x)
        for t, (s, p) in enumerate(zip(seq, pos)):
            page, slot = c.place(s, p)
            new, now = torch.from_numpy(codes[t]), c._pick(got[0], which)[page, :, slot, :dim]
            nan = (new & 0x7f) == 0x7f
            assert torch.equal((now & 0x7f) == 0x7f, nan) and torch.equal(now[~nan], new[~nan]), (which, t)
            c.rows(which)[page, :, slot] = now.cuda()
            c.row_scales(which)[page, :, slot] = torch.from_numpy(e[t]).cuda()
    assert torch.equal(c.store.cpu(), got[0]) and torch.equal(c.scales.cpu(), got[1])  # nothing else was written


def test_append_skips_what_has_no_place():
    c = Cache([20, 4], 2, 64, 8, True, seed=1)
    store, scales = c.store.clone(), c.scales.clone()
    x = torch.ones((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    B.lora_kv_append(c.view, x, x, i32(-1, 2, 0, 0, 1, -5), i32(0, 0, -1, 24, 8, 1 << 30))
    assert torch.equal(c.store, store) and torch.equal(c.scales, scales)
    B.lora_kv_append(c.view, x[:0], x[:0], i32(), i32())


@pytest.mark.parametrize("dim", [16, 64, 80, 256])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("layout", ["page", "token", "apart"])
def test_read_gives_back_what_is_stored(dim, fp8, layout):
    c = Cache([50, 9], 2, dim, 8, fp8, seed=dim, layout=layout)
    seq, pos = [0, 0, 1, -1, 0, 0, 1, 0], [0, 49, 8, 0, 31, 31, 9, 56]  # 31 twice; the last two have no row: a NaN one, no page
    wide = torch.full((2, 8, 2, dim + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    k, v = wide[0, :, :, 8: 8 + dim], wide[1, :, :, 8: 8 + dim]
    B.lora_kv_read(c.view, i32(*seq), i32(*pos), k, v)
    for got, rows in ((k, c.k), (v, c.v)):
        for t, (s, p) in enumerate(zip(seq, pos)):
            if t in (3, 7):
                assert bool((got[t] == 5).all())
            elif t != 6:
                assert torch.equal(got[t].cpu().double(), rows[s][p])
    assert bool((wide[..., :8] == 5).all()) and bool((wide[..., 8 + dim:] == 5).all())


def test_every_code_and_exponent_reads_back_exactly():
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 1, 256).expand(1, 1, 255, 256).contiguous()
    e = torch.arange(255, dtype=torch.uint8).view(1, 1, 255)
    table = torch.zeros((1, 1), dtype=torch.int32)
    view = B.KvView(codes.cuda().view(torch.float8_e4m3fn), codes.cuda().view(torch.float8_e4m3fn), table.cuda(), e.cuda(), e.cuda())
    pos = torch.arange(10, 248, dtype=torch.int32)  # what append writes
    k = torch.empty((238, 1, 256), dtype=torch.bfloat16, device="cuda")
    B.lora_kv_read(view, torch.zeros(238, dtype=torch.int32).cuda(), pos.cuda(), k, k.clone())
    want = dequantise(codes[0, 0, 10:248].numpy(), e[0, 0, 10:248].numpy())[:, None]
    got = k.cpu().double()
    ok = torch.isfinite(want) & (want.abs() < 2.0 ** 128)
    assert torch.equal(got[ok], want[ok]) and bool((torch.isnan(got) == torch.isnan(want)).all())


# ---------------------------------------------------------------- attention
def check(c, q_lens, heads, causal=True, window=0, max_parts=0, seqs=None, kv_lens=None, scale=None, label=""):
    seqs = list(range(len(q_lens))) if seqs is None else seqs
    kv_lens = [c.kv_lens[s] for s in seqs] if kv_lens is None else kv_lens
    starts = starts_of(q_lens)
    t = int(starts[-1])
    say(f"attention8 {label} q={q_lens} kv={kv_lens} heads={heads}/{c.heads} dim={c.dim} page={c.page} causal={causal} window={window}")
    gen = torch.Generator().manual_seed(t + heads)
    q = (torch.randn((t, heads, c.dim), generator=gen) * 1.5).bfloat16()
    plan = B.lora_kv_attn_plan(starts, seqs, kv_lens, heads, c.heads, c.dim, causal=causal, window=window, max_parts=max_parts).to("cuda")
    if plan.workspace is not None:
        plan.workspace.fill_(float("nan"))
    qd = torch.cat([q, torch.full((2, heads, c.dim), float("nan"), dtype=torch.bfloat16)]).cuda()
    out = torch.full(qd.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(qd.shape[:2], 9.0, device="cuda")
    B.lora_kv_attn(c.view, plan, qd, out, lse=lse, scale=scale)
    assert bool((out[t:] == 9).all()) and bool((lse[t:] == 9).all()), "rows behind the last token were written"
    for r, s in enumerate(seqs):
        a, b = int(starts[r]), int(starts[r + 1])
        n = kv_lens[r]
        want = attention(q[a:b], c.k[s][:n], c.v[s][:n], causal_keep(b - a, n, causal, window), c.dim ** -0.5 if scale is None else scale)
        compare(out[a:b], lse[a:b], *want, c.dim, (label, r))
    return plan, qd, out, lse


@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 128, 144, 192, 256])
def test_head_dims(dim):
    c = Cache([1, 77, 300, 33], 2, dim, 16, True, seed=dim)
    check(c, [1, 1, 1, 1], 8, label="decode")
    check(c, [1, 70, 40, 20], 8, label="chunks")


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (16, 1), (24, 8), (40, 1), (14, 2)])
def test_head_layouts(heads, kv_heads):
    c = Cache([130, 20], kv_heads, 64, 16, True, seed=heads)
    check(c, [1, 1], heads, label="decode")
    check(c, [9, 20], heads, label="chunk")


@pytest.mark.parametrize("page", [1, 3, 8, 24, 33, 128])
@pytest.mark.parametrize("layout", ["page", "token", "apart"])
def test_pages_and_strides(page, layout):
    c = Cache([200, 65, 1], 2, 64, page, True, seed=page, layout=layout)
    check(c, [1, 5, 1], 4, label=layout)
    check(c, [70, 65, 1], 4, label=layout)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 5, 64, 1000])
def test_masks(causal, window):
    c = Cache([300, 64, 65, 1], 2, 64, 24, True, seed=1)
    check(c, [90, 64, 2, 1], 4, causal, window)
    check(c, [1, 1, 1, 1], 4, causal, window)


@pytest.mark.parametrize("dim", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("q_len", [1, 40])
def test_many_requests(dim, q_len):
    kv_lens = [1 + (37 * i) % 190 for i in range(36)]
    c = Cache(kv_lens, 8, dim, 24, True, seed=dim)
    q_lens = [min(q_len, n) for n in kv_lens]
    check(c, q_lens, 8 if q_len > 1 else 24, label="many")
    check(c, q_lens, 8, window=50, label="many, windowed")


@pytest.mark.parametrize("max_parts", [1, 2, 7, 64, 0])
def test_ranges_joined(max_parts):
    c = Cache([1500, 700, 2], 2, 128, 16, True, seed=8)
    check(c, [1, 1, 1], 8, max_parts=max_parts)
    check(c, [40, 3, 2], 8, max_parts=max_parts)
    check(c, [40, 3, 2], 8, window=300, max_parts=max_parts)


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_keep_nothing(causal):
    c = Cache([10, 5, 40], 2, 64, 8, True, seed=4)
    check(c, [13, 3, 1], 4, causal, 0, kv_lens=[10, 0, 40])
    check(c, [30, 9, 50], 4, causal, 7, kv_lens=[3, 5, 40])


@pytest.mark.parametrize("std", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20])
def test_rows_of_other_magnitudes(std):
    c = Cache([90, 30], 2, 64, 16, True, seed=3, std=std)
    for scale in (1.0 / (8 * std), 0.0, -0.25 / std):
        check(c, [1, 1], 4, scale=scale)
        check(c, [40, 30], 4, scale=scale)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_chunk_is_what_the_same_rows_give_in_bf16(dim):
    """Widened rows enter the same products in the same order: chunks have the bits of a bf16 cache of the same values."""
    c = Cache([333, 90], 2, dim, 24, True, seed=dim)
    rows = torch.full((2, *c.rows(0).shape), float("nan"), dtype=torch.bfloat16, device="cuda")
    for s, n in enumerate(c.kv_lens):
        seq, pos = torch.full((n,), s, dtype=torch.int32).cuda(), torch.arange(n, dtype=torch.int32).cuda()
        k, v = (torch.empty((n, 2, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        B.lora_kv_read(c.view, seq, pos, k, v)
        page = c.table[s].cuda().long()[pos.long() // c.page]
        rows[0][page, :, pos.long() % c.page], rows[1][page, :, pos.long() % c.page] = k, v
    plan, q, out, lse = check(c, [120, 90], 8, label="chunk")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    B.lora_kv_attn(B.KvView(rows[0], rows[1], c.view.page_table), plan, q, o2, lse=l2)
    assert torch.equal(o2[:210], out[:210]) and torch.equal(l2[:210], lse[:210])


@pytest.mark.parametrize("q_len", [3, 70])
@pytest.mark.parametrize("what", ["nan codes", "exponent 255", "both"])
def test_values_behind_the_mask(q_len, what):
    """What stands in a place that a token does not keep never reaches it."""
    n, at = 150, 150 - q_len + 1  # a position that the chunk's first token does not keep
    c = Cache([n], 2, 64, 16, True, seed=6)
    plan, q, out, lse = check(c, [q_len], 4, label="clean")
    page, slot = c.place(0, at)
    for which in (0, 1):
        row, e = c.rows(which)[page, :, slot], c.row_scales(which)[page, :, slot]
        kept = row.clone(), e.clone()
        if what != "exponent 255":
            row[:, ::3] = 0x7f
            row[:, 1::7] = 0xff
        if what != "nan codes":
            e.fill_(255)
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        B.lora_kv_attn(c.view, plan, q, o2, lse=l2)
        assert torch.equal(o2[:1], out[:1]) and torch.equal(l2[:1], lse[:1])
        if which == 1 and what == "nan codes":
            bad = torch.zeros(64, dtype=torch.bool, device="cuda")
            bad[::3] = bad[1::7] = True
            assert bool(torch.isnan(o2[1:q_len][..., bad]).all()) and torch.equal(o2[1:q_len][..., ~bad], out[1:q_len][..., ~bad])
        row.copy_(kept[0]), e.copy_(kept[1])


def test_absent_pages_are_not_seen():
    c = Cache([100], 2, 64, 16, True, seed=5)
    for q_len, heads in ((1, 4), (80, 2)):
        plan = B.lora_kv_attn_plan([0, q_len], [0], [100], heads, 2, 64, causal=False).to("cuda")
        q = torch.zeros((q_len, heads, 64), dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((q_len, heads), device="cuda")
        for gone, want in (([1], 84), ([1, 6], 80), ([0, 1, 2, 3, 4, 5, 6], 0)):
            table = c.table.clone()
            table[0, gone] = torch.tensor([-1, 1 << 30, -7, 99, 99, 99, 99], dtype=torch.int32)[: len(gone)]
            B.lora_kv_attn(c.view_of(table), plan, q, out, lse=lse)
            assert bool(((lse.double().exp() - want).abs() <= 1e-4 * max(want, 1)).all()) and bool(torch.isfinite(out).all())


def test_written_read_and_attended_to_in_a_graph():
    c = Cache([900, 30, 400], 2, 128, 16, True, seed=9)
    q_lens = [1, 30, 20]
    plan, q, out, lse = check(c, q_lens, 8)
    t = sum(q_lens)
    seq = i32(*np.repeat([0, 1, 2], q_lens))
    pos = i32(*np.concatenate([np.arange(n - m, n) for m, n in zip(q_lens, c.kv_lens)]))
    new = torch.randn((2, t, 2, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    back = torch.empty_like(new)

    def run():
        B.lora_kv_append(c.view, new[0], new[1], seq, pos)
        B.lora_kv_read(c.view, seq, pos, back[0], back[1])
        B.lora_kv_attn(c.view, plan, q, out, lse=lse)
    replayed(run, run, [back, out[:t], lse[:t]], lambda: (c.store.sum(), q.float().sum()))


def test_cache_above_4_gib():
    """Places past 2^32 bytes from the first page."""
    page_bytes = 2 * 8 * 64 * 128
    pages = (9 << 30) // 2 // page_bytes
    store = torch.empty((pages, 2, 8, 64, 128), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, 2, 8, 64), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    view = B.KvView(store[:, 0].view(torch.float8_e4m3fn), store[:, 1].view(torch.float8_e4m3fn), table.cuda(), scales[:, 0], scales[:, 1])
    n = 150
    gen = torch.Generator().manual_seed(3)
    k, v = (torch.randn((n, 8, 128), generator=gen).bfloat16() for _ in range(2))
    seq, pos = torch.zeros(n, dtype=torch.int32).cuda(), torch.arange(n, dtype=torch.int32).cuda()
    B.lora_kv_append(view, k.cuda(), v.cuda(), seq, pos)
    k8, v8 = dequantise(*quantise(k)), dequantise(*quantise(v))
    got = torch.empty((2, n, 8, 128), dtype=torch.bfloat16, device="cuda")
    B.lora_kv_read(view, seq, pos, got[0], got[1])
    assert torch.equal(got[0].cpu().double(), k8) and torch.equal(got[1].cpu().double(), v8)
    for q_len in (1, 40):
        q = torch.randn((q_len, 16, 128), generator=gen).bfloat16()
        plan = B.lora_kv_attn_plan([0, q_len], [0], [n], 16, 8, 128).to("cuda")
        out, lse = torch.empty_like(q, device="cuda"), torch.empty((q_len, 16), device="cuda")
        B.lora_kv_attn(view, plan, q.cuda(), out, lse=lse)
        compare(out, lse, *attention(q, k8, v8, causal_keep(q_len, n), 128 ** -0.5), 128)
