"""8-bit caches, trees and listed pages without a GPU: plans, the layout of a lora_kv's pages, and what every call refuses
(nothing is launched by a refused call; device pointers here are never followed)."""
import ctypes
import itertools

import numpy as np
import pytest

from segmented_gather_gemm_segments_amd import binding as B
from segmented_gather_gemm_segments_amd import build as lbuild


@pytest.fixture(scope="module", autouse=True)
def library():
    if not lbuild.up_to_date():
        lbuild.build()
    return B.lib()


def refused(status, call, *args, **kw):
    with pytest.raises(B.LoraError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value
    return True


# ---------------------------------------------------------------- plans
def covered(plan):
    """(request's first token, row) -> positions of its items, in order; checks the joins on the way."""
    d, items = plan.desc, plan.host_items.tolist()
    main, joins = items[: d.num_row_items + d.num_tile_items], items[d.num_row_items + d.num_tile_items:]
    got = {}
    for qb, row0, rows, seq, pos0, begin, end, part in main:
        assert 1 <= rows <= (B.LORA_ATTN_TILE_ROWS if d.num_tile_items else B.LORA_ATTN_ROWS)
        for r in range(row0, row0 + rows):
            got.setdefault((qb, r), []).append((begin, end, part))
    parts = {}
    for qb, row0, rows, seq, pos0, base, end, n in joins:
        for r in range(row0, row0 + rows):
            parts[(qb, r)] = [base + p * rows for p in range(n)]
    for key, ranges in got.items():
        ranges.sort()
        if key in parts:
            assert sorted(p for _, _, p in ranges) == parts[key]
        else:
            assert len(ranges) == 1 and ranges[0][2] == -1
    assert set(parts) <= set(got)
    return got


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("nodes,kv,heads,kv_heads", [([26], [700], 32, 8), ([1, 61, 7], [40, 8000, 300], 64, 8), ([130], [3000], 16, 16),
                                                     ([10] * 40, [200 + 100 * i for i in range(40)], 64, 8), ([4], [2], 8, 2)])
def test_tree_plans_cover_what_a_node_may_keep(window, nodes, kv, heads, kv_heads):
    starts = np.concatenate([[0], np.cumsum(nodes)])
    for causal in (True, False):
        plan = B.lora_kv_attn_plan(starts, list(range(len(nodes))), kv, heads, kv_heads, 64, window=window, causal=causal, tree=True)
        got = covered(plan)
        group = heads // kv_heads
        for i, (n, m) in enumerate(zip(nodes, kv)):
            for r in range(n * group):
                ranges = got[(int(starts[i]), r)]
                lowest = max(0, m - n - window + 1) if window else 0  # of a node that hangs below the context
                highest = min(m, m - n + r // group + 1) if causal else m
                if highest > lowest:
                    assert ranges[0][0] <= lowest and ranges[-1][1] >= highest, (i, r)
                assert all(a[1] == b[0] for a, b in zip(ranges, ranges[1:]))
        assert plan.desc.flags == B.LORA_ATTN_TREE | (B.LORA_ATTN_CAUSAL if causal else 0)


@pytest.mark.parametrize("tokens,count,page,heads,kv_heads", [(1, 64, 64, 32, 8), (300, 4, 16, 12, 12), (3, 4096, 1, 40, 1), (40, 20, 24, 64, 8)])
def test_list_plans_cover_the_list(tokens, count, page, heads, kv_heads):
    plan = B.lora_kv_attn_plan(range(tokens + 1), [0] * tokens, [count * page] * tokens, heads, kv_heads, 64, blocks=True)
    got = covered(plan)
    assert len(got) == tokens * (heads // kv_heads) and plan.desc.num_tile_items == 0 and plan.desc.flags == B.LORA_ATTN_BLOCKS
    for ranges in got.values():
        assert ranges[0][0] == 0 and ranges[-1][1] == count * page and all(a[1] == b[0] for a, b in zip(ranges, ranges[1:]))


def test_plan_refusals():
    ok = dict(q_starts=[0, 1], seqs=[0], kv_lens=[4], q_heads=4, kv_heads=2, head_dim=64)
    refused(B.LORA_EINVAL, B.lora_kv_attn_plan, **{**ok, "q_starts": [0, 2]}, blocks=True)   # two tokens of one list
    refused(B.LORA_EINVAL, B.lora_kv_attn_plan, **ok, blocks=True, window=3)
    refused(B.LORA_EINVAL, B.lora_kv_attn_plan, **ok, blocks=True, tree=True)
    refused(B.LORA_EUNSUPPORTED, B.lora_kv_attn_plan, **{**ok, "q_starts": [0, 4097]}, tree=True)
    B.lora_kv_attn_plan(**{**ok, "q_starts": [0, 4096]}, tree=True)
    B.lora_kv_attn_plan(**{**ok, "q_starts": [0, 0]}, blocks=True)


# ---------------------------------------------------------------- pages of a lora_kv
class HostPool:
    def __init__(self, pages, page_rows=16, row_width=512):
        self._h, self._kv_handles, self.storage = ctypes.c_void_p(), [], np.zeros((pages, page_rows, row_width), np.uint16)
        B._check(B.lib().lora_pool_create(pages, page_rows, row_width, B.LORA_BF16, B.LORA_WFMT_PLAIN, self.storage.ctypes.data, None, 0,
                                          ctypes.byref(self._h)))


@pytest.mark.parametrize("fp8,bounds", list(itertools.product([False, True], [False, True])))
@pytest.mark.parametrize("heads,dim", [(2, 64), (1, 256), (3, 80), (4, 16)])
def test_positions_of_a_page(fp8, bounds, heads, dim):
    page_bytes = 16 * 512 * 2
    kv = B.KvCache(HostPool(6), heads, dim, 2, 4, host_only=True, fp8=fp8, bounds=bounds)
    row = B.lora_kv_bounds_row_bytes(dim)
    assert row == -(-2 * dim // 64) * 64 + 16
    room = page_bytes - (heads * row if bounds else 0)
    assert kv.stats()["page_tokens"] == room // (2 * heads * (dim + 1 if fp8 else 2 * dim))
    kv.extend([0], [kv.stats()["page_tokens"] + 1])
    assert kv.stats()["pages"] == 2


def test_positions_of_the_benchmarks_pages():
    """What bench.py's help says a page of its serving block holds: 16 rows of 8192, 8 KV heads of 128, with bounds."""
    import pathlib
    held = [B.KvCache(HostPool(2, row_width=8192), 8, 128, 2, 2, host_only=True, fp8=fp8, bounds=True).stats()["page_tokens"] for fp8 in (False, True)]
    text = " ".join((pathlib.Path(__file__).parent.parent / "bench.py").read_text().replace('"', " ").split())
    assert f"{held[0]} positions each, of 8-bit rows {held[1]}" in text


def test_cache_refusals():
    make = lambda **kw: B.KvCache(HostPool(6), **{**dict(kv_heads=2, head_dim=64, max_seqs=2, max_pages=4, host_only=True), **kw})
    refused(B.LORA_EUNSUPPORTED, make, head_dim=72, fp8=True)
    make(head_dim=72, bounds=True)
    refused(B.LORA_EUNSUPPORTED, make, kv_heads=60, head_dim=128, bounds=True)  # no room for a position
    refused(B.LORA_EUNSUPPORTED, lambda: B.lora_kv_bounds_row_bytes(12))
    refused(B.LORA_EUNSUPPORTED, lambda: B.lora_kv_bounds_row_bytes(264))
    kv = make(fp8=True, bounds=True)
    for call, out in (("lora_kv_get_view8", B.lora_kv8_view()), ("lora_kv_get_view", B.lora_kv_view()), ("lora_kv_get_bounds", B.lora_kv_bounds())):
        assert getattr(B.lib(), call)(kv._h, ctypes.byref(out)) == B.LORA_EINVAL  # host only
        assert getattr(B.lib(), call)(kv._h, None) == B.LORA_EINVAL and getattr(B.lib(), call)(None, ctypes.byref(out)) == B.LORA_EINVAL
    h = ctypes.c_void_p()
    assert B.lib().lora_kv_create(kv.pool._h, 2, 64, 2, 4, None, B.LORA_KV_HOST_ONLY | 16, ctypes.byref(h)) == B.LORA_EINVAL


# ---------------------------------------------------------------- refusals of the calls
def view8(**kw):
    d = dict(dtype=B.LORA_FP8_E4M3, head_dim=64, kv_heads=2, page_tokens=16, num_pages=4, num_seqs=1, max_pages=4, reserved=0,
             k=4096, v=8192, page_stride=4096, head_stride=1024, token_stride=64, page_table=64)
    e = dict(k_scales=16384, v_scales=16896, scale_page_stride=64, scale_head_stride=16, scale_token_stride=1)
    for key, value in kw.items():
        (e if key in e else d)[key] = value
    return B.lora_kv8_view(B.lora_kv_view(**d), *e.values())


BAD_VIEWS = [(dict(dtype=3), B.LORA_EUNSUPPORTED), (dict(head_dim=24), B.LORA_EUNSUPPORTED), (dict(head_dim=272), B.LORA_EUNSUPPORTED),
             (dict(k_scales=None), B.LORA_EINVAL), (dict(v_scales=None), B.LORA_EINVAL), (dict(page_stride=4104), B.LORA_EINVAL),
             (dict(token_stride=72), B.LORA_EINVAL), (dict(head_stride=-16), B.LORA_EINVAL), (dict(scale_page_stride=-1), B.LORA_EINVAL),
             (dict(scale_head_stride=-1), B.LORA_EINVAL), (dict(scale_token_stride=-1), B.LORA_EINVAL), (dict(k=4100), B.LORA_EINVAL),
             (dict(page_table=None), B.LORA_EINVAL), (dict(kv_heads=0), B.LORA_EINVAL), (dict(max_pages=2**28), B.LORA_EUNSUPPORTED)]
L = B.lib


def ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.mark.parametrize("name", ["lora_kv_append", "lora_kv_read"])
def test_row_call_refusals(name):
    def call(v, k=16, vv=16, ts=128, hs=64, seq=16, pos=16, n=1):
        return getattr(L(), name)(ref(v), k, vv, ts, hs, seq, pos, n, None)
    for kw, status in BAD_VIEWS:
        assert call(view8(**kw)) == status, kw
    assert call(None) == B.LORA_EINVAL
    for kw in (dict(k=None), dict(vv=None), dict(seq=None), dict(pos=None), dict(k=8), dict(seq=2), dict(ts=4), dict(hs=-8), dict(n=-1)):
        assert call(view8(), **kw) == B.LORA_EINVAL, kw
    assert call(view8(), n=0) == B.LORA_OK and call(view8(num_pages=0)) == B.LORA_OK
    assert call(view8(kv_heads=2**20), n=2**20) == B.LORA_EUNSUPPORTED


def attention_call(name, *mask):
    def call(v, p, m=mask, items=16, q=16, qt=256, qh=64, o=16, ot=256, oh=64, lse=None, scale=0.1, ws=None, wb=0):
        return getattr(L(), name)(ref(v), ref(p), items, *m, q, qt, qh, o, ot, oh, lse, scale, ws, wb, None)
    return call


def check_attention_refusals(call, plan, split):
    for kw, status in BAD_VIEWS:
        assert call(view8(**kw), plan) == status, kw
    assert call(None, plan) == B.LORA_EINVAL and call(view8(), None) == B.LORA_EINVAL
    assert call(view8(kv_heads=1), plan) == B.LORA_EINVAL and call(view8(head_dim=128), plan) == B.LORA_EINVAL
    assert call(view8(scale_page_stride=2**32), plan) == B.LORA_EUNSUPPORTED and call(view8(page_stride=2**37), plan) == B.LORA_EUNSUPPORTED
    for kw in (dict(items=None), dict(q=None), dict(o=None), dict(q=8), dict(o=8), dict(items=8), dict(lse=2),
               dict(qt=4), dict(oh=-8), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(view8(), plan, **kw) == B.LORA_EINVAL, kw
    assert split.workspace_bytes > 0
    for kw in (dict(), dict(ws=16, wb=split.workspace_bytes - 4), dict(ws=8, wb=1 << 30), dict(wb=1 << 30)):
        assert call(view8(), split, **kw) == B.LORA_EINVAL, kw
    # plans of another kind
    for other in (dict(), dict(causal=False), dict(tree=True), dict(blocks=True)):
        p = B.lora_kv_attn_plan([0, 1], [0], [4], 4, 2, 64, **other).desc
        if p.flags & ~B.LORA_ATTN_CAUSAL != plan.flags & ~B.LORA_ATTN_CAUSAL:
            assert call(view8(), p) == B.LORA_EINVAL, other
    bad = B.lora_attn_plan()
    for field, value in (("flags", plan.flags | 32), ("window", -1), ("num_tokens", -1), ("num_joins", 2**30), ("q_heads", 3)):
        ctypes.memmove(ctypes.byref(bad), ctypes.byref(plan), ctypes.sizeof(plan))
        setattr(bad, field, value)
        assert call(view8(), bad) == B.LORA_EINVAL, field


def test_attention_refusals():
    plan = lambda n, **kw: B.lora_kv_attn_plan([0, 1], [0], [n], 4, 2, 64, **kw).desc
    check_attention_refusals(attention_call("lora_kv_attn"), plan(4), plan(9000))


def test_tree_attention_refusals():
    plan = lambda n: B.lora_kv_attn_plan([0, 1], [0], [n], 4, 2, 64, tree=True).desc
    tree = B.lora_tree(64, 64, 1, 1)
    call = attention_call("lora_kv_attn_tree", ctypes.byref(tree))
    check_attention_refusals(call, plan(4), plan(9000))
    assert call(view8(), plan(4), m=(None,)) == B.LORA_EINVAL
    for fields, status in (((64, 64, 0, 1), B.LORA_EUNSUPPORTED), ((64, 64, 65, 1), B.LORA_EUNSUPPORTED), ((None, 64, 1, 1), B.LORA_EINVAL),
                           ((64, None, 1, 1), B.LORA_EINVAL), ((4, 64, 1, 1), B.LORA_EINVAL), ((64, 2, 1, 1), B.LORA_EINVAL),
                           ((64, 64, 1, -1), B.LORA_EINVAL), ((64, 64, 1, 0), B.LORA_EINVAL)):
        assert call(view8(), plan(4), m=(ctypes.byref(B.lora_tree(*fields)),)) == status, fields


def test_list_attention_refusals():
    plan = lambda n: B.lora_kv_attn_plan([0, 1], [0], [n], 4, 2, 64, blocks=True).desc
    call = attention_call("lora_kv_attn_blocks", 64, 4, 64)
    check_attention_refusals(call, plan(4), plan(9000))
    for mask, status in (((None, 4, 64), B.LORA_EINVAL), ((64, 4, None), B.LORA_EINVAL), ((64, 0, 64), B.LORA_EUNSUPPORTED),
                         ((64, 4097, 64), B.LORA_EUNSUPPORTED), ((66, 4, 64), B.LORA_EINVAL), ((64, 4, 62), B.LORA_EINVAL)):
        assert call(view8(), plan(4), m=mask) == status, mask
    assert call(view8(page_tokens=2**28, max_pages=1), plan(4), m=(64, 8, 64)) == B.LORA_EUNSUPPORTED
    tiles = B.lora_kv_attn_plan([0, 40], [0], [64], 4, 2, 64).desc
    tiles.flags = B.LORA_ATTN_BLOCKS
    assert tiles.num_tile_items == 1 and call(view8(), tiles) == B.LORA_EINVAL


def test_tree_mask_and_path_refusals():
    def mask(starts=16, n=1, parent=16, window=0, tree=(64, 64, 1, 1)):
        return L().lora_tree_mask(starts, n, parent, window, ref(None if tree is None else B.lora_tree(*tree)), None)
    for kw in (dict(starts=None), dict(parent=None), dict(starts=2), dict(parent=2), dict(n=-1), dict(window=-1), dict(tree=None), dict(tree=(None, 64, 1, 1))):
        assert mask(**kw) == B.LORA_EINVAL, kw
    assert mask(n=2**24) == B.LORA_EUNSUPPORTED and mask(tree=(64, 64, 65, 1)) == B.LORA_EUNSUPPORTED
    assert mask(n=0) == B.LORA_OK and mask(tree=(None, None, 1, 0)) == B.LORA_OK

    def path(v, seq=16, base=16, p=16, n=1, most=4):
        return L().lora_kv_keep_path(ref(v), seq, base, p, n, most, None)
    for kw, status in BAD_VIEWS:
        assert path(view8(**kw)) == status, kw
    assert path(None) == B.LORA_EINVAL
    for kw in (dict(seq=None), dict(base=None), dict(p=None), dict(seq=2), dict(base=6), dict(p=1), dict(n=-1), dict(most=-1)):
        assert path(view8(), **kw) == B.LORA_EINVAL, kw
    assert path(view8(), n=2**24) == B.LORA_EUNSUPPORTED
    assert path(view8(), n=0) == B.LORA_OK and path(view8(), most=0) == B.LORA_OK and path(view8(num_pages=0)) == B.LORA_OK


def test_bounds_and_selection_refusals():
    good = dict(rows=4096, page_stride=512, head_stride=144)
    bounds = lambda **kw: B.lora_kv_bounds(*{**good, **kw}.values())

    def update(v, b=bounds(), seq=16, begin=16, end=16, n=1, most=4):
        return L().lora_kv_bounds_update(ref(v), ref(b), seq, begin, end, n, most, None)

    def select(v, b=bounds(), seq=16, pos=16, n=1, q=16, qt=256, qh=64, heads=4, count=4, sink=1, recent=1, blocks=16, ws=None, wb=0):
        return L().lora_kv_block_select(ref(v), ref(b), seq, pos, n, q, qt, qh, heads, count, sink, recent, blocks, ws, wb, None)
    for kw, status in BAD_VIEWS:
        assert update(view8(**kw)) == status and select(view8(**kw)) == status, kw
    for call in (update, select):
        assert call(None) == B.LORA_EINVAL and call(view8(), None) == B.LORA_EINVAL
        for kw in (dict(rows=None), dict(rows=4104), dict(page_stride=-16), dict(head_stride=8)):
            assert call(view8(), bounds(**kw)) == B.LORA_EINVAL, kw
    for kw in (dict(seq=None), dict(begin=None), dict(end=None), dict(seq=2), dict(begin=2), dict(end=2), dict(n=-1), dict(most=-1)):
        assert update(view8(), **kw) == B.LORA_EINVAL, kw
    assert update(view8(max_pages=2**20), n=2**10, most=2**25) == B.LORA_EUNSUPPORTED
    assert update(view8(), n=0) == B.LORA_OK and update(view8(), most=0) == B.LORA_OK and update(view8(num_pages=0)) == B.LORA_OK
    for kw in (dict(seq=None), dict(pos=None), dict(q=None), dict(blocks=None), dict(q=8), dict(blocks=2), dict(qt=4), dict(qh=-8), dict(heads=3),
               dict(heads=0), dict(n=-1), dict(count=0), dict(sink=-1), dict(recent=0), dict(sink=3, recent=2), dict(ws=8, wb=64), dict(wb=-1)):
        assert select(view8(), **kw) == B.LORA_EINVAL, kw
    assert select(view8(), count=4097) == B.LORA_EUNSUPPORTED and select(view8(max_pages=32769)) == B.LORA_EUNSUPPORTED
    assert select(view8(), n=2**23) == B.LORA_EUNSUPPORTED and select(view8(), n=0) == B.LORA_OK
    n = ctypes.c_int64(-1)
    space = lambda v, tokens: L().lora_kv_block_select_workspace(ref(v), tokens, ctypes.byref(n))
    assert space(view8(), 4) == B.LORA_OK and n.value == 0
    assert space(view8(max_pages=9000), 4) == B.LORA_OK and n.value == 4 * 2 * 9000 * 4
    assert space(view8(max_pages=9000), 40) == B.LORA_OK and n.value == 0
    assert space(view8(), -1) == B.LORA_EINVAL and space(None, 1) == B.LORA_EINVAL
    assert L().lora_kv_block_select_workspace(ref(view8()), 1, None) == B.LORA_EINVAL


def test_selection_stays_within_one_launch():
    """2^22 lists of 1024 threads would be 2^32."""
    def select(tokens, max_pages, blocks):
        v, b = view8(max_pages=max_pages), B.lora_kv_bounds(4096, 512, 144)
        return L().lora_kv_block_select(ref(v), ref(b), 16, 16, tokens, 16, 256, 64, 4, 4, 1, 1, blocks, None, 0, None)
    for max_pages, most in ((2048, 2**24 - 1), (2049, 2**22 - 1), (32768, 2**22 - 1)):
        assert select(most // 2 + 1, max_pages, None) == B.LORA_EUNSUPPORTED
        assert select(most // 2, max_pages, None) == B.LORA_EINVAL  # taken as far as the null pointer


def test_path_pieces_are_counted_in_31_bits():
    v = view8(kv_heads=2**27, head_dim=128)
    assert L().lora_kv_keep_path(ref(v), 16, 16, 16, 1, 4, None) == B.LORA_EUNSUPPORTED


# ---------------------------------------------------------------- refusals of the binding, on tensors
def test_binding_refusals():
    torch = pytest.importorskip("torch")
    e4m3 = torch.float8_e4m3fn
    k, scales, table = torch.zeros((4, 2, 8, 64)).to(e4m3), torch.zeros((4, 2, 8), dtype=torch.uint8), torch.zeros((1, 4), dtype=torch.int32)
    view = B.KvView(k, k.clone(), table, scales, scales.clone())
    assert view.desc.dtype == B.LORA_FP8_E4M3 and view.desc8.scale_page_stride == 16
    bf = torch.zeros((4, 2, 8, 64), dtype=torch.bfloat16)
    for args in ((k, k), (bf, bf, table, scales, scales), (k, k, table, scales), (k, k, table, scales, scales.int()),
                 (k, k, table, scales, scales[:3]), (k, bf, table, scales, scales),
                 (k, k, table, scales, torch.zeros((4, 8, 2), dtype=torch.uint8).transpose(1, 2))):
        refused(B.LORA_EINVAL, B.KvView, *args) if len(args) > 2 else refused(B.LORA_EINVAL, B.KvView, *args, table)
    i = lambda *x: torch.tensor(x, dtype=torch.int32)
    rows = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    tree = B.Tree(3, 3, "cpu")
    assert tree.mask.shape == (3, 1) and B.Tree(3, 65, "cpu").desc.words == 2
    refused(B.LORA_EUNSUPPORTED, B.Tree, 3, 4097, "cpu")
    bounds = B.KvBounds(view, torch.zeros((4, 2, 144), dtype=torch.uint8))
    for bad in (torch.zeros((4, 2, 128), dtype=torch.uint8), torch.zeros((4, 2, 144), dtype=torch.int8), torch.zeros((3, 2, 144), dtype=torch.uint8)):
        refused(B.LORA_EINVAL, B.KvBounds, view, bad)
    blocks = torch.zeros((1, 2, 4), dtype=torch.int32)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    plan = B.lora_kv_attn_plan([0, 1], [0], [4], 4, 2, 64).to("cpu")
    for call in (lambda: B.lora_kv_read(view, i(0), i(0), rows, rows), lambda: B.lora_tree_mask(i(0, 3), i(-1, 0, 1), tree),
                 lambda: B.lora_kv_keep_path(view, i(0), i(0), i(1)[None]), lambda: B.lora_kv_bounds_update(view, bounds, i(0), i(0), i(1), 1),
                 lambda: B.lora_kv_block_select(view, bounds, i(0), i(0), q, blocks), lambda: B.lora_kv_attn_tree(view, plan, tree, q, q),
                 lambda: B.lora_kv_attn_blocks(view, plan, blocks, i(0), q, q)):
        refused(B.LORA_EINVAL, call)  # not on a GPU
    for call in (lambda: B.lora_tree_mask(i(0, 3).long(), i(-1, 0, 1), tree), lambda: B.lora_tree_mask(i(0, 3), i(-1, 0), tree), lambda: B.lora_tree_mask(i(), i(-1, 0, 1), tree),
                 lambda: B.lora_kv_keep_path(view, i(0), i(0, 1), i(1)[None]), lambda: B.lora_kv_keep_path(view, i(0), i(0), i(1)),
                 lambda: B.lora_kv_bounds_update(view, bounds, i(0), i(0), i(1, 2), 1), lambda: B.lora_kv_bounds_update(view, bounds, i(0, 0)[::2], i(0), i(1), 1),
                 lambda: B.lora_kv_block_select(view, bounds, i(0, 0), i(0, 0), q, blocks), lambda: B.lora_kv_block_select(view, bounds, i(0), i(0), q.float(), blocks),
                 lambda: B.lora_kv_block_select(view, bounds, i(0), i(0), q, blocks[:, :1]), lambda: B.lora_kv_attn_blocks(view, plan, blocks[:, 0], i(0), q, q),
                 lambda: B.lora_kv_attn_blocks(view, plan, blocks, i(), q, q), lambda: B.lora_kv_read(view, i(0), i(0), rows.float(), rows)):
        refused(B.LORA_EINVAL, call)


@pytest.mark.parametrize("pages,heads,dim", [(5, 2, 64), (4, 4, 64), (4, 1, 64), (4, 2, 48), (4, 2, 40), (4, 2, 128)])
def test_bounds_of_another_view(pages, heads, dim):
    """Rows that a view's pages, heads or head size would pass the end of, or read as another's, are refused by name."""
    torch = pytest.importorskip("torch")
    table, i = torch.zeros((1, 4), dtype=torch.int32), lambda *x: torch.tensor(x, dtype=torch.int32)
    make = lambda p, h, d: B.KvView(*(torch.zeros((p, h, 8, d), dtype=torch.bfloat16) for _ in "kv"), table)
    bounds = B.KvBounds(make(4, 2, 64), torch.zeros((4, 2, B.lora_kv_bounds_row_bytes(64)), dtype=torch.uint8))
    view = make(pages, heads, dim)
    for call in (lambda v, h, d: B.lora_kv_bounds_update(v, bounds, i(0), i(0), i(1), 1),
                 lambda v, h, d: B.lora_kv_block_select(v, bounds, i(0), i(0), torch.zeros((1, 4, d), dtype=torch.bfloat16), torch.zeros((1, h, 4), dtype=torch.int32))):
        with pytest.raises(B.LoraError, match="bounds of 4 pages, 2 KV heads of 64"):
            call(view, heads, dim)
        for fits in (make(4, 2, 64), make(3, 2, 64)):
            with pytest.raises(B.LoraError, match="on a GPU"):  # refused for its device alone
                call(fits, 2, 64)
