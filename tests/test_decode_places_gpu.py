"""The calls around 8-bit rows, trees and listed pages away from the usual place: on two streams at once, over pages and bounds
whose places pass 2^32 bytes, and with one position listed twice.  Results are compared bit for bit with those of the same
calls on one stream over a small cache, which other tests hold against 64 bits."""
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HEADS, KV, DIM, PAGE, N, NODES = 16, 8, 128, 64, 300, 20


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Place:
    """A cache of one sequence on the named pages, rows, exponents and bounds of a page side by side, and the calls of a
    step over it."""

    def __init__(self, fp8, pages, ids, max_pages, seed):
        part, row = KV * PAGE * DIM * (1 if fp8 else 2), B.lora_kv_bounds_row_bytes(DIM)
        sizes = [part, part, KV * PAGE, KV * PAGE, KV * row]
        at = [sum(sizes[:i]) for i in range(6)]
        self.buf = torch.empty((pages, at[5]), dtype=torch.uint8, device="cuda")
        cut = lambda i, *shape: self.buf[:, at[i]: at[i + 1]].view(pages, KV, *shape)
        typed = self.buf.view(torch.float8_e4m3fn if fp8 else torch.bfloat16)
        size = 1 if fp8 else 2
        rows = [typed[:, at[i] // size: at[i + 1] // size].view(pages, KV, PAGE, DIM) for i in (0, 1)]
        table = torch.full((1, max_pages), -1, dtype=torch.int32)
        table[0, : len(ids)] = torch.tensor(ids)
        self.view = B.KvView(*rows, table.cuda(), *([cut(2, PAGE), cut(3, PAGE)] if fp8 else []))
        self.bounds = B.KvBounds(self.view, cut(4, row))
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=gen).bfloat16().cuda()
        t = N + NODES
        self.k, self.v, self.q = rand(t, KV, DIM), rand(t, KV, DIM), rand(NODES, HEADS, DIM)
        self.seq, self.pos = torch.zeros(t, dtype=torch.int32, device="cuda"), torch.arange(t, dtype=torch.int32, device="cuda")
        self.one, self.begin, self.end, self.base = i32(0), i32(0), i32(N), i32(N)
        self.starts, self.parent = i32(0, NODES), torch.tensor([(i - 1) // 2 if i else -1 for i in range(NODES)], dtype=torch.int32).cuda()
        self.path = i32(0, 2, 6, 13, -1)[None]
        self.tree = B.Tree(NODES, NODES, "cuda")
        self.tree_plan = B.lora_kv_attn_plan([0, NODES], [0], [t], HEADS, KV, DIM, tree=True, max_parts=3).to("cuda")
        self.list_plan = B.lora_kv_attn_plan(list(range(NODES + 1)), [0] * NODES, [3 * PAGE] * NODES, HEADS, KV, DIM, blocks=True).to("cuda")
        self.blocks = torch.full((NODES, KV, 3), -7, dtype=torch.int32, device="cuda")
        like = lambda x: torch.zeros_like(x)
        self.out, self.listed, self.k_back, self.v_back = like(self.q), like(self.q), like(self.k), like(self.v)
        torch.cuda.synchronize()

    def calls(self):
        last = slice(N - NODES, N)
        return [
            lambda **kw: B.lora_kv_append(self.view, self.k, self.v, self.seq, self.pos, **kw),
            lambda **kw: B.lora_kv_bounds_update(self.view, self.bounds, self.one, self.begin, self.end, N, **kw),
            lambda **kw: B.lora_kv_block_select(self.view, self.bounds, self.seq[:4], self.pos[last][:4], self.q, self.blocks, **kw),
            lambda **kw: B.lora_kv_block_select(self.view, self.bounds, self.seq[last], self.pos[last], self.q, self.blocks, **kw),
            lambda **kw: B.lora_kv_attn_blocks(self.view, self.list_plan, self.blocks, self.pos[last], self.q, self.listed, **kw),
            lambda **kw: B.lora_tree_mask(self.starts, self.parent, self.tree, **kw),
            lambda **kw: B.lora_kv_attn_tree(self.view, self.tree_plan, self.tree, self.q, self.out, **kw),
            lambda **kw: B.lora_kv_keep_path(self.view, self.one, self.base, self.path, **kw),
            lambda **kw: B.lora_kv_read(self.view, self.seq, self.pos, self.k_back, self.v_back, **kw),
        ]

    def results(self):
        torch.cuda.synchronize()
        return [x.cpu() for x in (self.blocks, self.listed, self.tree.mask, self.tree.depth, self.out, self.k_back, self.v_back)]


def same(got, want):
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool(torch.isfinite(got[1]).all() and torch.isfinite(got[4]).all()) and int(got[0].min()) >= 0


def expected(fp8, max_pages, seed):
    p = Place(fp8, 8, [7, 3, 6, 0, 5], max_pages, seed)
    for call in p.calls():
        call()
    return p.results()


@pytest.mark.parametrize("max_pages", [5, 600])  # 600: few lists that may be long take a workspace of the call's stream
@pytest.mark.parametrize("fp8", [False, True])
def test_two_streams_at_once(fp8, max_pages):
    want = [expected(fp8, max_pages, seed) for seed in (1, 2)]
    places = [Place(fp8, 8, [2, 5, 0, 7, 1], max_pages, seed) for seed in (1, 2)]
    streams = [torch.cuda.Stream() for _ in places]
    for steps in zip(*(p.calls() for p in places)):
        for call, stream in zip(steps, streams):
            call(stream=stream)
    for p, w in zip(places, want):
        same(p.results(), w)


@pytest.mark.parametrize("fp8", [False, True])
def test_places_past_4_gib(fp8):
    pages = 36000  # of 131 KiB and more
    p = Place(fp8, pages, [pages - 1, 3, pages - 2, pages // 2, pages - 9], 5, 3)
    assert p.buf.nbytes > 1 << 32
    for call in p.calls():
        call()
    same(p.results(), expected(fp8, 5, 3))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_position_read_twice(fp8):
    p = Place(fp8, 8, [7, 3, 6, 0, 5], 5, 4)
    for call in p.calls():
        call()
    k, v = (torch.zeros((4, KV, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.lora_kv_read(p.view, i32(0, 0, -1, 0), i32(70, 70, 5, 0), k, v)
    for rows, whole in ((k, p.k_back), (v, p.v_back)):
        assert torch.equal(rows[0], whole[70]) and torch.equal(rows[1], whole[70]) and torch.equal(rows[3], whole[0])
        assert not bool(rows[2].any())
