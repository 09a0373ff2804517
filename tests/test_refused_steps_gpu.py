"""Refused steps of the serving block on the GPU, after which the cache goes on as one that never saw them, bit for bit; and drafts of
forks accepted where their pages part."""
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
D_MODEL, HEADS, KV_HEADS, DIM = 512, 8, 2, 64


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


def make(fp8, max_pages=12):
    from segmented_gather_gemm_segments_amd import runner as R
    return R.ServingBlock(D_MODEL, HEADS, KV_HEADS, DIM, 4, 16, max_seqs=4, max_pages=max_pages, pool_pages=64, seed=3, fp8=fp8, bounds=True)


def call(f, t, seed, *args, **kw):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return f(torch.randn((t, D_MODEL), generator=gen, device="cuda").bfloat16(), *args, torch.arange(t, dtype=torch.int32, device="cuda") % 4, **kw)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_selection_over_too_many_pages(fp8):
    block = make(fp8, max_pages=B.LORA_BLOCKS_MAX_PAGES + 1)
    call(block.step, 70, 1, [0, 1], [69, 1])
    store, lens = block.pool.storage.clone(), [block.kv.length(s) for s in range(4)]
    for seqs, new in (([0], [1]), ([0, 2], [2, 5])):
        with pytest.raises(B.LoraError) as e:
            call(block.step, sum(new), 2, seqs, new, pages=4)
        assert e.value.status == B.LORA_EUNSUPPORTED
    assert torch.equal(block.pool.storage.view(torch.int16), store.view(torch.int16))
    assert [block.kv.length(s) for s in range(4)] == lens
    assert bool(torch.isfinite(call(block.step, 2, 3, [0, 1], [1, 1])).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_a_step_that_fails_late(monkeypatch, fp8):
    """Its rows were appended and their bounds written; the steps after it have the results of a block without it."""
    results = []
    for fails in (False, True):
        block = make(fp8)
        page = block.kv.stats()["page_tokens"]
        call(block.step, 4 * page + 21, 1, [0, 1], [4 * page + 3, 18])
        call(block.draft, 3, 2, [1], [[-1, 0, 0]])
        if fails:
            def broken(*args, **kw):
                raise B.LoraError(B.LORA_EUNSUPPORTED, "too large")
            for name, f, args in (("lora_kv_attn", block.step, ([0, 1], [2 * page, 2])), ("lora_kv_attn_tree", block.draft, ([0, 1], [[-1] * 2 * page, [-1, 0]])),
                                  ("lora_kv_attn_blocks", lambda h, *a: block.step(h, *a, pages=3), ([0, 1], [2 * page, 2]))):
                with monkeypatch.context() as m:
                    m.setattr(B, name, broken)
                    with pytest.raises(B.LoraError):
                        call(f, 2 * page + 2, 7, *args)
        block.accept([1], [[0, 2]])
        k, v = (torch.empty((4 * page + 3, KV_HEADS, DIM), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        B.lora_kv_read(block.kv.view, torch.zeros(len(k), dtype=torch.int32, device="cuda"), torch.arange(len(k), dtype=torch.int32, device="cuda"), k, v)
        codes = block.kv.bounds.rows[torch.from_numpy(block.kv.pages(0)).cuda().long()][..., :-12].clone()
        results.append([k, v, codes, call(block.step, 2, 3, [0, 1], [1, 1], pages=3), call(block.step, 2, 4, [0, 1], [1, 1])])
        assert [block.kv.length(s) for s in range(4)] == [4 * page + 5, 22, -1, -1]
    for a, b in zip(*results):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_siblings_accepted_at_a_page_border(fp8):
    """The page before the drafts is both forks': its bounds are not written."""
    block = make(fp8)
    page = block.kv.stats()["page_tokens"]
    call(block.step, 2 * page, 1, [0], [2 * page])
    block.kv.fork(0, [1])
    call(block.draft, 5, 2, [0, 1], [[-1, 0, 0], [-1, -1]])
    shared = torch.from_numpy(block.kv.pages(0)[:2]).cuda().long()
    block.kv.bounds.rows[shared] = 0x55
    block.accept([0, 1], [[0, 2], []])
    assert bool((block.kv.bounds.rows[shared] == 0x55).all())
    assert [block.kv.length(s) for s in (0, 1)] == [2 * page + 2, 2 * page]
    own = int(block.kv.pages(0)[2])
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = block.kv.bounds.rows[own].clone()
    fresh = torch.zeros_like(block.kv.bounds.rows)
    B.lora_kv_bounds_update(block.kv.view, B.KvBounds(block.kv.view, fresh), i32(0), i32(2 * page), i32(2 * page + 2), 2)
    assert torch.equal(got[..., :-12], fresh[own][..., :-12])


@pytest.mark.parametrize("fp8", [False, True])
def test_bounds_of_a_prompt_beside_single_tokens(fp8):
    """Ranges cut into pieces write what whole ones write."""
    block = make(fp8)
    page = block.kv.stats()["page_tokens"]
    call(block.step, 30, 1, [1, 2, 3], [15, 14, 1])
    call(block.step, 7 * page + 8, 2, [0, 1, 2, 3], [7 * page + 5, 1, 2, 0])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lens = [block.kv.length(s) for s in range(4)]
    fresh = torch.zeros_like(block.kv.bounds.rows)
    B.lora_kv_bounds_update(block.kv.view, B.KvBounds(block.kv.view, fresh), i32([0, 1, 2, 3]), i32([0] * 4), i32(lens), max(lens))
    for s in range(4):
        pages = torch.from_numpy(block.kv.pages(s)).cuda().long()
        assert torch.equal(block.kv.bounds.rows[pages][..., :-12], fresh[pages][..., :-12])


def test_nothing_grows_in_a_capture():
    """Refused before anything is uploaded, which would end the capture: it goes on, and its graph replays."""
    block = make(False)
    call(block.step, 30, 1, [0, 1], [20, 10])
    call(block.draft, 2, 2, [1], [[-1, 0]])
    h, ids, x = torch.zeros((2, D_MODEL), dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    refusals = []
    with torch.cuda.graph(graph, stream=stream):
        x.add_(1)
        for f in (lambda: block.step(h, [0], [2], ids), lambda: block.step(h, [0], [2], ids, pages=3),
                  lambda: block.draft(h, [0], [[-1, 0]], ids), lambda: block.accept([1], [[0]])):
            try:
                f()
            except B.LoraError as e:
                refusals.append(e.status)
        x.add_(1)
    assert refusals == [B.LORA_EINVAL] * 4 and [block.kv.length(s) for s in (0, 1)] == [20, 12]
    graph.replay()
    torch.cuda.synchronize()
    assert bool((x == 2).all())
    block.accept([1], [[0]])
    assert block.kv.length(1) == 11
