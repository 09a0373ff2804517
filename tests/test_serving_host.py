"""What the serving block refuses, without a GPU: a step that cannot run as asked changes nothing and launches nothing,
since its deltas take bare addresses and its cache cannot take growth back."""
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")


class Recorder:
    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        return lambda *args, **kw: self.calls.append(name)


@pytest.fixture
def block(monkeypatch):
    from segmented_gather_gemm_segments_amd import runner as R
    calls = []
    for name in ("lora_base_w4", "lora_bgmv_fused", "lora_kv_append", "lora_kv_attn"):
        monkeypatch.setattr(B, name, getattr(Recorder(calls), name))
    b = object.__new__(R.ServingBlock)
    b.device, b.d_model, b.head_dim, b.q_heads, b.kv_heads = torch.device("cpu"), 128, 32, 4, 2
    b.widths = {"q": (128, 128), "k": (128, 64), "v": (128, 64), "o": (128, 128)}
    b.base = b.delta = dict.fromkeys("qkvo")
    b.kv, b.calls = Recorder(calls), calls
    return b


def rows(t, width=128):
    return torch.zeros((t, width), dtype=torch.bfloat16)


def ids(t):
    return torch.zeros(t, dtype=torch.int32)


@pytest.mark.parametrize("what,hidden,seqs,new,adapters", [
    ("more rows than tokens", rows(4), [0, 1], [1, 2], ids(4)),
    ("fewer rows than tokens", rows(2), [0, 1], [1, 2], ids(2)),
    ("ids for more tokens", rows(3), [0, 1], [1, 2], ids(4)),
    ("ids for fewer tokens", rows(3), [0, 1], [1, 2], ids(2)),
    ("ids in 64 bits", rows(3), [0, 1], [1, 2], ids(3).long()),
    ("ids with a stride", rows(3), [0, 1], [1, 2], ids(6)[::2]),
    ("another width", rows(3, 64), [0, 1], [1, 2], ids(3)),
    ("rows with a stride", rows(3, 256)[:, :128], [0, 1], [1, 2], ids(3)),
    ("another type", rows(3).float(), [0, 1], [1, 2], ids(3)),
    ("a count missing", rows(3), [0, 1], [3], ids(3)),
    ("a negative count", rows(3), [0, 1], [4, -1], ids(3))])
def test_a_refused_step_changes_nothing(block, what, hidden, seqs, new, adapters):
    with pytest.raises(B.LoraError) as e:
        block.step(hidden, seqs, new, adapters)
    assert e.value.status == B.LORA_EINVAL and block.calls == [], what


@pytest.mark.parametrize("x,y,adapters", [
    (rows(3), rows(3, 64), ids(4)), (rows(3), rows(3, 64), ids(2)), (rows(3), rows(3), ids(3)), (rows(2), rows(3, 64), ids(3)),
    (rows(3, 256)[:, :128], rows(3, 64), ids(3)), (rows(3), rows(3, 128)[:, :64], ids(3)), (rows(3), rows(3, 64), ids(3).long())])
def test_a_refused_projection_launches_nothing(block, x, y, adapters):
    with pytest.raises(B.LoraError) as e:
        block.project("k", x, y, adapters)
    assert e.value.status == B.LORA_EINVAL and block.calls == []


def test_a_step_of_no_tokens(block):
    """Sequences may be named with nothing new: they are extended by nothing."""
    y = block.step(rows(0), [0, 1], [0, 0], ids(0))
    assert y.shape == (0, 128) and block.calls == ["extend"]
    assert block.step(rows(0), [], [], ids(0)).shape == (0, 128)


@pytest.mark.parametrize("hidden,adapters", [(rows(3), ids(4)), (rows(3), ids(3).long()), (rows(3).float(), ids(3)),
                                             (rows(3, 256)[:, :128], ids(3)), (rows(3, 64), ids(3))])
def test_a_refused_run_launches_nothing(block, hidden, adapters):
    with pytest.raises(B.LoraError) as e:
        block.run(hidden, None, ids(3), ids(3), adapters)
    assert e.value.status == B.LORA_EINVAL and block.calls == []
