"""Attention at the ends of the range that lora_kv.h states for V: rows whose largest magnitude is about 2^-92 and about 2^100.  Weights
run up to 2^8 while the maximum lags, and 8-bit rows' factors multiply them, so that products and sums go further than
the rows; bounds as kv_plain.py derives them, relative to the rows' own magnitude."""
import pytest

from segmented_gather_gemm_segments_amd import binding as B

torch = pytest.importorskip("torch")
from kv_plain import Cache, attention, causal_keep, compare, starts_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lib()
    return True


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("power", [-92, 98])
@pytest.mark.parametrize("q_lens", [[1, 1], [40, 30]])
def test_rows_at_the_ends(fp8, power, q_lens):
    kv_lens, std, dim = [900, 30], 2.0 ** power, 64
    c = Cache(kv_lens, 2, dim, 16, fp8, seed=power, std=std)
    print(f"[case] range fp8={fp8} 2^{power} q={q_lens}", flush=True)
    scale = 2.0 ** (-power - 2)  # scores from about -20 to 20: weights of every size
    starts = starts_of(q_lens)
    t = int(starts[-1])
    q = (torch.randn((t, 8, dim), generator=torch.Generator().manual_seed(1)) * 1.5).bfloat16()
    plan = B.lora_kv_attn_plan(starts, [0, 1], kv_lens, 8, 2, dim).to("cuda")
    out, lse = torch.empty_like(q, device="cuda"), torch.empty((t, 8), device="cuda")
    B.lora_kv_attn(c.view, plan, q.cuda(), out, lse=lse, scale=scale)
    unit = 2.0 ** -power
    for r, n in enumerate(kv_lens):
        a, b = int(starts[r]), int(starts[r + 1])
        want, want_lse, mass, worst = attention(q[a:b], c.k[r], c.v[r], causal_keep(b - a, n), scale)
        compare(out[a:b].cpu().double() * unit, lse[a:b], want * unit, want_lse, mass * unit, worst, dim, (power, r))
