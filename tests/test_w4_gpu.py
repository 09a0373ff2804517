"""The 4-bit base projection (lora_w4.h) against its definition in 64 bits.

Two kinds of check.  With integer activations, integer zero points and power-of-two
scales every product and partial sum is exact in fp32, so the result has to
equal the once-rounded exact one bit for bit: any wrong index, code, scale or
zero point shows.  With random inputs the error is bounded by the arithmetic:
one rounding of y (bf16: at most 2^-8 of it), and per group the fp32 sums of
terms (128 + u) x and (128 + z) x, each at most 144 |x|, over at most group + 4
additions, so 2^-24 (group + 4) (144 + 144) s sum |x|; the sum over the groups
adds 2^-24 per group of the terms' magnitudes, below the same bound."""
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


def make(n, k, group, zeros, dtype, seed, exact, signed=False):
    """(unsigned codes [n, k], scales, zeros, row-major packed bytes) on the CPU."""
    rng = np.random.default_rng(seed)
    u = rng.integers(0, 16, (n, k))
    g = k // group
    if exact:
        s = torch.from_numpy(2.0 ** rng.integers(-6, -2, (g, n)))
    else:
        s = torch.from_numpy(rng.uniform(0.5, 1.5, (g, n)) / (4.6 * np.sqrt(k)))
    s = s.to(dtype)
    z = torch.from_numpy(rng.integers(0, 16, (g, n)).astype(np.float64)).to(dtype) if zeros else None
    nib = (u ^ 8) if signed else u
    rows = (nib[:, 0::2] | nib[:, 1::2] << 4).astype(np.uint8)
    return u, s, z, torch.from_numpy(rows)


def dense(u, s, z, group):
    w = torch.from_numpy(u).double()
    zz = 8.0 if z is None else z.double().t().repeat_interleave(group, 1)
    return (w - zz) * s.double().t().repeat_interleave(group, 1)


def device(w, s, z, rows, n, k, group, signed=False):
    codes = B.lora_w4_pack(rows.cuda(), twos_complement=signed)
    return B.W4Weights(n, k, group, codes, s.cuda(), None if z is None else z.cuda())


SHAPES = [(1, 8, 32), (1, 16, 128), (2, 24, 160), (16, 64, 512), (17, 72, 544), (33, 1000, 672), (64, 264, 1184),
          (65, 40, 2080), (130, 520, 96), (1, 4096, 4096), (5, 1288, 4128)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros,dtype", [(False, torch.bfloat16), (True, torch.bfloat16), (True, torch.float32)])
def test_exact_integers(m, n, k, group, zeros, dtype):
    k = max(group, k // group * group)
    say(f"w4 exact m={m} n={n} k={k} group={group} zeros={zeros} {dtype}")
    u, s, z, rows = make(n, k, group, zeros, dtype, m + n + k + group, True)
    x = torch.from_numpy(np.random.default_rng(m).integers(-3, 4, (m, k)).astype(np.float32)).bfloat16()
    # every partial sum is a multiple of 2^-6 below 2^17: k terms of at most 3 * 15 * 2^-3
    assert k * 3 * 15 / 8 < 2 ** 17
    want = (x.double() @ dense(u, s, z, group).t()).bfloat16()
    y = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    B.lora_base_w4(x.cuda(), device(u, s, z, rows, n, k, group), y)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("n", [8200, 16400])
@pytest.mark.parametrize("m", [3, 20, 50])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros,dtype", [(False, torch.bfloat16), (False, torch.float32), (True, torch.bfloat16),
                                         (True, torch.float32)])
def test_many_rows(n, m, group, zeros, dtype):
    """So many rows of W that a workgroup takes several row tiles, the last of them past the end."""
    test_exact_integers(m, n, 672, group, zeros, dtype)


@pytest.mark.parametrize("m,n,k,group,zeros,dtype", [
    (1, 4096, 4096, 128, False, torch.bfloat16), (16, 512, 8192, 64, True, torch.float32),
    (40, 136, 14336, 32, True, torch.bfloat16), (200, 256, 1024, 128, False, torch.float32)])
def test_random_against_64_bits(m, n, k, group, zeros, dtype):
    say(f"w4 random m={m} n={n} k={k} group={group}")
    u, s, z, rows = make(n, k, group, zeros, dtype, 7, False)
    gen = torch.Generator().manual_seed(3)
    x = (torch.randn((m, k), generator=gen) + 0.5).bfloat16()  # a mean, so that the offset's part is large
    want = x.double() @ dense(u, s, z, group).t()
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    B.lora_base_w4(x.cuda(), device(u, s, z, rows, n, k, group), y)
    xa = x.double().abs().view(m, k // group, group).sum(-1)  # [m, groups]
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -24 * (group + 4) * 288 * (xa @ s.double())
    assert bool(((y.cpu().double() - want).abs() <= tol).all())
    # and far below that bound as a whole: one rounding of y dominates
    err = (y.cpu().double() - want).norm() / want.norm()
    assert float(err) <= 2.0 ** -8


@pytest.mark.parametrize("signed", [False, True])
def test_pack_layout(signed):
    n, k = 24, 160
    u, s, z, rows = make(n, k, 32, False, torch.float32, 1, True, signed)
    codes = B.lora_w4_pack(rows.cuda(), twos_complement=signed).cpu().numpy()
    assert codes.shape == (2, 2, 64, 16) and codes.size == B.lora_w4_bytes(n, k)
    words = codes.reshape(2, 2, 64, 4, 4).view(np.uint32)[..., 0]
    nib = (0, 4, 1, 5, 2, 6, 3, 7)
    for i in range(32):
        for kk in range(256):
            got = int(words[i // 16, kk // 128, (kk % 32) // 8 * 16 + i % 16, (kk % 128) // 32]) >> (4 * nib[kk % 8]) & 15
            assert got == (u[i, kk] if i < n and kk < k else 8), (i, kk)


def test_column_blocks_and_rows_behind():
    """x and y as column blocks of wider arrays; what lies beside the block and behind the last token stays."""
    n, k, m, group = 72, 192, 19, 64
    u, s, z, rows = make(n, k, group, True, torch.bfloat16, 5, True)
    w = device(u, s, z, rows, n, k, group)
    wide = torch.from_numpy(np.random.default_rng(0).integers(-3, 4, (m, k + 64)).astype(np.float32)).bfloat16()
    out = torch.full((m + 3, n + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    B.lora_base_w4(wide.cuda()[:, 32:32 + k], w, out[:m, 16:16 + n])
    want = torch.full((m + 3, n + 40), 7.0, dtype=torch.bfloat16)
    want[:m, 16:16 + n] = (wide[:, 32:32 + k].double() @ dense(u, s, z, group).t()).bfloat16()
    assert torch.equal(out.cpu(), want)


def test_padding_codes_and_bad_tokens_stay_apart():
    """Codes of padded rows and columns are never used, and a non-finite token reaches its own row only."""
    n, k, m, group = 40, 160, 6, 32
    u, s, z, rows = make(n, k, group, False, torch.float32, 9, True)
    w = device(u, s, z, rows, n, k, group)
    x = torch.from_numpy(np.random.default_rng(2).integers(-3, 4, (m, k)).astype(np.float32)).bfloat16().cuda()
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    B.lora_base_w4(x, w, y)
    words = w.codes.view(3, 2, 4, 16, 4, 4)
    words[2, :, :, 8:] = 0xFF         # rows 40 ..
    words[:, 1, :, :, 1:] = 0xFF      # k 160 ..
    y2 = torch.empty_like(y)
    B.lora_base_w4(x, w, y2)
    assert torch.equal(y, y2)
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    B.lora_base_w4(x, w, y2)
    keep = [0, 1, 2, 5]
    assert torch.equal(y[keep], y2[keep]) and not bool(torch.isfinite(y2[3:5]).any())


def test_empty_call_streams_and_graph():
    n, k, m, group = 256, 512, 3, 128
    u, s, z, rows = make(n, k, group, True, torch.bfloat16, 4, True)
    w = device(u, s, z, rows, n, k, group)
    x = torch.from_numpy(np.random.default_rng(1).integers(-3, 4, (m, k)).astype(np.float32)).bfloat16().cuda()
    want = (x.cpu().double() @ dense(u, s, z, group).t()).bfloat16()
    B.lora_base_w4(x[:0], w, torch.empty((0, n), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    B.lora_base_w4(x, w, y, stream=st)
    st.synchronize()
    assert torch.equal(y.cpu(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        B.lora_base_w4(x, w, y)
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want)


def test_packing_on_another_stream():
    """Codes packed on a stream of their own are not memory that work queued on the current one still writes."""
    n, k = 512, 4096
    u, s, z, rows = make(n, k, 32, False, torch.float32, 6, True)
    rows = rows.cuda()
    want = B.lora_w4_pack(rows)
    big = torch.zeros(1 << 28, dtype=torch.float32, device="cuda")
    old, st = torch.empty_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):  # about 10 ms of work before the write
        big.add_(1)
    old.fill_(0x77)
    del old
    codes = B.lora_w4_pack(rows, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(codes, want)


@pytest.mark.parametrize("m", [1, 17, 40])
@pytest.mark.parametrize("group,power", [(128, 113), (64, 114), (32, 115)])
@pytest.mark.parametrize("zeros", [False, True])
def test_largest_activations(m, group, power, zeros):
    """143 group |x| just below 2^128 (2^127.75): every sum is finite, and exact since x is 1.5 times one power of two."""
    n, k = 48, 2 * group
    assert 2.0 ** 127.5 < 143 * group * 1.5 * 2.0 ** power < 2.0 ** 128
    u, s, z, rows = make(n, k, group, zeros, torch.float32, m + group, True)
    s = s * 2.0 ** -10
    x = torch.full((m, k), 1.5 * 2.0 ** power).bfloat16()
    x[m // 2:] *= -1
    want = (x.double() @ dense(u, s, z, group).t()).bfloat16()
    assert bool(torch.isfinite(want).all())
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    B.lora_base_w4(x.cuda(), device(u, s, z, rows, n, k, group), y)
    assert torch.equal(y.cpu(), want)
