"""Plain forms that the tests of the paged KV cache's 8-bit rows, trees and listed pages share: caches whose rows are known
in 64 bits, E4M3 rounding from its table of values, and attention with any mask.

Attention's bounds.  out: its own rounding and that of the softmax weights to bf16 are at most 2^-8 each, of |out| and of
sum p |v| (for 8-bit rows too: a weight is multiplied by a power of two before it is rounded, and rows enter
the products exactly).  A score of head_dim products summed in fp32 is off by at most 2^-24 head_dim sum |q k| scale, which
moves every weight by twice that; exp2, the running rescales and the join add a few 2^-22 each, taken as 2^-14
together.  lse: the score's error, plus 2^-24 per added term (below 2^-12 for these lengths) of 1."""
import math

import numpy as np
import torch

from segmented_gather_gemm_segments_amd import binding as B


def e4m3_values():
    """The value of each code, NaN for 0x7f and 0xff."""
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(c & 0x7f) == 0x7f] = np.nan
    return np.where(c & 0x80, -v, v)


_VALUES = e4m3_values()
_UP = _VALUES[:0x7f]  # 0 .. 448


def round_e4m3(x):
    """Codes of 64-bit values of magnitude up to 464, to nearest, ties to the even code (which is the even mantissa)."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_UP, a), 1, 126)
    lo = hi - 1
    up, down = _UP[hi] - a, a - _UP[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.signbit(x), c | 0x80, c).astype(np.uint8)


def quantise(x):
    """Codes and exponent bytes of rows (the last dimension) of a bf16 tensor."""
    x = x.double().numpy()
    top = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
    e = np.full(top.shape, -117)
    for bound in range(-117, 121):  # the least e that holds the row
        e = np.where(top > 448 * 2.0 ** bound, bound + 1, e)
    y = np.clip(x, -1.875 * 2.0 ** 127, 1.875 * 2.0 ** 127) * 2.0 ** -e[..., None].astype(np.float64)
    return np.where(np.isfinite(x), round_e4m3(np.where(np.isfinite(x), y, 0)), 0x7f).astype(np.uint8), (e + 127).astype(np.uint8)


def dequantise(codes, e):
    return torch.from_numpy(_VALUES[codes] * 2.0 ** (e.astype(np.float64) - 127)[..., None])


class Cache:
    """Sequences of kv_lens positions in shuffled pages; everything outside them is NaN (and exponent 255).  k and v: per
    sequence [n, kv_heads, dim] in 64 bits, as stored."""

    def __init__(self, kv_lens, kv_heads, dim, page, fp8, seed=0, layout="page", spare=3, std=1.0, max_pages=None):
        gen = torch.Generator().manual_seed(seed)
        self.kv_lens, self.page, self.dim, self.heads, self.fp8 = list(kv_lens), page, dim, kv_heads, fp8
        need = [-(-n // page) for n in kv_lens]
        total = sum(need) + spare
        ids = torch.randperm(total, generator=gen).int()
        width = max(need + [1]) if max_pages is None else max_pages
        self.table = torch.full((len(need), width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at: at + n]
            at += n
        pad = 16 if fp8 else 8
        shape = {"page": (total, 2, kv_heads, page, dim), "token": (total, page, 2, kv_heads, dim),
                 "apart": (2, kv_heads, total, page, dim + pad)}[layout]
        self._pick = {"page": lambda s, i: s[:, i], "token": lambda s, i: s[:, :, i].transpose(1, 2),
                      "apart": lambda s, i: s[i].transpose(0, 1)}[layout]
        rows = lambda s, i: self._pick(s, i)[..., :dim]
        store = torch.full(shape, 0x7f, dtype=torch.uint8) if fp8 else torch.full(shape, float("nan"), dtype=torch.bfloat16)
        scales = torch.full(shape[:-1], 255, dtype=torch.uint8)
        kept = []
        for which in (0, 1):
            kept.append([])
            for i, n in enumerate(kv_lens):
                x = (torch.randn((n, kv_heads, dim), generator=gen) * std).bfloat16()
                if fp8:
                    codes, e = quantise(x) if n else (np.zeros((0, kv_heads, dim), np.uint8), np.zeros((0, kv_heads), np.uint8))
                    kept[-1].append(dequantise(codes, e))
                else:
                    kept[-1].append(x.double())
                if n:
                    j = torch.arange(n)
                    p, slot = self.table[i].long()[j // page], j % page
                    rows(store, which)[p, :, slot] = torch.from_numpy(codes) if fp8 else x
                    if fp8:
                        self._pick(scales, which)[p, :, slot] = torch.from_numpy(e)
        self.k, self.v = kept
        self.store, self.scales = store.cuda(), scales.cuda()
        self.view = self.view_of(self.table)

    def rows(self, which):
        """Stored rows [pages, heads, page, dim]: codes or bf16."""
        return self._pick(self.store, which)[..., : self.dim]

    def row_scales(self, which):
        return self._pick(self.scales, which)

    def view_of(self, table):
        r = [self.rows(i) for i in (0, 1)]
        if not self.fp8:
            return B.KvView(r[0], r[1], table.cuda())
        return B.KvView(r[0].view(torch.float8_e4m3fn), r[1].view(torch.float8_e4m3fn), table.cuda(), self.row_scales(0), self.row_scales(1))

    def place(self, seq, pos):
        return int(self.table[seq, pos // self.page]), pos % self.page


def attention(q, k, v, keep, scale):
    """One request in 64 bits: q [t, heads, dim], k and v [n, kv_heads, dim], keep [t, n] or [t, kv_heads, n] (how often a
    position counts).  out, lse, sum p |v|, the largest sum |q k|."""
    t, heads, dim = q.shape
    kv_heads = k.shape[1]
    group = heads // kv_heads
    if keep.dim() == 2:
        keep = keep[:, None].expand(t, kv_heads, -1)
    keep = keep.double()
    out = torch.zeros((t, heads, dim), dtype=torch.float64)
    mass, lse, worst = torch.zeros_like(out), torch.full((t, heads), -math.inf, dtype=torch.float64), 0.0
    for h in range(heads):
        kk, vv, qq, w = k[:, h // group], v[:, h // group], q[:, h].double(), keep[:, h // group]
        some = w.sum(1) > 0
        if k.shape[0] == 0 or not bool(some.any()):
            continue
        s = torch.nan_to_num(qq @ kk.t(), nan=0.0, posinf=0.0, neginf=0.0) * scale
        worst = max(worst, float(((qq.abs() @ kk.abs().t()) * (w > 0)).nan_to_num(0).max()) * abs(scale))
        s = torch.where(w > 0, s + w.clamp(min=1).log(), -math.inf)
        lse[:, h] = torch.logsumexp(s, 1)
        p = torch.where(some[:, None], torch.softmax(s, 1), 0)
        out[:, h], mass[:, h] = p @ vv, p @ vv.abs()
    return out, lse, mass, worst


def compare(got, got_lse, want, lse, mass, worst, dim, label=""):
    ds = 2.0 ** -24 * dim * worst
    tol = 2.0 ** -8 * (want.abs() + mass) + (2 * ds + 2.0 ** -14) * mass + 1e-30
    off = (got.cpu().double() - want).abs()
    assert bool((off <= tol).all()), (label, float((off - tol).max()))
    none = lse == -math.inf
    got_lse = got_lse.cpu().double()
    assert bool((got_lse[none] == -math.inf).all()) and bool((got.cpu()[none] == 0).all()), label
    diff = (got_lse - lse)[~none].abs()
    assert bool((diff <= ds + 2.0 ** -12 + 2.0 ** -22 * lse[~none].abs()).all()), (label, float(diff.max()) if diff.numel() else 0)


def causal_keep(q_len, kv_len, causal=True, window=0):
    pos, j = torch.arange(kv_len - q_len, kv_len)[:, None], torch.arange(kv_len)[None]
    keep = torch.ones((q_len, kv_len), dtype=torch.bool)
    if causal:
        keep &= j <= pos
    if window:
        keep &= j > pos - window
    return keep


def starts_of(q_lens):
    return np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)


def replayed(eager, capture, outputs, other_work):
    """Captures `capture` on a stream of its own and checks several replays, with other work in between, against `eager`."""
    eager()
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        capture()
    for _ in range(3):
        for t in outputs:
            t.fill_(7)
        other_work()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outputs, want):
            assert torch.equal(t, w)
