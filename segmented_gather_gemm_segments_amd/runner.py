"""Puts a generated batch on the GPU and drives the C ABI over it.

Data movement and bookkeeping only: tensors for x, y, v and the adapter
weights (as a dense stack or in a shuffled page pool), the host segment build,
plans, and uploads.  All arithmetic of the delta runs in the library's kernels.
Used by the GPU tests, the benchmark and the smoke check.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional

import numpy as np

from . import binding as B
from .workloads import LoraProblem


def _torch():
    import torch
    return torch


def to_device(arr: np.ndarray, dtype: str, device):
    """numpy (float32, or uint16 bf16 patterns) -> torch tensor on `device`."""
    torch = _torch()
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(arr).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(arr, dtype=np.float32))
    return t.to(device)


def to_host(t, dtype: str) -> np.ndarray:
    """torch tensor -> numpy (float32, or uint16 bf16 patterns)."""
    torch = _torch()
    if dtype == "bf16":
        return t.detach().view(torch.int16).cpu().numpy().view(np.uint16)
    return t.detach().cpu().numpy().astype(np.float32, copy=False)


class DeviceProblem:
    """A LoraProblem resident on one GPU.

    layout: "dense" -- [N, r_max, d] stacks, rows r_a..r_max-1 filled with NaN;
            "paged" -- a lora_pool of 16-row pages, shuffled, unused page rows
                       NaN, A and B^T rows sharing one pool when d_in == d_out.
    Quantized rows (p.wq "fp8" / "int4") are stored as uint8 codes with fp32
    row scales; unused rows hold FP8 NaN codes (0x7f) or INT4 7s and NaN
    scales, so a stray read shows up in the results.
    """

    def __init__(self, p: LoraProblem, device="cuda", layout: Optional[str] = None,
                 page_rows: int = 16, pool_slack: float = 2.0, pool_seed: Optional[int] = None):
        torch = _torch()
        self.p = p
        self.device = torch.device(device)
        self.layout = layout or ("paged" if p.paged else "dense")
        self.tdtype = torch.bfloat16 if p.dtype == "bf16" else torch.float32
        self.cdtype = B.LORA_BF16 if p.dtype == "bf16" else B.LORA_F32
        self.wfmt = {"": B.LORA_WFMT_PLAIN, "fp8": B.LORA_WFMT_FP8_E4M3,
                     "int4": B.LORA_WFMT_INT4}[p.wq]
        assert self.wfmt == B.LORA_WFMT_PLAIN or p.dtype == "bf16"
        self.x = to_device(p.x, p.dtype, self.device)
        self.y0 = to_device(p.y, p.dtype, self.device)
        self.ids = torch.from_numpy(p.ids).to(self.device)
        self.rank = torch.from_numpy(p.ranks.astype(np.int32)).to(self.device)
        self.r_max = p.r_max
        self._pools = []
        self.w = to_device(p.extra["w"], p.dtype, self.device) if "w" in p.extra else None
        if self.layout == "dense":
            self._dense()
        else:
            self._paged(page_rows, pool_slack, p.pool_seed if pool_seed is None else pool_seed)
        self._seg = None

    # ------------------------------------------------------------- weights
    def _row_width(self, d: int) -> int:
        """Last dimension of a stored row: d elements, or its bytes when quantized."""
        return d // 2 if self.wfmt == B.LORA_WFMT_INT4 else d

    def _empty_rows(self, shape):
        torch = _torch()
        if self.wfmt == B.LORA_WFMT_PLAIN:
            return torch.full(shape, float("nan"), dtype=self.tdtype, device=self.device)
        fill = 0x7F if self.wfmt == B.LORA_WFMT_FP8_E4M3 else 0x77
        return torch.full(shape, fill, dtype=torch.uint8, device=self.device)

    def _rows_dev(self, rows):
        torch = _torch()
        if self.wfmt == B.LORA_WFMT_PLAIN:
            return to_device(rows, self.p.dtype, self.device)
        return torch.from_numpy(np.ascontiguousarray(rows, dtype=np.uint8)).to(self.device)

    def _stack(self, rows, scales, d):
        torch = _torch()
        n = len(rows)
        st = self._empty_rows((n, self.r_max, self._row_width(d)))
        sc = None
        if self.wfmt != B.LORA_WFMT_PLAIN:
            sc = torch.full((n * self.r_max,), float("nan"), dtype=torch.float32, device=self.device)
        for a, r in enumerate(rows):
            st[a, : r.shape[0]] = self._rows_dev(r)
            if sc is not None:
                sc[a * self.r_max: a * self.r_max + r.shape[0]] = torch.from_numpy(
                    np.asarray(scales[a], np.float32)).to(self.device)
        return st, sc

    def _dense(self):
        p = self.p
        self.a_pages, a_sc = self._stack(p.a_rows, p.a_scales, p.d_in)
        self.b_pages, b_sc = self._stack(p.bt_rows, p.bt_scales, p.d_out)
        self.weights = B.Weights(self.cdtype, p.d_in, p.d_out, self.r_max, self.r_max,
                                 self.a_pages, self.b_pages, self.rank, p.ranks.astype(np.int32),
                                 weight_format=self.wfmt, a_scales=a_sc, b_scales=b_sc)

    def _paged(self, page_rows, slack, seed):
        torch = _torch()
        p = self.p
        pages_a = sum((int(r) + page_rows - 1) // page_rows for r in p.ranks)
        shared = p.d_in == p.d_out
        max_pages = (self.r_max + page_rows - 1) // page_rows

        quant = self.wfmt != B.LORA_WFMT_PLAIN

        def make_pool(n_pages, d, s):
            storage = self._empty_rows((n_pages, page_rows, self._row_width(d)))
            scales = None
            if quant:
                scales = torch.full((n_pages * page_rows,), float("nan"), dtype=torch.float32,
                                    device=self.device)
            pool = B.Pool(storage, page_rows, shuffle_seed=s, weight_format=self.wfmt,
                          scales=scales)
            self._pools.append(pool)
            return pool

        def scales_dev(lst, a):
            if not quant:
                return None
            return torch.from_numpy(np.asarray(lst[a], np.float32)).to(self.device)

        if shared:
            cap = int(np.ceil(2 * pages_a * slack))
            pool_a = pool_b = make_pool(cap, p.d_in, seed * 7919 + 1)
        else:
            cap = int(np.ceil(pages_a * slack))
            pool_a = make_pool(cap, p.d_in, seed * 7919 + 1)
            pool_b = make_pool(cap, p.d_out, seed * 7919 + 2)
        a_pt = np.full((p.num_adapters, max_pages), -1, np.int32)
        b_pt = np.full((p.num_adapters, max_pages), -1, np.int32)
        for a in range(p.num_adapters):
            r = int(p.ranks[a])
            ia = pool_a.alloc(r)
            pool_a.write_rows(ia, self._rows_dev(p.a_rows[a]), scales_dev(p.a_scales, a))
            ib = pool_b.alloc(r)
            pool_b.write_rows(ib, self._rows_dev(p.bt_rows[a]), scales_dev(p.bt_scales, a))
            a_pt[a, : ia.size] = ia
            b_pt[a, : ib.size] = ib
        torch.cuda.synchronize(self.device)
        self.host_a_pt, self.host_b_pt = a_pt, b_pt
        self.a_pages, self.b_pages = pool_a.storage, pool_b.storage
        self.weights = B.Weights(self.cdtype, p.d_in, p.d_out, self.r_max, page_rows,
                                 self.a_pages, self.b_pages, self.rank, p.ranks.astype(np.int32),
                                 torch.from_numpy(a_pt).to(self.device),
                                 torch.from_numpy(b_pt).to(self.device), max_pages,
                                 weight_format=self.wfmt, a_scales=pool_a.scales,
                                 b_scales=pool_b.scales)

    def replica(self, with_base: bool = False):
        """The same batch at other device addresses: clones of x, y0 and the
        adapter rows (and row scales), with a descriptor of their own; ids,
        ranks, page tables, segments and (unless with_base) the base weight are
        shared.  Replicas let a benchmark rotate over more bytes than the
        last-level cache holds."""
        r = object.__new__(DeviceProblem)
        r.__dict__.update(self.__dict__)
        r.x = self.x.clone()
        r.y0 = self.y0.clone()
        w = self.weights
        a = w.a_pages.clone()
        b = a if w.b_pages is w.a_pages else w.b_pages.clone()
        sa = None if w.a_scales is None else w.a_scales.clone()
        sb = sa if (w.b_scales is w.a_scales) else (None if w.b_scales is None else w.b_scales.clone())
        r.a_pages, r.b_pages = a, b
        r.weights = dataclasses.replace(w, a_pages=a, b_pages=b, a_scales=sa, b_scales=sb)
        if with_base and self.w is not None:
            r.w = self.w.clone()
        r._pools = []
        return r

    # ------------------------------------------------------------- segments, plans
    def segments(self):
        if self._seg is None:
            torch = _torch()
            perm, starts, adapters = B.lora_segments_build(self.p.ids, self.p.num_adapters)
            self._seg = (perm, starts, adapters,
                         torch.from_numpy(np.ascontiguousarray(perm)).to(self.device))
        return self._seg

    def plan(self, phase: int, policy: int = B.LORA_PATH_AUTO,
             mfma_min_tokens: int = B.LORA_DEFAULT_MFMA_MIN_TOKENS, expand_tile_tokens: int = 0):
        torch = _torch()
        _, starts, adapters, _ = self.segments()
        dim = self.r_max if phase == B.LORA_PHASE_SHRINK else self.p.d_out
        items = B.lora_sgmv_plan(phase, starts, adapters, self.p.num_adapters, dim, policy,
                                 mfma_min_tokens, host_rank=self.p.ranks.astype(np.int32),
                                 expand_tile_tokens=expand_tile_tokens)
        return torch.from_numpy(np.ascontiguousarray(items)).to(self.device)

    def tiled_pays(self, tile_min_tokens: int = 0) -> bool:
        """The library's choice between the tiled and the one-launch shrink
        for this batch (lora_sgmv_tiled_pays)."""
        _, starts, adapters, _ = self.segments()
        return B.lora_sgmv_tiled_pays(starts, adapters, self.p.num_adapters, self.r_max, self.p.d_in, self.cdtype,
                                      self.wfmt, tile_min_tokens, host_rank=self.p.ranks.astype(np.int32))

    def plan_tiled(self, policy: int = B.LORA_PATH_AUTO, tile_min_tokens: int = 0, max_splits: int = 0):
        """Tiled shrink plan on the device: (items, k_splits, workspace or None)."""
        torch = _torch()
        _, starts, adapters, _ = self.segments()
        items, ks = B.lora_sgmv_plan_tiled(starts, adapters, self.p.num_adapters, self.r_max, self.p.d_in,
                                           policy, tile_min_tokens, max_splits,
                                           host_rank=self.p.ranks.astype(np.int32))
        nbytes = B.lora_sgmv_shrink_tiled_workspace(int(starts[-1]), self.r_max, ks)
        ws = torch.empty(nbytes // 4, dtype=torch.float32, device=self.device) if nbytes else None
        return torch.from_numpy(np.ascontiguousarray(items)).to(self.device), ks, ws

    # ------------------------------------------------------------- runs
    def new_v(self):
        torch = _torch()
        return torch.zeros((self.p.num_tokens, max(self.r_max, 1)), dtype=torch.float32,
                           device=self.device)

    def run_sgmv(self, policy: int = B.LORA_PATH_AUTO,
                 mfma_min_tokens: int = B.LORA_DEFAULT_MFMA_MIN_TOKENS, y=None, v=None,
                 tiled: bool = False, tile_min_tokens: int = 0, max_splits: int = 0,
                 expand_tile_tokens: int = 0):
        """shrink then expand over the segmented batch; returns (y, v).
        tiled: the tiled shrink (its own plan, threshold and workspace);
        expand_tile_tokens: the expand plan's MFMA token tile (0: the library's)."""
        _, _, _, perm_d = self.segments()
        ep = self.plan(B.LORA_PHASE_EXPAND, policy, mfma_min_tokens, expand_tile_tokens)
        y = self.y0.clone() if y is None else y
        v = self.new_v() if v is None else v
        if tiled:
            items, ks, ws = self.plan_tiled(policy, tile_min_tokens, max_splits)
            B.lora_sgmv_shrink_tiled(self.weights, perm_d, items, ks, self.x, v, ws)
        else:
            sp = self.plan(B.LORA_PHASE_SHRINK, policy, mfma_min_tokens)
            B.lora_sgmv_shrink(self.weights, perm_d, sp, self.x, v)
        B.lora_sgmv_expand(self.weights, perm_d, ep, v, y)
        return y, v

    def run_bgmv(self, order: int = B.LORA_BGMV_AUTO, y=None, v=None):
        y = self.y0.clone() if y is None else y
        v = self.new_v() if v is None else v
        B.lora_bgmv_shrink(self.weights, self.ids, self.x, v, order)
        B.lora_bgmv_expand(self.weights, self.ids, v, y, order)
        return y, v

    def run_bgmv_fused(self, order: int = B.LORA_BGMV_AUTO, y=None, v=None, grouped: bool = False,
                       token_order=None):
        """Fused per-token delta (one launch); returns (y, v).  grouped: place
        the tokens in the batch's segment order (tokens of an adapter together);
        token_order: an explicit device placement order instead."""
        y = self.y0.clone() if y is None else y
        v = self.new_v() if v is None else v
        if grouped:
            token_order = self.segments()[3]
        B.lora_bgmv_fused(self.weights, self.ids, self.x, y, v, order, token_order=token_order)
        return y, v

    def run_base(self, y=None):
        """Base projection y = x W^T (bf16, through lora_base_gemm); returns y."""
        torch = _torch()
        assert self.w is not None, "problem has no base weight"
        if y is None:
            y = torch.empty((self.p.num_tokens, self.p.d_out), dtype=self.tdtype, device=self.device)
        B.lora_base_gemm(self.x, self.w, y, workspace=self.base_workspace())
        return y

    def base_workspace(self):
        """The split-k workspace of this problem's base GEMM (None if it does
        not split), allocated once."""
        if not hasattr(self, "_base_ws"):
            self._base_ws = B.base_gemm_workspace(self.p.num_tokens, self.p.d_out, self.p.d_in,
                                                  device=self.device)
        return self._base_ws

    def serial_calls(self, y, v, stream=None, policy: int = B.LORA_PATH_AUTO):
        """Adapter-serial comparator: one (shrink, expand) pair of prepared
        launches per segment -- each adapter's tokens as a separate sub-batch,
        through the same kernels -- instead of one launch per phase for all of
        them.  Returns the list of pairs (plans kept alive on the object)."""
        torch = _torch()
        perm, starts, adapters, perm_d = self.segments()
        ranks = self.p.ranks.astype(np.int32)
        pairs, keep = [], []
        for sgi in range(adapters.size):
            st = starts[sgi:sgi + 2]
            ad = adapters[sgi:sgi + 1]
            sp = B.lora_sgmv_plan(B.LORA_PHASE_SHRINK, st, ad, self.p.num_adapters, self.r_max,
                                  policy, host_rank=ranks)
            ep = B.lora_sgmv_plan(B.LORA_PHASE_EXPAND, st, ad, self.p.num_adapters, self.p.d_out,
                                  policy)
            spd = torch.from_numpy(np.ascontiguousarray(sp)).to(self.device)
            epd = torch.from_numpy(np.ascontiguousarray(ep)).to(self.device)
            keep += [spd, epd]
            pairs.append(B.prepare_sgmv(self.weights, perm_d, spd, epd, self.x, v, y, stream=stream))
        self._serial_keep = keep
        return pairs


class ServingBlock:
    """The attention block of a decoder layer as a multi-adapter server runs it: q, k, v and o projections from 4-bit
    base weights, each with its adapters' deltas, and attention over a KV cache whose pages come from the pool that also
    holds the adapters' rows.  Weights and adapters are seeded; the arithmetic is the library's.

    ``step(hidden, seqs, new_tokens)`` runs the new tokens of some sequences (one each for decode, a chunk for a prompt)
    through the block and returns their output; ``fork``, ``free`` and ``compact`` of ``kv`` act on the cache.
    ``draft`` runs trees of drafted tokens instead, and ``accept`` keeps a path of each.  fp8: the cache holds 8-bit rows.
    bounds: its pages hold the bounds of their keys, and ``step`` can attend to a few pages of each sequence."""

    def __init__(self, d_model: int, q_heads: int, kv_heads: int, head_dim: int, num_adapters: int, rank: int,
                 max_seqs: int, max_pages: int, pool_pages: int, group: int = 128, seed: int = 0, device="cuda",
                 fp8: bool = False, bounds: bool = False):
        torch = _torch()
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        gen = torch.Generator(device=device).manual_seed(seed)
        self.device, self.d_model, self.head_dim = device, d_model, head_dim
        self.q_heads, self.kv_heads = q_heads, kv_heads
        self.widths = {"q": (d_model, q_heads * head_dim), "k": (d_model, kv_heads * head_dim),
                       "v": (d_model, kv_heads * head_dim), "o": (q_heads * head_dim, d_model)}
        if q_heads * head_dim != d_model:
            raise ValueError("the pool's rows are as long as the hidden state: q_heads * head_dim == d_model")
        with torch.cuda.device(self.device):
            rows = 16
            storage = torch.zeros((pool_pages, rows, d_model), dtype=torch.bfloat16, device=device)
            self.pool = B.Pool(storage, rows, shuffle_seed=seed + 1)
            # adapters of q and o (square) share the pool with the KV pages; those of k and v have B^T rows of another width
            # and keep them in stacks of their own
            self.base, self.delta, self.rows16, self.scales = {}, {}, {}, {}
            rank_dev = torch.full((num_adapters,), rank, dtype=torch.int32, device=device)
            ranks = np.full(num_adapters, rank, np.int32)
            pages = -(-rank // rows)

            def paged(d):
                table = np.zeros((num_adapters, pages), np.int32)
                for a in range(num_adapters):
                    table[a] = self.pool.alloc(rank)
                    r = (torch.randn((rank, d), generator=gen, device=device) * d ** -0.5).bfloat16()
                    self.pool.write_rows(table[a], r)
                return torch.from_numpy(table).to(device)

            for name, (k, n) in self.widths.items():
                codes = torch.randint(0, 256, (n, k // 2), generator=gen, device=device, dtype=torch.uint8)
                scales = ((0.5 + torch.rand((k // group, n), generator=gen, device=device)) / (4.6 * k ** 0.5)).bfloat16()
                self.rows16[name], self.scales[name] = codes, scales
                self.base[name] = B.W4Weights(n, k, group, B.lora_w4_pack(codes), scales)
                if n == k == d_model:
                    a_pt, b_pt = paged(k), paged(n)
                    self.delta[name] = B.Weights(B.LORA_BF16, k, n, rank, rows, storage, storage, rank_dev, ranks, a_pt, b_pt,
                                                 pages)
                else:
                    a = (torch.randn((num_adapters, rank, k), generator=gen, device=device) * k ** -0.5).bfloat16()
                    b = (torch.randn((num_adapters, rank, n), generator=gen, device=device) * rank ** -0.5).bfloat16()
                    self.delta[name] = B.Weights(B.LORA_BF16, k, n, rank, rank, a, b, rank_dev, ranks)
            self.kv = B.KvCache(self.pool, kv_heads, head_dim, max_seqs, max_pages, fp8=fp8, bounds=bounds)
            self._drafts = {}  # sequence: (its length before the draft, its nodes' parents)

    def project(self, name, x, y, token_adapter):
        """y = W x + B (A x), the base from 4-bit codes, the delta of each token's adapter.  x and y are contiguous, and
        token_adapter names an adapter (or -1) for each of their rows: the delta takes bare addresses."""
        k, n = self.widths[name]
        self._rows(token_adapter, ("x", x, k), ("y", y, n))
        with B._On(self.device, None):
            self._project(name, x, y, token_adapter)

    def _project(self, name, x, y, token_adapter):
        B.lora_base_w4(x, self.base[name], y)
        B.lora_bgmv_fused(self.delta[name], token_adapter, x, y)

    def _rows(self, token_adapter, *named):
        """Checks (name, tensor, width) triples of rows and the adapter ids that go with them; returns their number."""
        torch = _torch()
        t = token_adapter.numel()
        B._tensors(self.device, ("token_adapter", token_adapter, torch.int32),
                   *((name, rows, torch.bfloat16) for name, rows, _ in named))
        B._flat("token_adapter", token_adapter)
        for name, rows, width in named:
            B._flat(name, rows)
            if tuple(rows.shape) != (t, width):
                B._refuse(f"{name} {tuple(rows.shape)}: {(t, width)} wanted for {t} adapter ids")
        return t

    def _new(self, hidden, seqs, new_tokens, token_adapter):
        """Checks the rows of a step; returns its sequences, new tokens and number of tokens."""
        seqs, new_tokens = [int(s) for s in seqs], [int(n) for n in new_tokens]
        t = self._rows(token_adapter, ("hidden", hidden, self.d_model))
        if len(seqs) != len(new_tokens) or any(n < 0 for n in new_tokens) or sum(new_tokens) != t:
            B._refuse(f"{len(seqs)} sequences grow by {new_tokens}, hidden has {t} tokens")
        return seqs, new_tokens, t

    def _places(self, seqs, new_tokens):
        """What a step will need, before any sequence grows: lengths after it, starts, on the device each token's sequence and
        position, and the ranges whose bounds change."""
        with B._On(self.device, None):
            B._not_capturing("sequences cannot grow")
        lens = [max(self.kv.length(s), 0) + n for s, n in zip(seqs, new_tokens)]
        if max(lens) > self.kv.view.max_kv:
            B._refuse(f"sequences of {lens[:8]} positions, the cache holds {self.kv.view.max_kv} of each")
        starts = np.concatenate([[0], np.cumsum(new_tokens)]).astype(np.int32)
        seq = np.repeat(np.asarray(seqs, np.int32), new_tokens)
        pos = np.concatenate([np.arange(n - q, n, dtype=np.int32) for q, n in zip(new_tokens, lens)])
        return lens, starts, self._ints(seq), self._ints(pos), self._ranges(seqs, [n - q for q, n in zip(new_tokens, lens)], lens)

    @contextlib.contextmanager
    def _grown(self, seqs, new_tokens):
        """The sequences longer by their new tokens, which end their drafts (the sequence goes on as it is).  A body that
        raises leaves both as they were."""
        before = [self.kv.length(s) for s in seqs]
        self.kv.extend(seqs, new_tokens)
        drafts = {s: self._drafts.pop(s) for s, n in zip(seqs, new_tokens) if n and s in self._drafts}
        try:
            yield
        except BaseException:
            self._drafts.update(drafts)
            for s, n in zip(seqs, before):
                self.kv.free([s]) if n < 0 else self.kv.truncate(s, n)
            # the page that a growth began on may hold bounds of rows that are gone
            page = self.kv.view.desc.page_tokens
            part = [(s, n) for s, n, new in zip(seqs, before, new_tokens) if new and n > 0 and n % page]
            if self.kv.bounds is not None and part:
                self._bounds(self._ranges([s for s, _ in part], [n - 1 for _, n in part], [n for _, n in part]))
            raise

    def _ints(self, values):
        return _torch().from_numpy(np.ascontiguousarray(values, np.int32)).to(self.device)

    def step(self, hidden, seqs, new_tokens, token_adapter, pages: Optional[int] = None, sink: int = 1, recent: int = 2):
        """hidden [T, d_model] of the new tokens, sequence by sequence; token_adapter int32 [T] on the device.  A call that
        raises leaves the sequences and drafts as they are.  pages: each token attends to that many pages of its sequence
        at most for each KV head, the first `sink`, the last `recent` and those that the bounds of their keys choose; every
        token reads its own pages, so that this is for single tokens and short chunks, or lists that are a small part of the
        context (64 / 8 heads of 128, 64 pages of 64 out of 16384 positions: 1 token 24 us, without 23; 16 tokens 41 and 61,
        64 tokens 89 and 68, 2048 tokens 2450 and 1170; out of 65536: 27 and 53, 49 and 93, 106 and 191, 2900 and 4760)."""
        torch = _torch()
        if pages is not None:
            if self.kv.bounds is None:
                B._refuse("pages are chosen by the bounds of their keys: make the block with bounds=True")
            if not 0 <= sink < sink + recent <= pages <= B.LORA_BLOCKS_MAX_COUNT or recent < 1:
                B._refuse(f"{pages} pages, the first {sink} and the last {recent} among them")
        seqs, new_tokens, t = self._new(hidden, seqs, new_tokens, token_adapter)
        if t == 0:
            self.kv.extend(seqs, new_tokens)
            return torch.empty_like(hidden)
        view = self.kv.view
        if pages is not None:
            need = B.lora_kv_block_select_workspace(view, t)  # refuses what the selection would
        lens, starts, seq, pos, ranges = self._places(seqs, new_tokens)
        if pages is None:
            plan = B.lora_kv_attn_plan(starts, seqs, lens, self.q_heads, self.kv_heads, self.head_dim).to(self.device)
            with self._grown(seqs, new_tokens):
                return self.run(hidden, plan, seq, pos, token_adapter, ranges)
        most = min(pages, max(-(-n // view.desc.page_tokens) for n in lens)) * view.desc.page_tokens
        plan = B.lora_kv_attn_plan(np.arange(t + 1), np.repeat(seqs, new_tokens), [most] * t, self.q_heads, self.kv_heads,
                                   self.head_dim, blocks=True).to(self.device)
        blocks = torch.empty((t, self.kv_heads, pages), dtype=torch.int32, device=self.device)
        workspace = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None

        def attend(q, out):
            B.lora_kv_block_select(view, self.kv.bounds, seq, pos, q, blocks, sink=sink, recent=recent, workspace=workspace)
            B.lora_kv_attn_blocks(view, plan, blocks, pos, q, out)
        with self._grown(seqs, new_tokens):
            return self._run(hidden, seq, pos, token_adapter, ranges, attend)

    def draft(self, hidden, seqs, parents, token_adapter):
        """Runs a tree of drafted tokens for each sequence: parents lists, for each of them, its nodes' parents (a number
        below the node's own, or -1 for the context); hidden [T, d_model] of all nodes.  The nodes take the sequences' next
        positions until ``accept`` keeps a path of them.  A call that raises leaves the sequences and drafts as they are."""
        torch = _torch()
        parents = [[int(p) for p in row] for row in parents]
        for row in parents:
            if len(row) > B.LORA_TREE_MAX_NODES or any(not -1 <= p < i for i, p in enumerate(row)):
                B._refuse(f"parents {row[:8]}...: each is -1 or the number of an earlier node, {B.LORA_TREE_MAX_NODES} nodes at most")
        seqs, nodes, t = self._new(hidden, seqs, [len(row) for row in parents], token_adapter)
        if t == 0:
            self.kv.extend(seqs, nodes)
            return torch.empty_like(hidden)
        lens, starts, seq, pos, ranges = self._places(seqs, nodes)
        plan = B.lora_kv_attn_plan(starts, seqs, lens, self.q_heads, self.kv_heads, self.head_dim, tree=True).to(self.device)
        tree = B.Tree(t, max(nodes), self.device)
        dev_starts, dev_parents = self._ints(starts), self._ints(np.concatenate([np.asarray(row, np.int32) for row in parents]))

        def attend(q, out):
            B.lora_tree_mask(dev_starts, dev_parents, tree)
            B.lora_kv_attn_tree(self.kv.view, plan, tree, q, out)
        with self._grown(seqs, nodes):
            y = self._run(hidden, seq, pos, token_adapter, ranges, attend)
        self._drafts.update({s: (n - len(row), row) for s, row, n in zip(seqs, parents, lens) if row})
        return y

    def accept(self, seqs, paths):
        """Ends the drafts of some sequences: each keeps the nodes paths[r] (none, or one below the context and then each
        time a successor of the node before) and drops the others.  Nothing may have changed a sequence since its draft, nor
        another hold pages that the draft grew into (a fork of it).  A call that is refused leaves the cache as it is."""
        seqs, paths = [int(s) for s in seqs], [[int(n) for n in p] for p in paths]
        if len(seqs) != len(paths) or len(set(seqs)) != len(seqs):
            B._refuse(f"{len(seqs)} sequences and {len(paths)} paths, or a sequence twice")
        with B._On(self.device, None):
            B._not_capturing("a path cannot be accepted")
        page_tokens, bases, own = self.kv.view.desc.page_tokens, [], []
        for s, path in zip(seqs, paths):
            base, parents = self._drafts.get(s, (0, []))
            if not parents or self.kv.length(s) != base + len(parents):
                B._refuse(f"sequence {s} has no draft, or has changed since")
            if any(not 0 <= n < len(parents) or parents[n] != up for up, n in zip([-1] + path, path)):
                B._refuse(f"{path[:8]} is no path from the context of a tree of {len(parents)} nodes")
            bases.append(base)
            own += self.kv.pages(s)[base // page_tokens:].tolist()
        if self.kv.stats()["shared"]:
            held = np.concatenate([self.kv.pages(s) for s in range(self.kv.view.num_seqs)])
            if (np.bincount(held, minlength=self.kv.view.desc.num_pages)[own] > 1).any():
                B._refuse("another sequence holds pages of a draft")
        rows = np.full((len(seqs), max([len(p) for p in paths] + [1])), -1, np.int32)
        for r, path in enumerate(paths):
            rows[r, :len(path)] = path
        # the page that a draft began on may hold bounds of nodes that are gone; one that ends where it began holds none, and
        # may be another sequence's too
        ranges = self._ranges(seqs, [b - 1 if b % page_tokens else b for b in bases], [b + len(p) for b, p in zip(bases, paths)])
        with B._On(self.device, None):
            B.lora_kv_keep_path(self.kv.view, self._ints(seqs), self._ints(bases), self._ints(rows))
            for s, base, path in zip(seqs, bases, paths):
                self.kv.truncate(s, base + len(path))
                del self._drafts[s]
            self._bounds(ranges)

    def _ranges(self, seqs, begins, ends):
        """Positions whose pages' bounds have to be written, on the device (a sequence with none has no range); None without
        bounds.  Refuses what lora_kv_bounds_update would, so that it can be asked before anything changes."""
        if self.kv.bounds is None or not seqs:
            return None
        # The call has workgroups for as many pages of every range as the longest one holds: ranges are cut at page borders to
        # a mean one's pages, so that a prompt beside many single tokens takes as many as there are pages, about.
        d = self.kv.view.desc
        page = d.page_tokens
        held = [-(-e // page) - b // page if b < e else 0 for b, e in zip(begins, ends)]
        most = max(1, -(-sum(held) // len(held)))
        cut = [(s, max(b, j * page), min(e, (j + most) * page)) for s, b, e, n in zip(seqs, begins, ends, held)
               for j in range(b // page, b // page + n, most)]
        longest = max([e - b for _, b, e in cut] + [0])
        pages = min((longest + page - 2) // page + 1, d.max_pages)
        if pages * d.kv_heads * len(cut) >= 1 << 24:
            raise B.LoraError(B.LORA_EUNSUPPORTED, f"bounds of {len(cut)} ranges of up to {pages} pages, {d.kv_heads} heads each")
        return (*(self._ints([r[i] for r in cut]) for i in range(3)), longest)

    def _bounds(self, ranges):
        if ranges is not None:
            B.lora_kv_bounds_update(self.kv.view, self.kv.bounds, *ranges)

    def run(self, hidden, plan, token_seq, token_pos, token_adapter, ranges=None, attend=None):
        """The device work of a step, launches only (every buffer is new; the plan and indices may serve many layers).
        Rows behind the plan's tokens are padding (token_seq -1, token_adapter -1): what stands in their y is unspecified.
        ranges: of a cache with bounds, (seq, begin, end, most positions) for lora_kv_bounds_update.  attend(q, out): the
        attention, where it is another than lora_kv_attn with the plan."""
        return self._run(hidden, token_seq, token_pos, token_adapter, ranges,
                         attend or (lambda q, out: B.lora_kv_attn(self.kv.view, plan, q, out)))

    def _run(self, hidden, token_seq, token_pos, token_adapter, ranges, attend):
        torch = _torch()
        t = self._rows(token_adapter, ("hidden", hidden, self.d_model))
        new = lambda n: torch.empty((t, n), dtype=torch.bfloat16, device=self.device)
        heads = lambda y, h: y.view(t, h, self.head_dim)
        with B._On(self.device, None):
            q, k, v = (new(self.widths[n][1]) for n in "qkv")
            for name, y in (("q", q), ("k", k), ("v", v)):
                self._project(name, hidden, y, token_adapter)
            B.lora_kv_append(self.kv.view, heads(k, self.kv_heads), heads(v, self.kv_heads), token_seq, token_pos)
            self._bounds(ranges)
            out = new(self.q_heads * self.head_dim)
            attend(heads(q, self.q_heads), heads(out, self.q_heads))
            y = new(self.d_model)
            self._project("o", out, y, token_adapter)
        return y
