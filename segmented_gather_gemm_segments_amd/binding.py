"""Thin ctypes binding over ``liblora_sgmv.so`` -- argument marshalling only.

Functions carry the C names of ``include/lora_sgmv.h``.  Every step of the
delta path runs in the library's kernels; PyTorch supplies device memory and
the current HIP stream.  The library must have been built
(``python -m segmented_gather_gemm_segments_amd.build``); if it is missing this
module raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import math
import os
import sys
from dataclasses import dataclass
from typing import Optional

import numpy as np

from . import build as _build

LORA_OK, LORA_EINVAL, LORA_ERANGE, LORA_EUNSUPPORTED, LORA_ENOMEM, LORA_EHIP = 0, -1, -2, -3, -4, -5
LORA_F32, LORA_BF16, LORA_FP8_E4M3 = 0, 1, 2
LORA_WFMT_PLAIN, LORA_WFMT_FP8_E4M3, LORA_WFMT_INT4 = 0, 1, 2
LORA_CACHE_HOST_ONLY = 1
LORA_NO_ADAPTER = -1
LORA_MAX_RANK = 128
LORA_PHASE_SHRINK, LORA_PHASE_EXPAND = 0, 1
LORA_PATH_AUTO, LORA_PATH_GATHER, LORA_PATH_MFMA = 0, 1, 2
LORA_BGMV_AUTO, LORA_BGMV_TOKEN_MAJOR, LORA_BGMV_ADAPTER_MAJOR = 0, 1, 2
LORA_DEFAULT_MFMA_MIN_TOKENS = 16
LORA_SHRINK_GATHER_TOKENS, LORA_SHRINK_GATHER_ROWS, LORA_SHRINK_MFMA_TOKENS = 4, 4, 16
LORA_EXPAND_GATHER_TOKENS, LORA_EXPAND_MFMA_TOKENS = 4, 128
LORA_EXPAND_LONG_TILE_MIN_ITEMS = 256
LORA_EXPAND_GATHER_COLS, LORA_EXPAND_MFMA_COLS = 2048, 256
LORA_PATH_TILE = 3
LORA_SHRINK_TILE_TOKENS, LORA_SHRINK_TILE_K, LORA_SHRINK_TILE_ITEM_BYTES = 64, 64, 262144
LORA_DEFAULT_TILE_MIN_TOKENS, LORA_TILE_MIN_RANK_SHORT, LORA_MAX_K_SPLITS = 16, 32, 64
LORA_TILE_PAYS_BYTES = 24 << 20
LORA_ATTN_ROWS, LORA_ATTN_TILE_ROWS, LORA_ATTN_MAX_PARTS, LORA_ATTN_CAUSAL = 16, 128, 64, 1
LORA_ATTN_TREE, LORA_ATTN_BLOCKS = 8, 16
LORA_KV_HOST_ONLY, LORA_KV_FP8, LORA_KV_BOUNDS = 1, 4, 8
LORA_TREE_MAX_NODES, LORA_BLOCKS_MAX_PAGES, LORA_BLOCKS_MAX_COUNT = 4096, 32768, 4096


class LoraError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_name(status)}: {message}")
        self.status = status


class lora_item(ctypes.Structure):
    _fields_ = [("perm_begin", ctypes.c_int32), ("adapter", ctypes.c_int32),
                ("count_path", ctypes.c_int32), ("block", ctypes.c_int32)]


class lora_weights(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32),
                ("num_adapters", ctypes.c_int32), ("r_max", ctypes.c_int32),
                ("page_rows", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages_a", ctypes.c_int32), ("num_pages_b", ctypes.c_int32),
                ("weight_format", ctypes.c_int32),
                ("a_pages", ctypes.c_void_p), ("b_pages", ctypes.c_void_p),
                ("rank", ctypes.c_void_p), ("a_page_table", ctypes.c_void_p),
                ("b_page_table", ctypes.c_void_p), ("host_rank", ctypes.c_void_p),
                ("a_scales", ctypes.c_void_p), ("b_scales", ctypes.c_void_p)]


class lora_cache_stats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_int64), ("misses", ctypes.c_int64),
                ("evictions", ctypes.c_int64), ("bytes_uploaded", ctypes.c_int64),
                ("resident", ctypes.c_int32), ("scattered", ctypes.c_int32),
                ("free_pages_a", ctypes.c_int32), ("free_pages_b", ctypes.c_int32)]


class lora_w4_weights(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("k", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p)]


class lora_kv_view(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("dtype", "head_dim", "kv_heads", "page_tokens", "num_pages",
                                              "num_seqs", "max_pages", "reserved")] + \
               [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p)]


class lora_kv8_view(ctypes.Structure):
    _fields_ = [("kv", lora_kv_view), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("scale_token_stride", ctypes.c_int64)]


class lora_tree(ctypes.Structure):
    _fields_ = [("mask", ctypes.c_void_p), ("depth", ctypes.c_void_p), ("words", ctypes.c_int32),
                ("num_tokens", ctypes.c_int32)]


class lora_kv_bounds(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class lora_attn_plan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("q_heads", "kv_heads", "head_dim", "flags", "window", "num_tokens",
                                              "num_row_items", "num_tile_items", "num_joins", "num_part_rows")] + \
               [("workspace_bytes", ctypes.c_int64)]


class lora_kv_stats(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("seqs", "pages", "shared", "spare", "highest", "page_tokens")]


_lib = None
_P, _I32, _I64, _U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64

EXPORTS = {
    "lora_abi_version": ([], _I32),
    "lora_last_error": ([], ctypes.c_char_p),
    "lora_status_name": ([_I32], ctypes.c_char_p),
    "lora_segments_build": ([_P, _I32, _I32, _P, _P, _P, _P], _I32),
    "lora_sgmv_plan": ([_I32, _P, _P, _I32, _I32, _P, _I32, _I32, _I32, _P, _I32, _P], _I32),
    "lora_sgmv_plan_tile": ([_I32, _P, _P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _P, _I32, _P], _I32),
    "lora_sgmv_shrink": ([_P, _P, _I32, _P, _I32, _I32, _P, _P, _P], _I32),
    "lora_sgmv_expand": ([_P, _P, _I32, _P, _I32, _I32, _P, _P, _P], _I32),
    "lora_sgmv_plan_tiled": ([_P, _P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I32, _P, _I32, _P, _P],
                             _I32),
    "lora_sgmv_shrink_tiled_workspace": ([_I32, _I32, _I32, ctypes.POINTER(ctypes.c_int64)], _I32),
    "lora_sgmv_tiled_pays": ([_P, _P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I32, _P], _I32),
    "lora_sgmv_shrink_tiled": ([_P, _P, _I32, _P, _I32, _I32, _I32, _P, _P, _P, ctypes.c_int64, _P], _I32),
    "lora_bgmv_shrink": ([_P, _P, _I32, _I32, _P, _P, _P], _I32),
    "lora_bgmv_expand": ([_P, _P, _I32, _I32, _P, _P, _P], _I32),
    "lora_bgmv_fused": ([_P, _P, _I32, _P, _I32, _I32, _P, _P, _P, _P], _I32),
    "lora_bgmv_fused_multi": ([_P, _I32, _P, _I32, _P, _I32, _P, _P, _P, _P], _I32),
    "lora_pool_create": ([_I32, _I32, _I32, _I32, _I32, _P, _P, _U64, _P], _I32),
    "lora_pool_alloc": ([_P, _I32, _P], _I32),
    "lora_pool_free": ([_P, _P, _I32], _I32),
    "lora_pool_num_free": ([_P, _P], _I32),
    "lora_pool_write_rows": ([_P, _P, _I32, _P, _P, _P], _I32),
    "lora_pool_destroy": ([_P], None),
    "lora_pool_info": ([_P, _P, _P, _P, _P, _P], _I32),
    "lora_cache_create": ([_P, _P, _I32, _I32, _P, _P, _P, _I32, _P], _I32),
    "lora_cache_register": ([_P, _I32, _I32, _P, _P, _P, _P], _I32),
    "lora_cache_prepare": ([_P, _P, _I32, _P], _I32),
    "lora_cache_get_stats": ([_P, _P], _I32),
    "lora_cache_pages": ([_P, _I32, _P, _P, _P], _I32),
    "lora_cache_destroy": ([_P], None),
    "lora_base_gemm": ([_I32, _I32, _I32, _I32, _P, _P, _P, _P, ctypes.c_int64, _P], _I32),
    "lora_base_gemm_workspace": ([_I32, _I32, _I32, ctypes.POINTER(ctypes.c_int64)], _I32),
    "lora_base_gemm_noalloc": ([_I32, _I32, _I32, _I32, _P, _P, _P, _P], _I32),
    "lora_probe_stream_read": ([_P, ctypes.c_int64, _I32, _I32, _I32, _P, _P], _I32),
    "lora_probe_release": ([_I32, _I32, _P, _P, _P, _P], _I32),
    "lora_debug_flags": ([_P, _I32], _I32),
    "lora_w4_bytes": ([_I32, _I32, ctypes.POINTER(_I64)], _I32),
    "lora_w4_pack": ([_I32, _I32, _I32, _P, _P, _P], _I32),
    "lora_base_w4": ([_I32, _I32, _P, _P, _I64, _P, _I64, _P], _I32),
    "lora_pages_copy": ([_P, _I64, _I32, _P, _P, _I32, _P], _I32),
    "lora_page_table_remap": ([_P, _I32, _P, _P, _I64, _P], _I32),
    "lora_kv_append": ([_P, _P, _P, _I64, _I64, _P, _P, _I32, _P], _I32),
    "lora_kv_read": ([_P, _P, _P, _I64, _I64, _P, _P, _I32, _P], _I32),
    "lora_kv_attn_plan": ([_P, _P, _P, _I32, _I32, _I64, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P, _I32], _I32),
    "lora_kv_attn": ([_P, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _P, ctypes.c_float, _P, _I64, _P], _I32),
    "lora_tree_mask": ([_P, _I32, _P, _I32, _P, _P], _I32),
    "lora_kv_attn_tree": ([_P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _P, ctypes.c_float, _P, _I64, _P], _I32),
    "lora_kv_keep_path": ([_P, _P, _P, _P, _I32, _I32, _P], _I32),
    "lora_kv_bounds_row_bytes": ([_I32, _P], _I32),
    "lora_kv_bounds_update": ([_P, _P, _P, _P, _P, _I32, _I32, _P], _I32),
    "lora_kv_block_select": ([_P, _P, _P, _P, _I32, _P, _I64, _I64, _I32, _I32, _I32, _I32, _P, _P, _I64, _P], _I32),
    "lora_kv_block_select_workspace": ([_P, _I32, _P], _I32),
    "lora_kv_attn_blocks": ([_P, _P, _P, _P, _I32, _P, _P, _I64, _I64, _P, _I64, _I64, _P, ctypes.c_float, _P, _I64, _P],
                            _I32),
    "lora_kv_create": ([_P, _I32, _I32, _I32, _I32, _P, _I32, _P], _I32),
    "lora_kv_extend": ([_P, _P, _P, _I32, _P], _I32),
    "lora_kv_fork": ([_P, _I32, _P, _I32, _P], _I32),
    "lora_kv_truncate": ([_P, _I32, _I32, _P], _I32),
    "lora_kv_free": ([_P, _P, _I32, _P], _I32),
    "lora_kv_compact": ([_P, _P, _P], _I32),
    "lora_kv_trim": ([_P, _I32, _P], _I32),
    "lora_kv_seq": ([_P, _I32, _P, _P, _P], _I32),
    "lora_kv_get_stats": ([_P, _P], _I32),
    "lora_kv_get_view": ([_P, _P], _I32),
    "lora_kv_get_view8": ([_P, _P], _I32),
    "lora_kv_get_bounds": ([_P, _P], _I32),
    "lora_kv_destroy": ([_P], None),
    "lora_kv_debug_flags": ([_P, _I32], _I32),
}
LORA_DEBUG_BAD_PAGE, LORA_DEBUG_BAD_ADAPTER, LORA_DEBUG_BAD_RANK = 1, 2, 4
LORA_DEBUG_BAD_TOKEN, LORA_DEBUG_BAD_ITEM = 8, 16


_debug = False
_loaded = {}


def lib_path() -> str:
    return _build.DEBUG_LIB if _debug else _build.LIB


def select_library(debug: bool) -> None:
    """Route every call of this module to the debug build of the library
    (kernels record bad device-side values, read by lora_debug_flags) or back
    to the release build."""
    global _debug, _lib
    _debug = bool(debug)
    _lib = None


def lib():
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = lib_path()
        if path not in _loaded:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m segmented_gather_gemm_segments_amd.build`")
            h = ctypes.CDLL(path)
            for name, (args, res) in EXPORTS.items():
                f = getattr(h, name)
                f.argtypes = args
                f.restype = res
            _loaded[path] = h
        _lib = _loaded[path]
    return _lib


def lora_debug_flags(clear: bool = False) -> int:
    """The debug build's error word (LORA_DEBUG_* bits); waits for the device."""
    out = ctypes.c_uint32(0)
    _check(lib().lora_debug_flags(ctypes.byref(out), int(clear)))
    return int(out.value)


def lora_kv_debug_flags(clear: bool = False) -> int:
    """The debug build's error word of the paged KV cache's kernels; waits for the device."""
    out = ctypes.c_uint32(0)
    _check(lib().lora_kv_debug_flags(ctypes.byref(out), int(clear)))
    return int(out.value)


def status_name(status: int) -> str:
    return lib().lora_status_name(status).decode()


def lora_last_error() -> str:
    return lib().lora_last_error().decode()


def _check(status: int):
    if status != LORA_OK:
        raise LoraError(status, lora_last_error())


def _np_ptr(a: Optional[np.ndarray]):
    return None if a is None else ctypes.c_void_p(a.ctypes.data)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


# ---------------------------------------------------------------- host calls
def lora_segments_build(token_adapter, num_adapters: int):
    """Host segment build.  Returns (token_perm, seg_starts, seg_adapter)."""
    ids = _i32(token_adapter)
    t = ids.size
    perm = np.empty(max(t, 1), np.int32)
    starts = np.empty(t + 1, np.int32)
    adapters = np.empty(max(t, 1), np.int32)
    s = ctypes.c_int32(0)
    _check(lib().lora_segments_build(_np_ptr(ids), t, num_adapters, _np_ptr(perm), _np_ptr(starts),
                                     _np_ptr(adapters), ctypes.byref(s)))
    s = s.value
    return perm[: starts[s]].copy(), starts[: s + 1].copy(), adapters[:s].copy()


def lora_sgmv_plan(phase: int, seg_starts, seg_adapter, num_adapters: int, dim: int,
                   path_policy: int = LORA_PATH_AUTO,
                   mfma_min_tokens: int = LORA_DEFAULT_MFMA_MIN_TOKENS,
                   host_rank=None, expand_tile_tokens: int = 0) -> np.ndarray:
    """Work plan as an int32 array [num_items, 4] (perm_begin, adapter, count|path<<16, block).
    dim: r_max for a shrink plan, d_out for an expand plan.  expand_tile_tokens:
    0 = the library's width table (lora_sgmv_plan), 64 or 128 = that MFMA
    expand tile (lora_sgmv_plan_tile)."""
    starts, adapters = _i32(seg_starts), _i32(seg_adapter)
    ranks = None if host_rank is None else _i32(host_rank)
    s = adapters.size
    n = ctypes.c_int32(0)
    head = (phase, _np_ptr(starts), _np_ptr(adapters), s, num_adapters, _np_ptr(ranks), dim, path_policy,
            mfma_min_tokens)
    if expand_tile_tokens:
        call = lambda *tail: lib().lora_sgmv_plan_tile(*head, int(expand_tile_tokens), *tail)
    else:
        call = lambda *tail: lib().lora_sgmv_plan(*head, *tail)
    _check(call(None, 0, ctypes.byref(n)))
    items = np.zeros((max(n.value, 1), 4), np.int32)
    _check(call(_np_ptr(items), n.value, ctypes.byref(n)))
    return items[: n.value]


def lora_sgmv_plan_tiled(seg_starts, seg_adapter, num_adapters: int, r_max: int, d_in: int,
                         path_policy: int = LORA_PATH_AUTO, tile_min_tokens: int = 0,
                         max_splits: int = 0, host_rank=None):
    """Tiled shrink plan: (int32 items [num_items, 4], k_splits)."""
    starts, adapters = _i32(seg_starts), _i32(seg_adapter)
    ranks = None if host_rank is None else _i32(host_rank)
    n, ks = ctypes.c_int32(0), ctypes.c_int32(0)
    args = (_np_ptr(starts), _np_ptr(adapters), adapters.size, num_adapters, _np_ptr(ranks), r_max, d_in,
            path_policy, tile_min_tokens, max_splits)
    _check(lib().lora_sgmv_plan_tiled(*args, None, 0, ctypes.byref(n), ctypes.byref(ks)))
    items = np.zeros((max(n.value, 1), 4), np.int32)
    _check(lib().lora_sgmv_plan_tiled(*args, _np_ptr(items), n.value, ctypes.byref(n), ctypes.byref(ks)))
    return items[: n.value], int(ks.value)


def lora_sgmv_tiled_pays(seg_starts, seg_adapter, num_adapters: int, r_max: int, d_in: int, dtype: int,
                         weight_format: int = LORA_WFMT_PLAIN, tile_min_tokens: int = 0, host_rank=None) -> bool:
    """Whether the library prefers the tiled shrink for this batch."""
    starts, adapters = _i32(seg_starts), _i32(seg_adapter)
    ranks = None if host_rank is None else _i32(host_rank)
    out = ctypes.c_int32(0)
    _check(lib().lora_sgmv_tiled_pays(_np_ptr(starts), _np_ptr(adapters), adapters.size, num_adapters,
                                      _np_ptr(ranks), r_max, d_in, dtype, weight_format, tile_min_tokens,
                                      ctypes.byref(out)))
    return bool(out.value)


def lora_sgmv_shrink_tiled_workspace(num_perm: int, r_max: int, k_splits: int) -> int:
    out = ctypes.c_int64(0)
    _check(lib().lora_sgmv_shrink_tiled_workspace(num_perm, r_max, k_splits, ctypes.byref(out)))
    return int(out.value)


# ---------------------------------------------------------------- device helpers
def _torch():
    import torch
    return torch


def _dptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


@dataclass
class Weights:
    """Device-resident adapter weights plus the lora_weights descriptor.

    ``a_pages`` [num_pages_a, page_rows, ...] and ``b_pages`` [num_pages_b,
    page_rows, ...] are torch tensors: bf16 or fp32 rows of d_in / d_out
    elements, or, for a quantized ``weight_format``, uint8 rows of the stored
    codes with fp32 row scales ``a_scales`` [num_pages_a * page_rows] and
    ``b_scales``; ``rank`` int32 [N] on device; page tables int32 [N,
    max_pages] on device or None (dense stack: page a = adapter a)."""
    dtype: int
    d_in: int
    d_out: int
    r_max: int
    page_rows: int
    a_pages: object
    b_pages: object
    rank: object
    host_rank: np.ndarray
    a_page_table: object = None
    b_page_table: object = None
    max_pages: int = 1
    weight_format: int = LORA_WFMT_PLAIN
    a_scales: object = None
    b_scales: object = None

    @property
    def num_adapters(self) -> int:
        return int(self.host_rank.size)

    def desc(self) -> lora_weights:
        self._host_rank_c = _i32(self.host_rank)
        hr = self._host_rank_c.ctypes.data if getattr(self, "host_rank_valid", True) else None
        return lora_weights(
            self.dtype, self.d_in, self.d_out, self.num_adapters, self.r_max, self.page_rows,
            self.max_pages, int(self.a_pages.shape[0]), int(self.b_pages.shape[0]),
            self.weight_format, _dptr(self.a_pages), _dptr(self.b_pages), _dptr(self.rank),
            _dptr(self.a_page_table), _dptr(self.b_page_table), hr,
            _dptr(self.a_scales), _dptr(self.b_scales))


def lora_sgmv_shrink(w: Weights, token_perm, items, x, v, num_tokens: Optional[int] = None,
                     stream=None):
    d = w.desc()
    n_tok = x.shape[0] if num_tokens is None else num_tokens
    _check(lib().lora_sgmv_shrink(ctypes.byref(d), _dptr(token_perm), int(token_perm.numel()),
                                  _dptr(items), int(items.shape[0]), n_tok, _dptr(x), _dptr(v),
                                  _stream(stream)))


def lora_sgmv_expand(w: Weights, token_perm, items, v, y, num_tokens: Optional[int] = None,
                     stream=None):
    d = w.desc()
    n_tok = y.shape[0] if num_tokens is None else num_tokens
    _check(lib().lora_sgmv_expand(ctypes.byref(d), _dptr(token_perm), int(token_perm.numel()),
                                  _dptr(items), int(items.shape[0]), n_tok, _dptr(v), _dptr(y),
                                  _stream(stream)))


def _ws_args(workspace):
    return (_dptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())


def lora_sgmv_shrink_tiled(w: Weights, token_perm, items, k_splits: int, x, v, workspace=None,
                           num_tokens: Optional[int] = None, stream=None):
    d = w.desc()
    n = int(x.shape[0]) if num_tokens is None else num_tokens
    wp, wb = _ws_args(workspace)
    _check(lib().lora_sgmv_shrink_tiled(ctypes.byref(d), _dptr(token_perm), int(token_perm.numel()),
                                        _dptr(items), int(items.shape[0]), n, int(k_splits), _dptr(x),
                                        _dptr(v), wp, wb, _stream(stream)))


def lora_bgmv_shrink(w: Weights, token_adapter, x, v, order: int = LORA_BGMV_AUTO, stream=None):
    d = w.desc()
    _check(lib().lora_bgmv_shrink(ctypes.byref(d), _dptr(token_adapter), int(token_adapter.numel()),
                                  order, _dptr(x), _dptr(v), _stream(stream)))


def lora_bgmv_expand(w: Weights, token_adapter, v, y, order: int = LORA_BGMV_AUTO, stream=None):
    d = w.desc()
    _check(lib().lora_bgmv_expand(ctypes.byref(d), _dptr(token_adapter), int(token_adapter.numel()),
                                  order, _dptr(v), _dptr(y), _stream(stream)))


def lora_bgmv_fused(w: Weights, token_adapter, x, y, v=None, order: int = LORA_BGMV_AUTO,
                    stream=None, token_order=None):
    """token_order: optional device int32 placement order (e.g. the segment
    permutation of the batch)."""
    d = w.desc()
    n_ord = 0 if token_order is None else int(token_order.numel())
    _check(lib().lora_bgmv_fused(ctypes.byref(d), _dptr(token_adapter), int(token_adapter.numel()),
                                 _dptr(token_order), n_ord, order, _dptr(x), _dptr(v), _dptr(y),
                                 _stream(stream)))


def _multi_args(ws, ys, vs):
    descs = [w.desc() for w in ws]
    n = len(descs)
    warr = (ctypes.POINTER(lora_weights) * n)(*[ctypes.pointer(d) for d in descs])
    yarr = (ctypes.c_void_p * n)(*[_dptr(y) for y in ys])
    varr = None if vs is None else (ctypes.c_void_p * n)(*[_dptr(v) for v in vs])
    return descs, warr, yarr, varr


def lora_bgmv_fused_multi(ws, token_adapter, x, ys, vs=None, stream=None, token_order=None):
    """Fused per-token deltas of several projections sharing x, one launch."""
    descs, warr, yarr, varr = _multi_args(ws, ys, vs)
    n_ord = 0 if token_order is None else int(token_order.numel())
    _check(lib().lora_bgmv_fused_multi(warr, len(ws), _dptr(token_adapter), int(token_adapter.numel()),
                                       _dptr(token_order), n_ord, _dptr(x), varr, yarr,
                                       _stream(stream)))


def prepare_bgmv_fused_multi(ws, token_adapter, x, ys, vs=None, stream=None, token_order=None):
    descs, warr, yarr, varr = _multi_args(ws, ys, vs)
    n_ord = 0 if token_order is None else int(token_order.numel())
    keep = (descs, warr, yarr, varr, ws, token_adapter, x, ys, vs, token_order)
    return Prepared("lora_bgmv_fused_multi", (warr, len(ws), _dptr(token_adapter),
                                              int(token_adapter.numel()), _dptr(token_order), n_ord,
                                              _dptr(x), varr, yarr, _stream(stream)), keep)


def base_gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    """Workspace bytes with which lora_base_gemm splits k (0: no split)."""
    out = ctypes.c_int64(0)
    _check(lib().lora_base_gemm_workspace(m, n, k, ctypes.byref(out)))
    return int(out.value)


def base_gemm_workspace(m: int, n: int, k: int, device="cuda"):
    """A workspace tensor for lora_base_gemm on this shape, or None."""
    nbytes = base_gemm_workspace_bytes(m, n, k)
    if nbytes == 0:
        return None
    return _torch().empty((nbytes + 3) // 4, dtype=_torch().float32, device=device)


def _ws(workspace):
    return (_dptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())


def lora_base_gemm(x, w, y, workspace=None, stream=None):
    m, k = x.shape
    n = w.shape[0]
    wp, wb = _ws(workspace)
    _check(lib().lora_base_gemm(LORA_BF16, m, n, k, _dptr(x), _dptr(w), _dptr(y), wp, wb,
                                _stream(stream)))


def lora_base_gemm_noalloc(x, w, y, stream=None):
    """lora_base_gemm without a workspace argument: split-k partials go to the
    library's own device scratch (allocates nothing)."""
    m, k = x.shape
    n = w.shape[0]
    _check(lib().lora_base_gemm_noalloc(LORA_BF16, m, n, k, _dptr(x), _dptr(w), _dptr(y),
                                        _stream(stream)))


class Pool:
    """lora_pool over caller-owned device storage: a torch tensor [num_pages,
    page_rows, row_width] of bf16 or fp32, or for a quantized weight_format a
    uint8 tensor [num_pages, page_rows, row_bytes] with fp32 row scales
    ``scales`` [num_pages * page_rows]."""

    def __init__(self, storage, page_rows: int, shuffle_seed: int = 0,
                 weight_format: int = LORA_WFMT_PLAIN, scales=None):
        self.storage = storage
        self.scales = scales
        num_pages, pr, width = storage.shape
        assert pr == page_rows
        torch = _torch()
        if weight_format == LORA_WFMT_PLAIN:
            dtype = LORA_BF16 if storage.dtype == torch.bfloat16 else LORA_F32
        else:
            dtype = LORA_BF16
            width = width * 2 if weight_format == LORA_WFMT_INT4 else width
        self.page_rows = page_rows
        h = ctypes.c_void_p()
        _check(lib().lora_pool_create(num_pages, page_rows, width, dtype, weight_format,
                                      _dptr(storage), _dptr(scales), shuffle_seed,
                                      ctypes.byref(h)))
        self._h = h

    def alloc(self, rows: int) -> np.ndarray:
        ids = np.empty((rows + self.page_rows - 1) // self.page_rows, np.int32)
        _check(lib().lora_pool_alloc(self._h, rows, _np_ptr(ids)))
        return ids

    def free(self, page_ids):
        ids = _i32(page_ids)
        _check(lib().lora_pool_free(self._h, _np_ptr(ids), ids.size))

    def num_free(self) -> int:
        n = ctypes.c_int32(0)
        _check(lib().lora_pool_num_free(self._h, ctypes.byref(n)))
        return n.value

    def write_rows(self, page_ids, src, src_scales=None, stream=None):
        """src: torch tensor [rows, row] on device (or pinned host); src_scales
        fp32 [rows] for a quantized pool."""
        ids = _i32(page_ids)
        _check(lib().lora_pool_write_rows(self._h, _np_ptr(ids), int(src.shape[0]), _dptr(src),
                                          _dptr(src_scales), _stream(stream)))

    def close(self):
        """Destroys the pool, and before it every KvCache over it (which waits for the device, so that it is refused
        while the current stream is being captured)."""
        if self._h:
            boxes = self.__dict__.get("_kv_handles", [])
            if any(box[0] and box[1] is not None for box in boxes):
                _not_capturing("a pool with KV caches cannot be closed")
            for box in boxes:
                _kv_destroy(box)
            lib().lora_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            _close_later(self)
        except Exception:  # at the interpreter's end the module's names may be gone
            pass


class Cache:
    """lora_cache: LRU residency of adapters (ids 0..num_ids-1) in two pools,
    owning the device page tables and ranks (torch int32 tensors it is given,
    or none in host-only mode).  ``weights(dtype, d_in, d_out)`` is the
    descriptor the kernels read through it."""

    def __init__(self, pool_a: Pool, pool_b: Pool, num_ids: int, r_max: int, page_table_a=None,
                 page_table_b=None, rank=None, host_only: bool = False):
        self.pool_a, self.pool_b = pool_a, pool_b
        self.num_ids, self.r_max = num_ids, r_max
        self.page_rows = pool_a.page_rows
        self.max_pages = (r_max + self.page_rows - 1) // self.page_rows
        self.pt_a, self.pt_b, self.rank = page_table_a, page_table_b, rank
        self._keep = {}
        h = ctypes.c_void_p()
        _check(lib().lora_cache_create(pool_a._h, pool_b._h, num_ids, r_max, _dptr(page_table_a),
                                       _dptr(page_table_b), _dptr(rank),
                                       LORA_CACHE_HOST_ONLY if host_only else 0, ctypes.byref(h)))
        self._h = h

    def register(self, id_: int, rank: int, rows_a, rows_b, scales_a=None, scales_b=None):
        """Host rows (numpy or torch CPU, ideally pinned) kept alive by the cache."""
        self._keep[id_] = (rows_a, rows_b, scales_a, scales_b)
        ptr = lambda t: None if t is None else (t.ctypes.data if isinstance(t, np.ndarray) else t.data_ptr())
        _check(lib().lora_cache_register(self._h, id_, rank, ptr(rows_a), ptr(rows_b), ptr(scales_a),
                                         ptr(scales_b)))

    def prepare(self, ids, stream=None, host_only: bool = False):
        a = _i32(ids)
        s = None if host_only else _stream(stream)
        _check(lib().lora_cache_prepare(self._h, _np_ptr(a), a.size, s))

    def stats(self) -> dict:
        st = lora_cache_stats()
        _check(lib().lora_cache_get_stats(self._h, ctypes.byref(st)))
        return {f: getattr(st, f) for f, _ in lora_cache_stats._fields_}

    def pages(self, id_: int):
        pa = np.empty(self.max_pages, np.int32)
        pb = np.empty(self.max_pages, np.int32)
        n = ctypes.c_int32(0)
        _check(lib().lora_cache_pages(self._h, id_, _np_ptr(pa), _np_ptr(pb), ctypes.byref(n)))
        return pa[: n.value].copy(), pb[: n.value].copy()

    def weights(self, dtype: int, d_in: int, d_out: int, weight_format: int = LORA_WFMT_PLAIN) -> "Weights":
        w = Weights(dtype, d_in, d_out, self.r_max, self.page_rows, self.pool_a.storage,
                    self.pool_b.storage, self.rank, np.ones(self.num_ids, np.int32), self.pt_a,
                    self.pt_b, self.max_pages, weight_format, self.pool_a.scales, self.pool_b.scales)
        w.host_rank_valid = False
        return w

    def close(self):
        if self._h:
            lib().lora_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def prepare_probe_stream_read(src, bytes_per_group: int, groups: int, threads: int, sink, stream=None,
                              nontemporal: bool = False):
    """Prepared bare streaming read (a measurement floor, not the delta path);
    nontemporal: loads with the non-temporal hint."""
    assert src.numel() * src.element_size() >= bytes_per_group * groups
    assert sink.numel() * sink.element_size() >= 4 * groups
    return Prepared("lora_probe_stream_read", (_dptr(src), int(bytes_per_group), int(groups), int(threads),
                                               int(bool(nontemporal)), _dptr(sink), _stream(stream)), (src, sink))


def prepare_probe_release(pairs: int, fence: bool, part, counters, out, stream=None):
    """Prepared release-per-workgroup probe (a measurement, not the delta path);
    counters must start at zero (every call leaves them zero)."""
    assert part.numel() * part.element_size() >= 2 * pairs * 64 * 4
    assert out.numel() * out.element_size() >= pairs * 64 * 4
    assert counters.numel() * counters.element_size() >= pairs * 4
    return Prepared("lora_probe_release", (int(pairs), int(bool(fence)), _dptr(part), _dptr(counters), _dptr(out),
                                           _stream(stream)), (part, counters, out))


# ---------------------------------------------------------------- prepared launches
class Prepared:
    """A device call with its ctypes arguments marshalled once; calling it only
    enqueues the launch (for launch-bound loops and graph capture).  Keeps the
    descriptor and every tensor it points to alive."""

    def __init__(self, fn_name: str, args: tuple, keep: tuple):
        self._fn = getattr(lib(), fn_name)
        self._args = args
        self._keep = keep

    def __call__(self):
        _check(self._fn(*self._args))


def prepare_bgmv(w: Weights, token_adapter, x, v, y, order: int = LORA_BGMV_AUTO, stream=None):
    """(shrink, expand) prepared BGMV launches on `stream` (default: current)."""
    d = w.desc()
    s = _stream(stream)
    n = int(token_adapter.numel())
    keep = (d, w, token_adapter, x, v, y)
    shrink = Prepared("lora_bgmv_shrink", (ctypes.byref(d), _dptr(token_adapter), n, order, _dptr(x),
                                           _dptr(v), s), keep)
    expand = Prepared("lora_bgmv_expand", (ctypes.byref(d), _dptr(token_adapter), n, order, _dptr(v),
                                           _dptr(y), s), keep)
    return shrink, expand


def prepare_sgmv(w: Weights, token_perm, shrink_items, expand_items, x, v, y, stream=None):
    """(shrink, expand) prepared SGMV launches on `stream` (default: current)."""
    d = w.desc()
    s = _stream(stream)
    keep = (d, w, token_perm, shrink_items, expand_items, x, v, y)
    npm = int(token_perm.numel())
    shrink = Prepared("lora_sgmv_shrink", (ctypes.byref(d), _dptr(token_perm), npm, _dptr(shrink_items),
                                           int(shrink_items.shape[0]), int(x.shape[0]), _dptr(x),
                                           _dptr(v), s), keep)
    expand = Prepared("lora_sgmv_expand", (ctypes.byref(d), _dptr(token_perm), npm, _dptr(expand_items),
                                           int(expand_items.shape[0]), int(y.shape[0]), _dptr(v),
                                           _dptr(y), s), keep)
    return shrink, expand


def prepare_sgmv_tiled(w: Weights, token_perm, tile_items, k_splits: int, workspace, expand_items, x, v, y,
                       stream=None):
    """(shrink, expand) prepared launches: the tiled shrink (with its reduce
    launch when k_splits > 1) and the segmented expand, on `stream`."""
    d = w.desc()
    s = _stream(stream)
    keep = (d, w, token_perm, tile_items, expand_items, x, v, y, workspace)
    npm = int(token_perm.numel())
    wp, wb = _ws_args(workspace)
    shrink = Prepared("lora_sgmv_shrink_tiled", (ctypes.byref(d), _dptr(token_perm), npm, _dptr(tile_items),
                                                 int(tile_items.shape[0]), int(x.shape[0]), int(k_splits),
                                                 _dptr(x), _dptr(v), wp, wb, s), keep)
    expand = Prepared("lora_sgmv_expand", (ctypes.byref(d), _dptr(token_perm), npm, _dptr(expand_items),
                                           int(expand_items.shape[0]), int(y.shape[0]), _dptr(v),
                                           _dptr(y), s), keep)
    return shrink, expand


def prepare_base_gemm(x, w, y, workspace=None, stream=None):
    """Prepared lora_base_gemm launch y = x w^T on `stream` (default: current)."""
    m, k = x.shape
    n = w.shape[0]
    wp, wb = _ws(workspace)
    return Prepared("lora_base_gemm", (LORA_BF16, m, n, k, _dptr(x), _dptr(w), _dptr(y), wp, wb,
                                       _stream(stream)), (x, w, y, workspace))


def prepare_bgmv_fused(w: Weights, token_adapter, x, y, v=None, order: int = LORA_BGMV_AUTO,
                       stream=None, token_order=None):
    """Prepared fused BGMV launch (shrink + expand in one kernel) on `stream`."""
    d = w.desc()
    keep = (d, w, token_adapter, x, v, y, token_order)
    n_ord = 0 if token_order is None else int(token_order.numel())
    return Prepared("lora_bgmv_fused", (ctypes.byref(d), _dptr(token_adapter),
                                        int(token_adapter.numel()), _dptr(token_order), n_ord,
                                        order, _dptr(x), _dptr(v), _dptr(y), _stream(stream)), keep)


# ---------------------------------------------------------------- 4-bit base projection, paged KV cache
# These calls take strides from their tensors, so they check what a bare address cannot say: the
# type, a contiguous last dimension, and that every tensor is on the device the call runs on.
def _refuse(message: str):
    raise LoraError(LORA_EINVAL, message)


def _tensors(device, *named):
    """Checks (name, tensor, dtype) triples; None tensors pass."""
    for name, t, dtype in named:
        if t is None:
            continue
        if t.dtype != dtype:
            _refuse(f"{name} is {t.dtype}, not {dtype}")
        if t.device != device:
            _refuse(f"{name} is on {t.device}, not {device}")
        if t.dim() and t.shape[-1] > 1 and t.stride(-1) != 1 and t.numel():
            _refuse(f"{name}'s last dimension is not contiguous")


def _flat(name, t):
    if not t.is_contiguous():
        _refuse(f"{name} is not contiguous")


class _On:
    """The device of a call made current (a launch goes to the current device), and its stream."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            _refuse(f"tensors must be on a GPU, not {device}")
        cuda = _torch().cuda
        self._guard = None if device.index == cuda.current_device() else cuda.device(device)
        self._device, self._arg = device, stream

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()
        s = _torch().cuda.current_stream(self._device) if self._arg is None else self._arg
        return ctypes.c_void_p(s.cuda_stream)

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)


def _launch(name: str, index: int, stream, *args):
    """Calls a device function on the current stream of device `index` (or `stream`); what these calls cost on the
    host is what a small one costs in all, so this is the short way to what _On does."""
    fn = getattr(_lib or lib(), name)
    torch = _torch()
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != LORA_OK:
        _check(status)


def _gpu(device) -> int:
    if device.type != "cuda":
        _refuse(f"tensors must be on a GPU, not {device}")
    return device.index


def lora_w4_bytes(n: int, k: int) -> int:
    out = ctypes.c_int64(0)
    _check(lib().lora_w4_bytes(n, k, ctypes.byref(out)))
    return int(out.value)


def lora_w4_pack(rows, twos_complement: bool = False, stream=None):
    """Tiled codes [ceil(n/16), ceil(k/128), 64, 16] of row-major ones: rows uint8 [n, k/2] on the
    device, element 2i in the low nibble.  The codes are memory of the stream that writes them."""
    torch = _torch()
    _tensors(rows.device, ("rows", rows, torch.uint8))
    _flat("rows", rows)
    n, k = int(rows.shape[0]), int(rows.shape[1]) * 2
    lora_w4_bytes(n, k)
    with _On(rows.device, stream) as s, torch.cuda.stream(stream):
        codes = torch.empty((-(-n // 16), -(-k // 128), 64, 16), dtype=torch.uint8, device=rows.device)
        _check(lib().lora_w4_pack(n, k, int(bool(twos_complement)), _dptr(rows), _dptr(codes), s))
    return codes


class W4Weights:
    """4-bit weights of an n x k projection and their lora_w4_weights descriptor: codes as
    lora_w4_pack gives them, scales and optional zeros [k / group, n] fp32 or bf16."""

    def __init__(self, n: int, k: int, group: int, codes, scales, zeros=None):
        torch = _torch()
        if scales.dtype not in (torch.float32, torch.bfloat16):
            _refuse(f"scales are {scales.dtype}, not float32 or bfloat16")
        _tensors(codes.device, ("codes", codes, torch.uint8), ("scales", scales, scales.dtype),
                 ("zeros", zeros, scales.dtype))
        for name, t in (("codes", codes), ("scales", scales), ("zeros", zeros)):
            if t is not None:
                _flat(name, t)
        if codes.numel() != lora_w4_bytes(n, k):
            _refuse(f"codes hold {codes.numel()} bytes, {n} x {k} needs {lora_w4_bytes(n, k)}")
        for name, t in (("scales", scales), ("zeros", zeros)):
            if t is not None and (group <= 0 or t.numel() != k // group * n):
                _refuse(f"{name} hold {t.numel()} values, not [{k} / {group}, {n}]")
        self.n, self.k, self.group = n, k, group
        self.codes, self.scales, self.zeros = codes, scales, zeros
        self.desc = lora_w4_weights(n, k, group, LORA_BF16 if scales.dtype == torch.bfloat16 else LORA_F32,
                                    _dptr(codes), _dptr(scales), _dptr(zeros))
        self.ref, self.index, self.bf16 = ctypes.byref(self.desc), codes.get_device(), torch.bfloat16
        self.one_x, self.one_y = k + -k % 8, n + -n % 8  # the row strides of a single row, whose own say nothing


def lora_base_w4(x, w: W4Weights, y, stream=None):
    """y [m, n] = x [m, k] W^T; x and y may be column blocks of wider arrays (row strides kept)."""
    index, bf16 = w.index, w.bf16
    m = x.shape[0]
    xs, ys = x.stride(), y.stride()
    if not (x.dtype is bf16 and y.dtype is bf16 and x.get_device() == index and y.get_device() == index and
            x.shape == (m, w.k) and y.shape == (m, w.n) and xs[1] == 1 and ys[1] == 1):
        _tensors(w.codes.device, ("x", x, bf16), ("y", y, bf16))
        if tuple(x.shape) != (m, w.k) or tuple(y.shape) != (m, w.n):
            _refuse(f"x {tuple(x.shape)} and y {tuple(y.shape)} for weights of {w.n} x {w.k}")
    if index < 0:
        _gpu(w.codes.device)
    _launch("lora_base_w4", index, stream, LORA_BF16, m, w.ref, x.data_ptr(), xs[0] if m > 1 else w.one_x,
            y.data_ptr(), ys[0] if m > 1 else w.one_y)


class KvView:
    """A paged KV cache as the kernels read it: k and v [num_pages, kv_heads, page_tokens, head_dim] tensors of the same
    strides (views of one storage, usually), page_table int32 [num_seqs, max_pages].  bf16, or of 8-bit rows:
    float8_e4m3fn with k_scales and v_scales, uint8 [num_pages, kv_heads, page_tokens], the rows' exponents plus 127."""

    def __init__(self, k, v, page_table, k_scales=None, v_scales=None):
        torch = _torch()
        dtype = torch.bfloat16 if k_scales is None and v_scales is None else torch.float8_e4m3fn
        _tensors(k.device, ("k", k, dtype), ("v", v, dtype), ("page_table", page_table, torch.int32))
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            _refuse(f"k {tuple(k.shape)} {k.stride()} and v {tuple(v.shape)} {v.stride()} differ or are not 4-d")
        if page_table.dim() != 2:
            _refuse("page_table is [num_seqs, max_pages]")
        _flat("page_table", page_table)
        self.k, self.v, self.page_table = k, v, page_table
        self.k_scales, self.v_scales = k_scales, v_scales
        pages, heads, tokens, dim = (int(n) for n in k.shape)
        strides = lambda t: (st if n > 1 else 0 for n, st in zip(t.shape[:3], t.stride()))
        fields = (dim, heads, tokens, pages, int(page_table.shape[0]), int(page_table.shape[1]), 0, _dptr(k), _dptr(v),
                  *strides(k), _dptr(page_table))
        if dtype is torch.bfloat16:
            self.desc = lora_kv_view(LORA_BF16, *fields)
            self.ref = ctypes.byref(self.desc)
        else:
            if k_scales is None or v_scales is None:
                _refuse("8-bit rows need the scales of both k and v")
            for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
                if t.dtype != torch.uint8 or t.device != k.device or t.shape != k.shape[:3]:
                    _refuse(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}: uint8 {tuple(k.shape[:3])} on {k.device} wanted")
            if k_scales.stride() != v_scales.stride():
                _refuse(f"k_scales and v_scales have strides {k_scales.stride()} and {v_scales.stride()}")
            self.desc8 = lora_kv8_view(lora_kv_view(LORA_FP8_E4M3, *fields), _dptr(k_scales), _dptr(v_scales), *strides(k_scales))
            self.desc, self.ref = self.desc8.kv, ctypes.byref(self.desc8)
        self.index, self.device = k.get_device(), k.device
        self.num_seqs, self.max_kv = self.desc.num_seqs, self.desc.max_pages * tokens
        self.bf16, self.int32, self.fp32 = torch.bfloat16, torch.int32, torch.float32


def lora_pages_copy(storage, src, dst, stream=None):
    """Copies page src[i] to page dst[i]; storage [num_pages, ...] contiguous, src and dst int32 on its device."""
    index, n = storage.get_device(), src.numel()
    i32 = _torch().int32
    if not (index >= 0 and src.dtype is i32 and dst.dtype is i32 and src.get_device() == index and
            dst.get_device() == index and dst.numel() == n and storage.is_contiguous() and src.is_contiguous() and
            dst.is_contiguous()):
        _gpu(storage.device)
        _tensors(storage.device, ("src", src, i32), ("dst", dst, i32))
        for name, t in (("storage", storage), ("src", src), ("dst", dst)):
            _flat(name, t)
        _refuse(f"{src.numel()} source and {dst.numel()} destination pages")
    pages = storage.shape[0]
    _launch("lora_pages_copy", index, stream, storage.data_ptr(), storage.nbytes // max(pages, 1), pages, src.data_ptr(),
            dst.data_ptr(), n)


def lora_page_table_remap(remap, table_in, table_out, stream=None):
    """table_out = remap[table_in], entries outside [0, len(remap)) kept; int32 on one device."""
    index, n = remap.get_device(), table_in.numel()
    i32 = _torch().int32
    if not (index >= 0 and remap.dtype is i32 and table_in.dtype is i32 and table_out.dtype is i32 and
            table_in.get_device() == index and table_out.get_device() == index and table_out.numel() == n and
            remap.is_contiguous() and table_in.is_contiguous() and table_out.is_contiguous()):
        _tensors(remap.device, ("remap", remap, i32), ("table_in", table_in, i32), ("table_out", table_out, i32))
        for name, t in (("remap", remap), ("table_in", table_in), ("table_out", table_out)):
            _flat(name, t)
        if table_in.numel() != table_out.numel():
            _refuse(f"tables of {table_in.numel()} and {table_out.numel()} entries")
        _gpu(remap.device)
    _launch("lora_page_table_remap", index, stream, remap.data_ptr(), remap.numel(), table_in.data_ptr(),
            table_out.data_ptr(), n)


def _row_strides(t):
    """Token and head strides of [T, heads, dim] (0 for a dimension of one: its stride says nothing)."""
    a, b, _ = t.stride()
    n, h, _ = t.shape
    return (a if n > 1 else 0, b if h > 1 else 0) if n else (0, 0)


def lora_kv_append(view: KvView, k_new, v_new, token_seq, token_pos, stream=None, *, _call="lora_kv_append",
                   _names=("k_new", "v_new")):
    """Writes k_new, v_new [T, kv_heads, head_dim] bf16 at positions token_pos [T] of sequences token_seq [T], quantised where
    the cache holds 8-bit rows."""
    d, index, bf16, i32 = view.desc, view.index, view.bf16, view.int32
    n = k_new.shape[0]
    shape = (n, d.kv_heads, d.head_dim)
    if not (k_new.dtype is bf16 and v_new.dtype is bf16 and token_seq.dtype is i32 and token_pos.dtype is i32 and
            k_new.get_device() == index and v_new.get_device() == index and token_seq.get_device() == index and
            token_pos.get_device() == index and k_new.shape == shape and v_new.shape == shape and
            token_seq.numel() == n and token_pos.numel() == n and token_seq.is_contiguous() and
            token_pos.is_contiguous() and (n == 0 or (k_new.stride(2) == 1 and v_new.stride(2) == 1))):
        _tensors(view.device, (_names[0], k_new, bf16), (_names[1], v_new, bf16), ("token_seq", token_seq, i32),
                 ("token_pos", token_pos, i32))
        if tuple(k_new.shape) != shape or tuple(v_new.shape) != shape or token_seq.numel() != n or token_pos.numel() != n:
            _refuse(f"{_names[0]} {tuple(k_new.shape)}, {_names[1]} {tuple(v_new.shape)}, {token_seq.numel()} sequences and "
                    f"{token_pos.numel()} positions: {shape} wanted")
        _flat("token_seq", token_seq)
        _flat("token_pos", token_pos)
    if index < 0:
        _gpu(view.device)
    ts, hs = _row_strides(k_new)
    if _row_strides(v_new) != (ts, hs):
        _refuse(f"{_names[0]} and {_names[1]} have strides {k_new.stride()} and {v_new.stride()}")
    _launch(_call, index, stream, view.ref, k_new.data_ptr(), v_new.data_ptr(), ts, hs, token_seq.data_ptr(), token_pos.data_ptr(), n)


def lora_kv_read(view: KvView, token_seq, token_pos, k_out, v_out, stream=None):
    """The rows of those positions in k_out, v_out [T, kv_heads, head_dim] bf16; rows of absent ones are left as they are."""
    lora_kv_append(view, k_out, v_out, token_seq, token_pos, stream, _call="lora_kv_read", _names=("k_out", "v_out"))


class AttnPlan:
    """A batch's attention plan: the host items, and after ``to(device)`` the device copy and workspace."""

    def __init__(self, desc: lora_attn_plan, items: np.ndarray):
        self.desc, self.host_items, self.ref = desc, items, ctypes.byref(desc)
        self.items = self.workspace = None
        # what the items reach: sequences below num_seqs, positions below max_kv
        self.num_seqs = int(items[:, 3].max()) + 1 if len(items) else 0
        self.max_kv = int(items[:, 6].max()) if len(items) else 0

    def to(self, device) -> "AttnPlan":
        """Uploads the items and allocates a workspace (calls that share the plan must not overlap).  Both stay where
        they are when they are on the device already: a captured graph may hold their addresses.  They are memory of the
        current stream: a call on another one comes behind it, and before the plan goes, as with any tensor."""
        torch = _torch()
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        if self.items is not None and self.items.device == device:
            return self
        self.items = torch.from_numpy(self.host_items).to(device)
        n = self.desc.workspace_bytes
        self.workspace = torch.empty(n // 4, dtype=torch.float32, device=device) if n else None
        return self


def lora_kv_attn_plan(q_starts, seqs, kv_lens, q_heads: int, kv_heads: int, head_dim: int, causal: bool = True,
                      window: int = 0, max_parts: int = 0, num_seqs: Optional[int] = None,
                      max_kv: int = 2**31 - 1, tree: bool = False, blocks: bool = False) -> AttnPlan:
    """Plan of a batch: request r has tokens q_starts[r] .. q_starts[r + 1] of q, sequence seqs[r] of kv_lens[r]
    positions.  num_seqs, max_kv: the bounds to check against (lora_kv_attn checks the view's).  tree: for
    lora_kv_attn_tree.  blocks: for lora_kv_attn_blocks, a request for each token, kv_lens of its list's pages (there is
    no other mask then, `causal` says nothing)."""
    starts, sq, kv = _i32(q_starts), _i32(seqs), _i32(kv_lens)
    if starts.size < 1 or sq.size != starts.size - 1 or kv.size != sq.size:
        _refuse(f"{starts.size} starts, {sq.size} sequences and {kv.size} lengths")
    plan = lora_attn_plan()
    args = (_np_ptr(starts), _np_ptr(sq), _np_ptr(kv), sq.size, 2**31 - 1 if num_seqs is None else num_seqs, max_kv,
            q_heads, kv_heads, head_dim,
            LORA_ATTN_BLOCKS | (LORA_ATTN_TREE if tree else 0) if blocks else
            (LORA_ATTN_CAUSAL if causal else 0) | (LORA_ATTN_TREE if tree else 0), window, max_parts, ctypes.byref(plan))
    _check(lib().lora_kv_attn_plan(*args, None, 0))
    n = plan.num_row_items + plan.num_tile_items + plan.num_joins
    items = np.zeros((max(n, 1), 8), np.int32)
    _check(lib().lora_kv_attn_plan(*args, _np_ptr(items), n))
    return AttnPlan(plan, items[:n])


def lora_kv_attn(view: KvView, plan: AttnPlan, q, out, lse=None, scale: Optional[float] = None, workspace=None,
                 stream=None, *, _call="lora_kv_attn", _mask=(), _max_kv=None):
    """out [T, q_heads, head_dim] (and lse [T, q_heads] fp32) of q over the cache; scale defaults to
    head_dim ** -0.5, workspace to the plan's own.  A plan that reaches past the view is refused (LORA_ERANGE); the debug
    library runs it, skips those items and records them."""
    items = plan.items
    if items is None:
        _refuse("the plan has not been uploaded: call plan.to(device)")
    max_kv = view.max_kv if _max_kv is None else _max_kv  # _mask: what another kind of mask has behind the items
    if (plan.num_seqs > view.num_seqs or plan.max_kv > max_kv) and not _debug:
        raise LoraError(LORA_ERANGE, f"the plan reaches {plan.num_seqs} sequences of up to {plan.max_kv} positions, the "
                                     f"view holds {view.num_seqs} of {max_kv}")
    p, index, bf16, fp32 = plan.desc, view.index, view.bf16, view.fp32
    ws = plan.workspace if workspace is None else workspace
    heads, dim, tokens = p.q_heads, p.head_dim, p.num_tokens
    t = q.shape[0]
    if not (q.dtype is bf16 and out.dtype is bf16 and q.get_device() == index and out.get_device() == index and
            items.get_device() == index and t >= tokens and q.shape == (t, heads, dim) and out.shape == q.shape and
            (t == 0 or (q.stride(2) == 1 and out.stride(2) == 1))):
        _tensors(view.device, ("q", q, bf16), ("out", out, bf16), ("the plan's items", items, view.int32))
        if q.dim() != 3 or q.shape != out.shape or tuple(q.shape[1:]) != (heads, dim) or t < tokens:
            _refuse(f"q {tuple(q.shape)} and out {tuple(out.shape)}: [{tokens} or more, {heads}, {dim}] wanted")
    lse_ptr = None
    if lse is not None:
        if not (lse.dtype is fp32 and lse.get_device() == index and lse.is_contiguous() and lse.dim() == 2 and
                lse.shape[0] >= tokens and lse.shape[1] == heads):
            _tensors(view.device, ("lse", lse, fp32))
            _flat("lse", lse)
            _refuse(f"lse {tuple(lse.shape)}: [{tokens} or more, {heads}] wanted")
        lse_ptr = lse.data_ptr()
    wp, wb = None, 0
    if ws is not None:
        if not ws.is_contiguous() or ws.get_device() != index:
            _flat("workspace", ws)
            _refuse(f"workspace is on {ws.device}, not {view.device}")
        wp, wb = ws.data_ptr(), ws.nbytes
    if index < 0:
        _gpu(view.device)
    qs, os_ = _row_strides(q), _row_strides(out)
    _launch(_call, index, stream, view.ref, plan.ref, items.data_ptr(), *_mask, q.data_ptr(), *qs, out.data_ptr(), *os_,
            lse_ptr, dim ** -0.5 if scale is None else scale, wp, wb)


class Tree:
    """What a tree's attention reads of the nodes of a batch: mask int64 [num_tokens, words], depth int32 [num_tokens].
    max_nodes: the most that a request has."""

    def __init__(self, num_tokens: int, max_nodes: int, device):
        torch = _torch()
        if not 0 <= max_nodes <= LORA_TREE_MAX_NODES:
            raise LoraError(LORA_EUNSUPPORTED, f"a tree of {max_nodes} nodes, not up to {LORA_TREE_MAX_NODES}")
        words = max(1, -(-max_nodes // 64))
        self.mask = torch.empty((num_tokens, words), dtype=torch.int64, device=device)
        self.depth = torch.empty(num_tokens, dtype=torch.int32, device=device)
        self.desc = lora_tree(_dptr(self.mask), _dptr(self.depth), words, num_tokens)
        self.ref, self.index, self.device = ctypes.byref(self.desc), self.mask.get_device(), self.mask.device


def _i32s(device, *named):
    """Checks (name, tensor) pairs: int32, contiguous, on the device."""
    i32 = _torch().int32
    for name, t in named:
        if t.dtype is not i32 or t.device != device or not t.is_contiguous():
            _tensors(device, (name, t, i32))
            _flat(name, t)


def lora_tree_mask(q_starts, parent, tree: Tree, window: int = 0, stream=None):
    """Masks and depths of a batch's trees: q_starts int32 [num_reqs + 1] and parent int32 [num_tokens] on the device (a
    parent's number within its request, -1 for the context)."""
    _i32s(tree.device, ("q_starts", q_starts), ("parent", parent))
    if q_starts.numel() < 1 or parent.numel() != tree.desc.num_tokens:
        _refuse(f"{q_starts.numel()} starts and {parent.numel()} parents for a tree of {tree.desc.num_tokens} tokens")
    if tree.index < 0:
        _gpu(tree.device)
    _launch("lora_tree_mask", tree.index, stream, q_starts.data_ptr(), q_starts.numel() - 1, parent.data_ptr(), window, tree.ref)


def lora_kv_attn_tree(view: KvView, plan: AttnPlan, tree: Tree, q, out, lse=None, scale: Optional[float] = None,
                      workspace=None, stream=None):
    """lora_kv_attn for nodes of trees, with a plan made with tree=True."""
    if tree.device != view.device:
        _refuse(f"the tree is on {tree.device}, not {view.device}")
    lora_kv_attn(view, plan, q, out, lse, scale, workspace, stream, _call="lora_kv_attn_tree", _mask=(tree.ref,))


def lora_kv_keep_path(view: KvView, seq, base, path, stream=None):
    """Moves the rows of accepted paths: path int32 [num_reqs, max_path] of ascending nodes, -1 behind the last, of trees
    whose node 0 stands at position base [num_reqs] of sequence seq [num_reqs]."""
    _i32s(view.device, ("seq", seq), ("base", base), ("path", path))
    n = seq.numel()
    if path.dim() != 2 or path.shape[0] != n or base.numel() != n:
        _refuse(f"{n} sequences, {base.numel()} positions and paths {tuple(path.shape)}")
    if view.index < 0:
        _gpu(view.device)
    _launch("lora_kv_keep_path", view.index, stream, view.ref, seq.data_ptr(), base.data_ptr(), path.data_ptr(), n, path.shape[1])


def lora_kv_bounds_row_bytes(head_dim: int) -> int:
    out = ctypes.c_int64(0)
    _check(lib().lora_kv_bounds_row_bytes(head_dim, ctypes.byref(out)))
    return int(out.value)


class KvBounds:
    """Bounds of the keys of a cache's pages: rows uint8 [num_pages, kv_heads, lora_kv_bounds_row_bytes(head_dim)]."""

    def __init__(self, view: KvView, rows):
        torch, d = _torch(), view.desc
        _tensors(view.device, ("rows", rows, torch.uint8))
        shape = (d.num_pages, d.kv_heads, lora_kv_bounds_row_bytes(d.head_dim))
        if tuple(rows.shape) != shape:
            _refuse(f"rows {tuple(rows.shape)}: {shape} wanted")
        ps, hs = (st if n > 1 else 0 for n, st in zip(rows.shape[:2], rows.stride()))
        self.rows, self.desc = rows, lora_kv_bounds(_dptr(rows), ps, hs)
        self.ref, self.index = ctypes.byref(self.desc), rows.get_device()
        self.pages, self.heads = d.num_pages, (d.kv_heads, d.head_dim)


def _bounds_of(view: KvView, bounds: KvBounds):
    """Checks that the bounds have a row for every page and head of this view, which need not be the one they were made with."""
    d = view.desc
    if bounds.index != view.index:
        _refuse(f"bounds are on {bounds.rows.device}, not {view.device}")
    if bounds.pages < d.num_pages or bounds.heads != (d.kv_heads, d.head_dim):
        _refuse(f"bounds of {bounds.pages} pages, {bounds.heads[0]} KV heads of {bounds.heads[1]}: the view has {d.num_pages}, "
                f"{d.kv_heads} of {d.head_dim}")


def lora_kv_bounds_update(view: KvView, bounds: KvBounds, seq, begin, end, max_tokens: int, stream=None):
    """Bounds of the pages that hold positions begin[r] .. end[r] of sequence seq[r] (int32 [n]); max_tokens: the most
    positions of a range."""
    _i32s(view.device, ("seq", seq), ("begin", begin), ("end", end))
    n = seq.numel()
    if begin.numel() != n or end.numel() != n:
        _refuse(f"{n} sequences, {begin.numel()} first and {end.numel()} last positions")
    _bounds_of(view, bounds)
    if view.index < 0:
        _gpu(view.device)
    _launch("lora_kv_bounds_update", view.index, stream, view.ref, bounds.ref, seq.data_ptr(), begin.data_ptr(), end.data_ptr(), n,
            max_tokens)


def lora_kv_block_select_workspace(view: KvView, num_tokens: int) -> int:
    """Bytes of workspace; refuses a view and a number of tokens that lora_kv_block_select would."""
    out = ctypes.c_int64(0)
    _check(lib().lora_kv_block_select_workspace(view.ref, num_tokens, ctypes.byref(out)))
    return int(out.value)


def lora_kv_block_select(view: KvView, bounds: KvBounds, token_seq, token_pos, q, blocks, sink: int = 1, recent: int = 1,
                         workspace=None, stream=None):
    """The pages that token t, at position token_pos[t] of sequence token_seq[t] (int32 [T]), attends to, for each KV
    head: blocks int32 [T, kv_heads, count], ascending, -1 behind the last.  q [T or more, q_heads, head_dim] bf16.
    workspace: None allocates what the call takes on its stream, where it takes any."""
    d, n = view.desc, token_seq.numel()
    _i32s(view.device, ("token_seq", token_seq), ("token_pos", token_pos), ("blocks", blocks))
    _tensors(view.device, ("q", q, view.bf16))
    if (token_pos.numel() != n or q.dim() != 3 or q.shape[0] < n or q.shape[2] != d.head_dim or blocks.dim() != 3 or
            blocks.shape[0] < n or blocks.shape[1] != d.kv_heads):
        _refuse(f"{n} sequences, {token_pos.numel()} positions, q {tuple(q.shape)} and blocks {tuple(blocks.shape)} for "
                f"{d.kv_heads} KV heads of {d.head_dim}")
    _bounds_of(view, bounds)
    if view.index < 0:
        _gpu(view.device)
    if workspace is None:
        need = lora_kv_block_select_workspace(view, n)
        if need:
            torch = _torch()
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=view.device)
    elif not workspace.is_contiguous() or workspace.device != view.device:
        _flat("workspace", workspace)
        _refuse(f"workspace is on {workspace.device}, not {view.device}")
    wp, wb = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _launch("lora_kv_block_select", view.index, stream, view.ref, bounds.ref, token_seq.data_ptr(), token_pos.data_ptr(), n,
            q.data_ptr(), *_row_strides(q), q.shape[1], blocks.shape[2], sink, recent, blocks.data_ptr(), wp, wb)


def lora_kv_attn_blocks(view: KvView, plan: AttnPlan, blocks, token_pos, q, out, lse=None, scale: Optional[float] = None,
                        workspace=None, stream=None):
    """lora_kv_attn over the pages that blocks [T, kv_heads, count] lists, up to token_pos [T], with a plan made with
    blocks=True."""
    d, n = view.desc, plan.desc.num_tokens
    _i32s(view.device, ("blocks", blocks), ("token_pos", token_pos))
    if blocks.dim() != 3 or blocks.shape[0] < n or blocks.shape[1] != d.kv_heads or token_pos.numel() < n:
        _refuse(f"blocks {tuple(blocks.shape)} and {token_pos.numel()} positions: [{n} or more, {d.kv_heads}, pages] wanted")
    count = blocks.shape[2]
    lora_kv_attn(view, plan, q, out, lse, scale, workspace, stream, _call="lora_kv_attn_blocks",
                 _mask=(blocks.data_ptr(), count, token_pos.data_ptr()), _max_kv=count * d.page_tokens)


def _capturing() -> bool:
    torch = sys.modules.get("torch")
    return torch is not None and torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


def _not_capturing(what: str):
    if _capturing():
        _refuse(f"{what} while the current stream is being captured")


def _kv_destroy(box: list):
    """box: the handle (None once it is gone) and the device whose work it waits for (None: host only)."""
    handle, device = box
    if not handle:
        return
    if device is not None:
        cuda, st = _torch().cuda, lora_kv_stats()
        _check(lib().lora_kv_get_stats(handle, ctypes.byref(st)))
        if st.pages or st.spare:
            cuda.synchronize(device)
        with cuda.device(device):
            lib().lora_kv_destroy(handle)
    else:
        lib().lora_kv_destroy(handle)
    box[0] = None


_waiting = []  # closes of objects that were collected during a capture


def _close_later(owner):
    """What __del__ does: closes, or under capture, which a wait for the device would end, leaves it to the next call that
    makes, changes or closes a KvCache."""
    try:
        try:
            owner.close()
        except LoraError:
            if _capturing():
                _waiting.append(owner.close)
    except Exception:
        pass


def _close_waiting():
    while _waiting and not _capturing():
        _waiting.pop()()


class KvCache:
    """lora_kv: sequences over the pages of a Pool (which may hold adapters too).  The pool's storage is a
    bf16 tensor [num_pages, page_rows, row_width]; the cache owns a device page table it makes itself.  All calls and the
    kernels that read the pages use one stream, which is the compute stream of a Cache over the same pool.  fp8: 8-bit rows;
    bounds: each page holds the bounds of its keys too (`self.bounds`, a KvBounds)."""

    def __init__(self, pool: Pool, kv_heads: int, head_dim: int, max_seqs: int, max_pages: int, host_only: bool = False,
                 fp8: bool = False, bounds: bool = False):
        torch = _torch()
        _close_waiting()
        self.pool, self.max_pages, self._host_only = pool, max_pages, host_only
        self.page_table = self.bounds = None
        flags = (LORA_KV_FP8 if fp8 else 0) | (LORA_KV_BOUNDS if bounds else 0)
        h = ctypes.c_void_p()
        if host_only:
            _check(lib().lora_kv_create(pool._h, kv_heads, head_dim, max_seqs, max_pages, None, LORA_KV_HOST_ONLY | flags,
                                        ctypes.byref(h)))
            self._own(h, None)
            return
        dev = pool.storage.device
        with _On(dev, None):
            stream = torch.cuda.current_stream(dev)
            if torch.cuda.is_current_stream_capturing():
                _refuse("a KvCache cannot be made while its stream is being captured")
            self.page_table = torch.empty((max_seqs, max_pages), dtype=torch.int32, device=dev)
            # the table may be memory that work still queued on this stream uses, and lora_kv_create, which fills it,
            # knows nothing of the stream
            stream.synchronize()
            _check(lib().lora_kv_create(pool._h, kv_heads, head_dim, max_seqs, max_pages, _dptr(self.page_table), flags,
                                        ctypes.byref(h)))
        self._own(h, dev)
        tokens, size = self.stats()["page_tokens"], kv_heads * head_dim
        flat = pool.storage.view(pool.storage.shape[0], -1)
        if fp8 or bounds:
            bytes8 = flat.view(torch.uint8)
        if fp8:
            codes = bytes8.view(torch.float8_e4m3fn)
            part = lambda t, i, *shape: t[:, i:i + math.prod(shape)].view(-1, *shape)
            rows, n = (kv_heads, tokens, head_dim), kv_heads * tokens
            self.view = KvView(part(codes, 0, *rows), part(codes, size * tokens, *rows), self.page_table,
                               part(bytes8, 2 * size * tokens, kv_heads, tokens), part(bytes8, 2 * size * tokens + n, kv_heads, tokens))
        else:
            part = lambda i: flat[:, i * size * tokens:(i + 1) * size * tokens].view(-1, kv_heads, tokens, head_dim)
            self.view = KvView(part(0), part(1), self.page_table)
        if bounds:
            row = lora_kv_bounds_row_bytes(head_dim)
            self.bounds = KvBounds(self.view, bytes8[:, bytes8.shape[1] - kv_heads * row:].view(-1, kv_heads, row))

    def _own(self, handle, device):
        """The handle in a box that the pool knows too: whichever goes first, the cache is destroyed before the pool."""
        self._box = [handle, device]
        self.pool.__dict__.setdefault("_kv_handles", []).append(self._box)

    @property
    def _h(self):
        return self._box[0]

    def _call(self, name, *args, stream=None):
        _close_waiting()
        if self._host_only:
            _check(getattr(lib(), name)(self._h, *args, None))
            return
        with _On(self.page_table.device, stream) as s:
            _check(getattr(lib(), name)(self._h, *args, s))

    def extend(self, seqs, new_tokens, stream=None):
        a, b = _i32(seqs), _i32(new_tokens)
        if a.size != b.size:
            _refuse(f"{a.size} sequences and {b.size} counts")
        self._call("lora_kv_extend", _np_ptr(a), _np_ptr(b), a.size, stream=stream)

    def fork(self, src: int, dst, stream=None):
        a = _i32(dst)
        self._call("lora_kv_fork", src, _np_ptr(a), a.size, stream=stream)

    def truncate(self, seq: int, new_len: int, stream=None):
        self._call("lora_kv_truncate", seq, new_len, stream=stream)

    def free(self, seqs, stream=None):
        a = _i32(seqs)
        self._call("lora_kv_free", _np_ptr(a), a.size, stream=stream)

    def compact(self, stream=None) -> int:
        n = ctypes.c_int32(0)
        self._call("lora_kv_compact", ctypes.byref(n), stream=stream)
        return n.value

    def trim(self, wait: bool = False) -> int:
        """Pages still spare afterwards; refused under capture, where the marks of their readers cannot be asked."""
        n = ctypes.c_int32(0)
        if not self._host_only:
            _not_capturing("spares cannot be given back")
        _close_waiting()
        _check(lib().lora_kv_trim(self._h, int(wait), ctypes.byref(n)))
        return n.value

    def length(self, seq: int) -> int:
        n = ctypes.c_int32(0)
        _check(lib().lora_kv_seq(self._h, seq, ctypes.byref(n), None, None))
        return n.value

    def pages(self, seq: int) -> np.ndarray:
        ids, n = np.empty(self.max_pages, np.int32), ctypes.c_int32(0)
        _check(lib().lora_kv_seq(self._h, seq, None, _np_ptr(ids), ctypes.byref(n)))
        return ids[: n.value].copy()

    def stats(self) -> dict:
        st = lora_kv_stats()
        _check(lib().lora_kv_get_stats(self._h, ctypes.byref(st)))
        return {f: getattr(st, f) for f, _ in lora_kv_stats._fields_}

    def close(self):
        """Waits for the device and gives the pages back to the pool; refused under capture."""
        box = getattr(self, "_box", None)
        if box is not None:
            if box[0] and box[1] is not None:
                _not_capturing("a KvCache cannot be closed")
            _kv_destroy(box)
            boxes = self.pool.__dict__.get("_kv_handles", [])
            boxes[:] = [b for b in boxes if b is not box]

    def __del__(self):
        try:
            _close_later(self)
        except Exception:  # at the interpreter's end the module's names may be gone
            pass
