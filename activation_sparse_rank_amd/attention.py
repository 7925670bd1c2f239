"""Torch-facing binding of the attention side of a decode layer: rotary
positions (``Rope``, ``qk_rope``), the 8-bit key/value cache (``KVCache``,
``kv_append``, ``kv_read``), attention over it (``attend``) and eviction by
accumulated attention weight (``kv_evict``).

As in ``api``, each function checks what the C ABI cannot see (devices,
types, shapes, strides) and forwards pointers and the current HIP stream;
include/pi_attn.h says what each call computes.  The checks are native
(csrc/bind_attn.cpp): these calls run for a few microseconds each, once or more per
layer and token.  Token rows are
[n_tok, n_heads, head_dim] tensors whose last dimension is contiguous, so
views into a fused projection's output are taken as they are.  Calls run on
the tensors' device.
"""

from __future__ import annotations

import ctypes
import importlib
import math

import torch

from . import _lib as L
from .api import _DTYPES, PiError, _dev, _ptr

_LAYOUTS = {"half": L.PI_ROPE_HALF, "interleaved": L.PI_ROPE_INTERLEAVED}

_native = None


def load_native():
    """Load the native module that checks the tensors and calls libpi (bind_attn.cpp); raise if it has not been built."""
    global _native
    if _native is None:
        lib = L.load()
        try:
            native = importlib.import_module("._attn", __package__)
        except ImportError as e:
            raise ImportError("the attention side's binding is not built; run `python -m "
                              f"activation_sparse_rank_amd.build` ({e})") from e
        native.use_library(lib._handle)
        _native = native
    return _native


def _handle(stream):
    """The raw handle of a stream; None stays None (the tensors' device's current stream)."""
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


class Rope:
    """A rotation of heads (pi_rope).

    ``freqs``: float64 [rot / 2], turns per position (radians / 2 pi) of each
    rotated pair, with whatever scaling for long contexts the model uses
    (plain: ``base ** (-2 i / rot) / (2 pi)``);
    ``layout``: "half" pairs (i, i + rot / 2), "interleaved" pairs (2 i, 2 i + 1);
    ``scale`` multiplies the rotated elements; ``q_norm`` / ``k_norm``:
    float32 [head_dim] weights of an RMS norm of each head before the rotation.
    """

    def __init__(self, freqs, head_dim: int, layout: str = "half", scale: float = 1.0, q_norm=None, k_norm=None,
                 eps: float = 1e-6):
        if layout not in _LAYOUTS:
            raise ValueError(f"unknown layout {layout!r}")
        _dev(freqs, "freqs")
        if freqs.dtype != torch.float64 or freqs.dim() != 1:
            raise TypeError("freqs must be float64 [rot / 2]")
        head_dim, rot = int(head_dim), 2 * freqs.shape[0]
        if head_dim < 8 or head_dim > 256 or head_dim % 8:
            raise ValueError("head_dim must be a multiple of 8, at most 256")
        if rot < 2 or rot > head_dim:
            raise ValueError("freqs must have 1 to head_dim / 2 entries")
        for w, n in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if w is not None:
                _dev(w, n)
                if w.dtype != torch.float32 or w.shape != (head_dim,):
                    raise ValueError(f"{n} must be float32 [head_dim]")
                if w.device != freqs.device:
                    raise ValueError(f"{n} must be on the device of freqs")
        if not (math.isfinite(scale) and math.isfinite(eps) and eps >= 0):
            raise ValueError("scale and eps must be finite, eps not negative")
        self.freqs, self.q_norm, self.k_norm = freqs, q_norm, k_norm
        self.head_dim, self.rot, self.layout, self.scale, self.eps = head_dim, rot, layout, scale, eps
        self._dev = freqs.get_device()
        self.desc = L.PiRope(head_dim, rot, _LAYOUTS[layout], scale, eps, freqs.data_ptr(), _ptr(q_norm), _ptr(k_norm))
        self._addr = ctypes.addressof(self.desc)


def qk_rope(rope: Rope, q, k, pos, q_out=None, k_out=None, stream=None):
    """Norms (where rope has weights) and rotation of queries and keys at the
    positions ``pos`` (int32 [n_tok]), in one pass (pi_qk_rope).  Without
    ``q_out`` / ``k_out`` the inputs are rotated in place.  Returns (q_out, k_out)."""
    q_out, k_out = q if q_out is None else q_out, k if k_out is None else k_out
    st = (_native or load_native()).qk_rope(rope._addr, rope._dev, q, k, pos, q_out, k_out, _handle(stream))
    if st:
        raise PiError(st, "pi_qk_rope")
    return q_out, k_out


class KVCache:
    """The 8-bit cache of one layer (pi_kv_cache).

    ``pages``: uint8 [n_pages, 2, 32 * head_dim]; ``scales``: float32
    [n_pages, 2]; ``open``: float16 or float32 [n_seqs, n_kv_heads, 2, 32,
    head_dim], the last block's rows as they came; ``table``: int32 [n_seqs,
    n_kv_heads, max_blocks] page numbers; ``score``: float32 like table, the
    accumulated attention weight (optional).  All stay the caller's.
    """

    def __init__(self, pages, scales, open, table, score=None):
        for t, n in ((pages, "pages"), (scales, "scales"), (open, "open"), (table, "table")):
            _dev(t, n)
        if open.dim() != 5 or open.shape[2] != 2 or open.shape[3] != L.PI_KV_BLOCK or open.dtype not in _DTYPES:
            raise ValueError("open must be float16 or float32 [n_seqs, n_kv_heads, 2, 32, head_dim]")
        s, h, _, _, d = open.shape
        if s < 1 or h < 1:
            raise ValueError("open must have sequences and heads")
        if d not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        if pages.dtype != torch.uint8 or pages.dim() != 3 or pages.shape[1:] != (2, L.PI_KV_BLOCK * d):
            raise ValueError("pages must be uint8 [n_pages, 2, 32 * head_dim]")
        if pages.shape[0] < 1:
            raise ValueError("pages must have a page")
        if scales.dtype != torch.float32 or scales.shape != (pages.shape[0], 2):
            raise ValueError("scales must be float32 [n_pages, 2]")
        if table.dtype != torch.int32 or table.dim() != 3 or table.shape[:2] != (s, h):
            raise ValueError("table must be int32 [n_seqs, n_kv_heads, max_blocks]")
        if table.shape[2] < 1:
            raise ValueError("table must have blocks")
        if score is not None:
            _dev(score, "score")
            if score.dtype != torch.float32 or score.shape != table.shape:
                raise ValueError("score must be float32 with the shape of table")
        for t, n in ((scales, "scales"), (open, "open"), (table, "table"), (score, "score")):
            if t is not None and t.device != pages.device:
                raise ValueError(f"{n} must be on the device of pages")
        self.pages, self.scales, self.open, self.table, self.score = pages, scales, open, table, score
        self.n_seqs, self.n_kv_heads, self.head_dim, self.max_blocks = s, h, d, table.shape[2]
        self.dtype = open.dtype
        self._dev = pages.get_device()
        self.desc = L.PiKVCache(s, h, d, self.max_blocks, pages.shape[0], _DTYPES[open.dtype], pages.data_ptr(),
                                scales.data_ptr(), open.data_ptr(), table.data_ptr(), _ptr(score))
        self._ref, self._addr = ctypes.byref(self.desc), ctypes.addressof(self.desc)


def kv_append(cache: KVCache, k, v, lens, q_start=None, max_new=None, stream=None):
    """Append token rows to the cache (pi_kv_append).  ``lens`` (int32
    [n_seqs]) counts the tokens held after the call; ``q_start`` (int32
    [n_seqs + 1]) gives each sequence's rows, at most ``max_new`` of them
    (default: all rows of k, or as many as a table row holds); without it every
    sequence has max_new rows, one after the other (default: n_tok / n_seqs)."""
    st = (_native or load_native()).kv_append(cache._addr, cache._dev, k, v, lens, q_start, max_new, _handle(stream))
    if st:
        raise PiError(st, "pi_kv_append")


def kv_read(cache: KVCache, lens, k_out, v_out, q_start=None, max_new=None, stream=None):
    """The values that the cache holds for the last rows of each sequence
    (pi_kv_read); lens, q_start and max_new as for kv_append."""
    st = (_native or load_native()).kv_read(cache._addr, cache._dev, k_out, v_out, lens, q_start, max_new, _handle(stream))
    if st:
        raise PiError(st, "pi_kv_read")


def attend_workspace_bytes(cache: KVCache, n_heads: int, max_q: int, max_len=None, add_score: bool = False) -> int:
    """Bytes of workspace attend needs for these bounds (pi_attend_workspace_bytes)."""
    if max_len is None:
        max_len = cache.max_blocks * L.PI_KV_BLOCK
    n = L.load().pi_attend_workspace_bytes(cache._ref, int(n_heads), int(max_q), int(max_len), int(add_score))
    if n == 0:
        raise PiError(L.PI_E_SHAPE, "pi_attend_workspace_bytes")
    return int(n)


def alloc_attend_workspace(cache: KVCache, n_heads: int, max_q: int, max_len=None,
                           add_score: bool = False) -> torch.Tensor:
    """A workspace for attend with these bounds, its header zero (so its fault flags start clear)."""
    ws = torch.empty(attend_workspace_bytes(cache, n_heads, max_q, max_len, add_score), dtype=torch.uint8,
                     device=cache.pages.device)
    ws[:L.PI_WS_HEADER_BYTES].zero_()
    return ws


def attend(cache: KVCache, q, lens, out, q_start=None, max_q=None, max_len=None, scale=None, add_score: bool = False,
           ws=None, stream=None):
    """out = softmax(scale * q k^T) v over the cache (pi_attend).

    ``q``, ``out``: [n_tok, n_heads, head_dim]; the rows of a sequence are its
    last tokens, each sees the tokens up to itself.  ``lens``, ``q_start``,
    ``max_q`` as for kv_append (max_q by default all rows of q); ``max_len``: bound on lens (default: what the
    table holds); ``scale``: 1 / sqrt(head_dim) by default; ``add_score``: add the
    weights of each block to cache.score.  ``ws`` from alloc_attend_workspace
    with the same bounds (one is allocated where it is None)."""
    if max_len is None:
        max_len = cache.max_blocks * L.PI_KV_BLOCK
    if ws is None:
        ws = _temp_attend_workspace(cache, q, max_q, max_len, add_score, q_start, stream)
    st = (_native or load_native()).attend(cache._addr, cache._dev, q, lens, out, q_start, max_q, max_len,
                                     cache.head_dim ** -0.5 if scale is None else scale, add_score, ws,
                                     _handle(stream))
    if st:
        raise PiError(st, "pi_attend")


def _temp_attend_workspace(cache, q, max_q, max_len, add_score, q_start, stream):
    """A workspace for one call, allocated on the call's stream, so that its
    memory is handed out again only in that stream's order."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 3):
        raise TypeError("q must be a tensor [n_tok, n_heads, head_dim]")
    if max_q is None:
        max_q = q.shape[0] if q_start is not None else q.shape[0] // cache.n_seqs
    if stream is None:
        return alloc_attend_workspace(cache, q.shape[1], max(1, max_q), max_len, add_score)
    s = stream
    if not isinstance(s, torch.cuda.Stream):
        s = torch.cuda.ExternalStream(int(stream), device=cache.pages.device)
    with torch.cuda.stream(s):
        return alloc_attend_workspace(cache, q.shape[1], max(1, max_q), max_len, add_score)


def kv_evict(table, score, lens, keep: int, recent: int, lens_out, table_out=None, score_out=None, stream=None):
    """Evict the blocks with the least accumulated weight (pi_kv_evict): of
    each (sequence, kv head) with more than ``keep`` blocks stay the last
    ``recent`` and the heaviest others; the pages that leave follow them in the
    table.  Without ``table_out`` and ``score_out`` table and score are
    rewritten in place; ``lens_out`` (int32 [n_seqs]) is never ``lens``."""
    if (table_out is None) != (score_out is None):
        raise ValueError("table_out and score_out go together")
    if table_out is None:
        table_out, score_out = table, score
    st = (_native or load_native()).kv_evict(table, score, lens, keep, recent, lens_out, table_out, score_out,
                                       _handle(stream))
    if st:
        raise PiError(st, "pi_kv_evict")
