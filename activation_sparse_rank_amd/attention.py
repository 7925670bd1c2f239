"""Torch-facing binding of the attention side of a decode layer: rotary
positions (``Rope``, ``qk_rope``), the 8-bit key/value cache (``KVCache``,
``kv_append``, ``kv_read``), attention over it (``attend``) and eviction by
accumulated attention weight (``kv_evict``).

As in ``api``, each function checks what the C ABI cannot see (devices,
types, shapes, strides) and forwards pointers and the current HIP stream;
include/pi.h says what each call computes.  Token rows are
[n_tok, n_heads, head_dim] tensors whose last dimension is contiguous, so
views into a fused projection's output are taken as they are.  Calls run on
the tensors' device.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _lib as L
from .api import _DTYPES, _check, _dev, _ptr

_LAYOUTS = {"half": L.PI_ROPE_HALF, "interleaved": L.PI_ROPE_INTERLEAVED}

# A decode step's calls take a few microseconds on the GPU, less than careless
# checks take here: each check below reads a tensor's attributes once, and
# says what is wrong only after something is (8.2 -> 5.5 us for a
# one-token qk_rope, of which 2.5 are the launch).
_Tensor = torch.Tensor
_int32 = torch.int32
# The current stream's handle without an object around it (1.1 -> 0.1 us).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(stream, dev: int):
    """The raw handle of stream, or of the current stream of device dev."""
    if stream is None:
        return _current_stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _rows(t, name, heads, d, dtype, dev):
    """Checks token rows; returns (pointer, token stride, head stride, tokens)."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev:
        shape = t.shape
        if len(shape) == 3:
            n, h, e = shape
            ts, hs, es = t.stride()
            if h == heads and e == d and es == 1:
                return t.data_ptr(), ts, hs, n
    _bad_rows(t, name, heads, d, dtype, dev)


def _bad_rows(t, name, heads, d, dtype, dev):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must live in GPU memory, on the same device as the rest")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{name} must be [n_tok, {heads}, {d}]")
    raise ValueError(f"{name}: the elements of a head must be contiguous")


def _i32(t, name, n, dev):
    """Checks a contiguous int32 vector of n entries on device dev; returns its pointer."""
    if (isinstance(t, _Tensor) and t.dtype is _int32 and t.get_device() == dev and t.shape == (n,)
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != _int32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 [{n}]")
    raise ValueError(f"{name} must live in GPU memory, on the same device as the rest")


def _same(t, name, like, dtype, dev):
    """Checks a contiguous tensor of dtype with the shape ``like`` on device dev; returns its pointer."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == like and t.is_contiguous():
        return t.data_ptr()
    _dev(t, name)
    if t.dtype != dtype or t.shape != like:
        raise ValueError(f"{name} must be {dtype} {list(like)}")
    raise ValueError(f"{name} must be on the same device as the rest")


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
        self._ref = ctypes.byref(self.desc)


def qk_rope(rope: Rope, q, k, pos, q_out=None, k_out=None, stream=None):
    """Norms (where rope has weights) and rotation of queries and keys at the
    positions ``pos`` (int32 [n_tok]), in one pass (pi_qk_rope).  Without
    ``q_out`` / ``k_out`` the inputs are rotated in place.  Returns (q_out, k_out)."""
    if not (isinstance(q, _Tensor) and isinstance(k, _Tensor) and q.dim() == 3 and k.dim() == 3):
        raise TypeError("q and k must be tensors [n_tok, heads, head_dim]")
    dev, dt, d = rope._dev, q.dtype, rope.head_dim
    if dt not in _DTYPES:
        raise TypeError("q must be float16 or float32")
    h, hk = q.shape[1], k.shape[1]
    q_out, k_out = q if q_out is None else q_out, k if k_out is None else k_out
    qp, qt, qh, n = _rows(q, "q", h, d, dt, dev)
    kp, kt, kh, nk = _rows(k, "k", hk, d, dt, dev)
    qo, qot, qoh, nqo = _rows(q_out, "q_out", h, d, dt, dev)
    ko, kot, koh, nko = _rows(k_out, "k_out", hk, d, dt, dev)
    if not n == nk == nqo == nko:
        raise ValueError("q, k and their outputs must have the same tokens")
    if n == 0:
        return q_out, k_out
    _check(L.load().pi_qk_rope(rope._ref, qp, qt, qh, h, kp, kt, kh, hk, _i32(pos, "pos", n, dev), n, _DTYPES[dt],
                               qo, qot, qoh, ko, kot, koh, _stream(stream, dev)), "pi_qk_rope")
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
        if d not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        if pages.dtype != torch.uint8 or pages.dim() != 3 or pages.shape[1:] != (2, L.PI_KV_BLOCK * d):
            raise ValueError("pages must be uint8 [n_pages, 2, 32 * head_dim]")
        if scales.dtype != torch.float32 or scales.shape != (pages.shape[0], 2):
            raise ValueError("scales must be float32 [n_pages, 2]")
        if table.dtype != torch.int32 or table.dim() != 3 or table.shape[:2] != (s, h):
            raise ValueError("table must be int32 [n_seqs, n_kv_heads, max_blocks]")
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
        self._ref = ctypes.byref(self.desc)


def kv_append(cache: KVCache, k, v, lens, q_start=None, max_new=None, stream=None):
    """Append token rows to the cache (pi_kv_append).  ``lens`` (int32
    [n_seqs]) counts the tokens held after the call; ``q_start`` (int32
    [n_seqs + 1]) gives each sequence's rows, at most ``max_new`` of them
    (default: all rows of k); without it every sequence has max_new rows, one after the other
    (default: n_tok / n_seqs)."""
    h, d, dt, dev = cache.n_kv_heads, cache.head_dim, cache.dtype, cache._dev
    kp, kt, kh, n = _rows(k, "k", h, d, dt, dev)
    vp, vt, vh, nv = _rows(v, "v", h, d, dt, dev)
    if n != nv:
        raise ValueError("k and v must have the same tokens")
    lp, qp, max_new = _bounds(cache, lens, q_start, max_new, n, dev)
    if n == 0:
        return
    _check(L.load().pi_kv_append(cache._ref, kp, kt, kh, vp, vt, vh, n, lp, qp, max_new, _stream(stream, dev)),
           "pi_kv_append")


def kv_read(cache: KVCache, lens, k_out, v_out, q_start=None, max_new=None, stream=None):
    """The values that the cache holds for the last rows of each sequence
    (pi_kv_read); lens, q_start and max_new as for kv_append."""
    h, d, dt, dev = cache.n_kv_heads, cache.head_dim, cache.dtype, cache._dev
    kp, kt, kh, n = _rows(k_out, "k_out", h, d, dt, dev)
    vp, vt, vh, nv = _rows(v_out, "v_out", h, d, dt, dev)
    if n != nv:
        raise ValueError("k_out and v_out must have the same tokens")
    lp, qp, max_new = _bounds(cache, lens, q_start, max_new, n, dev)
    if n == 0:
        return
    _check(L.load().pi_kv_read(cache._ref, lp, qp, max_new, kp, kt, kh, vp, vt, vh, n, _stream(stream, dev)),
           "pi_kv_read")


def _bounds(cache, lens, q_start, max_q, n, dev):
    """Pointers of lens and q_start, and the bound on a sequence's rows."""
    s = cache.n_seqs
    lp = _i32(lens, "lens", s, dev)
    if q_start is None:
        if max_q is None:
            max_q = n // s
        if n != s * max_q:
            raise ValueError("without q_start there must be n_seqs * max rows")
        return lp, None, max_q
    return lp, _i32(q_start, "q_start", s + 1, dev), n if max_q is None else max_q


def attend_workspace_bytes(cache: KVCache, n_heads: int, max_q: int, max_len=None, add_score: bool = False) -> int:
    """Bytes of workspace attend needs for these bounds (pi_attend_workspace_bytes)."""
    from .api import PiError
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
    ``max_q`` as for kv_append; ``max_len``: bound on lens (default: what the
    table holds); ``scale``: 1 / sqrt(head_dim) by default; ``add_score``: add the
    weights of each block to cache.score.  ``ws`` from alloc_attend_workspace
    with the same bounds (one is allocated where it is None)."""
    d, dt, dev = cache.head_dim, cache.dtype, cache._dev
    if not (isinstance(q, _Tensor) and q.dim() == 3):
        raise TypeError("q must be a tensor [n_tok, n_heads, head_dim]")
    h = q.shape[1]
    qp, qt, qh, n = _rows(q, "q", h, d, dt, dev)
    op, ot, oh, no = _rows(out, "out", h, d, dt, dev)
    if n != no:
        raise ValueError("q and out must have the same tokens")
    lp, sp, max_q = _bounds(cache, lens, q_start, max_q, n, dev)
    if n == 0:
        return
    if max_len is None:
        max_len = cache.max_blocks * L.PI_KV_BLOCK
    if add_score and cache.score is None:
        raise ValueError("add_score needs a cache with a score")
    if ws is None:
        ws = _temp_attend_workspace(cache, h, max_q, max_len, add_score, stream)
    elif ws.dtype != torch.uint8 or not ws.is_contiguous() or ws.get_device() != dev:
        raise ValueError("ws must be contiguous uint8 on the cache's device")
    _check(L.load().pi_attend(cache._ref, qp, qt, qh, h, n, lp, sp, max_q, max_len,
                              d ** -0.5 if scale is None else scale, bool(add_score), op, ot, oh, ws.data_ptr(),
                              ws.numel(), _stream(stream, dev)), "pi_attend")


def _temp_attend_workspace(cache, h, max_q, max_len, add_score, stream):
    """A workspace for one call, allocated on the call's stream, so that its
    memory is handed out again only in that stream's order."""
    if stream is None:
        return alloc_attend_workspace(cache, h, max_q, max_len, add_score)
    s = stream
    if not isinstance(s, torch.cuda.Stream):
        s = torch.cuda.ExternalStream(int(stream), device=cache.pages.device)
    with torch.cuda.stream(s):
        return alloc_attend_workspace(cache, h, max_q, max_len, add_score)


def kv_evict(table, score, lens, keep: int, recent: int, lens_out, table_out=None, score_out=None, stream=None):
    """Evict the blocks with the least accumulated weight (pi_kv_evict): of
    each (sequence, kv head) with more than ``keep`` blocks stay the last
    ``recent`` and the heaviest others; the pages that leave follow them in the
    table.  Without ``table_out`` and ``score_out`` table and score are
    rewritten in place; ``lens_out`` (int32 [n_seqs]) is never ``lens``."""
    if not isinstance(table, _Tensor) or table.dtype is not _int32 or table.dim() != 3:
        raise ValueError("table must be an int32 tensor [n_seqs, n_kv_heads, max_blocks]")
    shape, dev = table.shape, table.get_device()
    if dev < 0:
        raise ValueError("table must live in GPU memory")
    tp, sp = _same(table, "table", shape, _int32, dev), _same(score, "score", shape, torch.float32, dev)
    if (table_out is None) != (score_out is None):
        raise ValueError("table_out and score_out go together")
    if table_out is None:
        to, so = tp, sp
    else:
        to = _same(table_out, "table_out", shape, _int32, dev)
        so = _same(score_out, "score_out", shape, torch.float32, dev)
    s, h, n = shape
    _check(L.load().pi_kv_evict(tp, sp, _i32(lens, "lens", s, dev), s, h, n, keep, recent, to, so,
                                _i32(lens_out, "lens_out", s, dev), _stream(stream, dev)), "pi_kv_evict")
