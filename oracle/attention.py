"""The attention side of a decode layer in numpy float64: rotation of heads,
the 8-bit cache's quantisation and byte order, attention, eviction."""

from __future__ import annotations

import numpy as np

BLOCK = 32


def rope(x, pos, freqs, layout="half", scale=1.0, norm=None, eps=1e-6):
    """x [n, heads, d] at positions pos [n]; freqs [rot / 2] in turns per position."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    if norm is not None:
        y = y / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(norm, np.float64)
    half = len(freqs)
    i = np.arange(half)
    ia, ib = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
    turns = np.asarray(pos, np.float64)[:, None] * np.asarray(freqs, np.float64)
    ang = 2.0 * np.pi * (turns - np.floor(turns))
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = y[..., ia], y[..., ib]
    out = y.copy()
    out[..., ia] = scale * (a * c - b * s)
    out[..., ib] = scale * (b * c + a * s)
    return out


def quantise(rows):
    """Codes [32, d] (uint8) and the fp32 scale of one half of a block; rows [<= 32, d]."""
    rows = np.asarray(rows, np.float64)
    codes = np.full((BLOCK, rows.shape[1]), 128, np.uint8)
    if not np.isfinite(rows).all():
        return codes, np.float32(np.nan)
    amax = np.abs(rows).max() if rows.size else 0.0
    if amax > 0:
        codes[:len(rows)] = (128 + np.rint(127.0 * rows / amax)).astype(np.uint8)
    return codes, np.float32(amax / 127.0)


def key_offset(t, e, d):
    return (((t // 16) * (d // 64) + e // 64) * 4 + e // 16 % 4) * 256 + t % 16 * 16 + e % 16


def value_offset(t, e, d):
    return (e // 32 * 4 + t % 16 // 4) * 256 + e % 16 * 16 + e // 16 % 2 * 8 + t // 16 * 4 + t % 4


def to_page(key_codes, value_codes):
    """A page's bytes [2, 32 d] from the codes [32, d] of keys and values."""
    d = key_codes.shape[1]
    t, e = np.arange(BLOCK)[:, None], np.arange(d)[None]
    page = np.zeros((2, BLOCK * d), np.uint8)
    page[0, key_offset(t, e, d)] = key_codes
    page[1, value_offset(t, e, d)] = value_codes
    return page


def page_values(page, scales, d):
    """Keys and values [32, d] that a page holds, in float64."""
    t, e = np.arange(BLOCK)[:, None], np.arange(d)[None]
    k = (page[0][key_offset(t, e, d)].astype(np.float64) - 128) * np.float64(scales[0])
    v = (page[1][value_offset(t, e, d)].astype(np.float64) - 128) * np.float64(scales[1])
    return k, v


def attend(q, k, v, sees, scale):
    """One kv head: q [rows, d] over k, v [tokens, d]; row i sees the first
    sees[i] tokens.  Returns out [rows, d], weights [rows, tokens], and per row
    what bounds its rounding: sum of weight * |v| and the largest sum |q k| * scale."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out, w = np.zeros((len(q), v.shape[1])), np.zeros((len(q), len(k)))
    mag, slog = np.zeros_like(out), np.zeros(len(q))
    for i, n in enumerate(sees):
        n = int(min(max(n, 0), len(k)))
        if n == 0:
            continue
        s = k[:n] @ q[i] * scale
        p = np.exp(s - s.max())
        p /= p.sum()
        w[i, :n] = p
        out[i] = p @ v[:n]
        mag[i] = p @ np.abs(v[:n])
        slog[i] = (np.abs(k[:n]) @ np.abs(q[i])).max() * scale
    return out, w, mag, slog


def evict(table, score, length, keep, recent):
    """One row of the table: (table, score, length) after eviction."""
    table, score = list(table), list(score)
    nb = min((max(int(length), 0) + BLOCK - 1) // BLOCK, len(table))
    length = min(max(int(length), 0), len(table) * BLOCK)
    if nb <= keep:
        return np.array(table, np.int32), np.array(score, np.float32), length

    def key(b):
        x = float(score[b])
        return (0, 0.0, b) if np.isnan(x) else (1, -x, b)

    order = sorted(range(nb - recent), key=key)
    stay = sorted(order[:keep - recent]) + list(range(nb - recent, nb))
    leave = sorted(order[keep - recent:])
    t = [table[b] for b in stay + leave] + table[nb:]
    s = [score[b] for b in stay] + [0.0] * len(leave) + score[nb:]
    return np.array(t, np.int32), np.array(s, np.float32), length - BLOCK * (nb - keep)
