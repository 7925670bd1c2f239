"""What the attention tests share beside test_gpu_attention's cache: calls that
between them take every kernel and way of cutting the work, and a check against
the formula in 64 bits, a kv head at a time."""

import math

import numpy as np
import torch

import activation_sparse_rank_amd as pi
from helpers import host
from test_gpu_attention import DEV, HALF, Cache, _attend, _filled

f16, f32 = torch.float16, torch.float32

# name: dtype, head size, lengths, new rows of a sequence (at most), kv heads, query heads to each
CALLS = {
    "one tile": (f16, 64, (700, 90), 1, 2, 8),
    "one tile, split": (f16, 128, (3000,), 1, 1, 8),
    "one tile, split by lengths": (f16, 64, (4000, 40, 2500), 1, 2, 8),
    "two tiles": (f16, 64, (700, 90), 3, 2, 8),
    "two tiles, wide": (f16, 128, (700, 90), 3, 2, 8),
    "fp32, one tile": (f32, 128, (700, 90), 1, 2, 8),
    "fp32, two tiles": (f32, 64, (700, 90), 3, 2, 8),
    "fp32, split": (f32, 64, (3000,), 1, 1, 8),
    "fp32, a few splits": (f32, 128, (1500,), 5, 8, 6),
    "fp32, split by lengths": (f32, 64, (4000, 40, 2500), 1, 2, 8),
    "fp32, three workgroups": (f32, 128, (700, 90), 5, 2, 8),
    "two waves": (f16, 128, (1100,) + (60,) * 7, 5, 8, 8),
    "four waves": (f16, 128, (1100,) + (60,) * 7, 9, 8, 8),
    "eight waves": (f16, 128, (1100,) + (60,) * 7, 17, 8, 8),
    "eight waves, two tiles": (f16, 128, (1500,), 400, 8, 8),
    "two groups": (f16, 64, (1100,), 40, 2, 8),
    "two tiles, many sequences": (f16, 64, (900,) + (340,) * 4, 300, 8, 16),
    "short prompts": (f16, 64, (300, 129), 60, 1, 8),
    "short prompts, wide": (f16, 128, (300, 129), 60, 1, 8),
    "fp32, two waves": (f32, 64, (1000,) + (50,) * 8, 5, 8, 8),
    "fp32, four waves": (f32, 64, (1000,) + (50,) * 8, 9, 8, 8),
    "fp32, eight waves": (f32, 64, (1000,) + (50,) * 8, 17, 8, 8),
    "fp32, eight waves, two tiles": (f32, 64, (1500,), 500, 8, 8),
    "fp32, wide, two waves": (f32, 128, (1000,) + (50,) * 8, 3, 8, 8),
    "fp32, wide, four waves": (f32, 128, (1000,) + (50,) * 8, 5, 8, 8),
    "fp32, wide, eight waves": (f32, 128, (1000,) + (50,) * 8, 9, 8, 8),
}


class Call:
    """A filled cache and the queries of a call, which a test may change before run()."""

    def __init__(self, call, score=False, seed=0, slack=2):
        self.dt, self.d, self.lens, new, self.hk, self.group = call
        self.c = _filled(len(self.lens), self.hk, self.d, self.dt, self.lens, seed, score, slack)
        self.new = [min(new, n) for n in self.lens]
        self.max_new = new
        n = sum(self.new)
        g = torch.Generator(device=DEV).manual_seed(seed + n)
        self.q = torch.randn((n, self.hk * self.group, self.d), generator=g, device=DEV).to(self.dt)
        self.ln = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.start = np.concatenate(([0], np.cumsum(self.new)))
        self.qs = torch.from_numpy(self.start.astype(np.int32)).to(DEV)
        self.score = score
        self.gen = g

    def run(self, **kw):
        self.score0 = self.c.score.clone() if self.score else None
        self.out, self.ws = _attend(self.c, self.q, self.ln, self.qs, self.max_new, self.score, **kw)
        return self.out

    def pages(self, s, h):
        """Page numbers of the blocks that a kv head of a sequence holds."""
        return self.c.table[s, h, :(self.lens[s] + 31) // 32].long()

    def check(self, scale=None, seqs=None, heads=None, two_parts=False, alike=False):
        """Every row against the formula, tolerances as in test_gpu_attention; two_parts: weights to 2^-22 in fp16
        too; alike: the blocks' terms are all alike, so the sums' roundings (2^-24 each) add up and do not average out."""
        scale = self.d ** -0.5 if scale is None else scale
        for s in range(len(self.lens)) if seqs is None else seqs:
            for h in range(self.hk) if heads is None else heads:
                self._check_head(s, h, scale, two_parts, alike)

    def _check_head(self, s, h, scale, two_parts, alike):
        n, new, group, d = self.lens[s], self.new[s], self.group, self.d
        rows = slice(int(self.start[s]), int(self.start[s + 1])), slice(h * group, (h + 1) * group)
        k, v = self.c.values(s, h)
        q = host(self.q[rows]).astype(np.float64).reshape(new * group, d)
        got = host(self.out[rows]).astype(np.float64).reshape(new * group, d)
        sees = np.repeat(n - new + 1 + np.arange(new), group)
        logit = q @ k.T * scale
        hidden = np.arange(n)[None] >= sees[:, None]
        size = np.where(hidden, 0, np.abs(q) @ np.abs(k).T * scale).max(1)
        logit[hidden] = -np.inf
        w = np.exp(logit - logit.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        ref, mag = w @ v, w @ np.abs(v)
        nb = (n + 31) // 32
        part = 2.0 ** -22 if two_parts or self.dt == f32 else 2.0 ** -11
        rel = 2.0 ** -20 * size[:, None] + 2.0 ** -22 * (8 + (nb / 4 if alike else math.sqrt(nb)))
        tol = HALF[self.dt] * np.abs(ref) + (part + rel) * mag + 2.0 ** -31 * np.where(hidden, 0, 1) @ np.abs(v)
        tol = tol + 2.0 ** -25 * (self.dt == f16)
        err = np.abs(got - ref)
        assert (err <= tol).all(), (s, h, float(np.max(err / np.maximum(tol, 1e-300))))
        if self.score:
            s0, s1 = (host(x[s, h]).astype(np.float64) for x in (self.score0, self.c.score))
            pad = np.zeros((len(w), nb * 32))
            pad[:, :n] = w
            wb = pad.reshape(len(w), nb, 32).sum(2)
            tol = (wb * rel).sum(0) + 2.0 ** -23 * (s0[:nb] + wb.sum(0)) + 1e-30
            err = np.abs(s1[:nb] - (s0[:nb] + wb.sum(0)))
            assert (err <= tol).all(), (s, h, float(np.max(err / tol)))
            assert np.array_equal(s1[nb:], s0[nb:])


class Tail(Call):
    """A long sequence, among so many of one token that nothing is split over workgroups (their table rows name its
    pages too).  The first token of each of its first eight blocks takes the row; every other token's weight is 2^-bits
    of one of theirs.  Values: the heavy tokens' are 64 of their block's scale, the others' -100 of theirs.  Keys and
    queries have one element."""

    tokens, seqs = 1 << 17, 300

    def __init__(self, dt, d, new, heads, bits=21.6):
        self.dt, self.d, self.hk, self.group, self.score = dt, d, 1, heads, False
        nb = self.tokens // 32
        self.c = c = Cache(1, 1, d, nb, dt)
        c.rows = [np.zeros((2, 1, self.tokens, d), np.float16)]
        c.pages.fill_(128)
        at = c.table[0, 0].long()
        c.pages[at, 1] = 28
        c.pages[at[:8], 0, 0] = 255                              # the first token's first element: code 127
        e = torch.arange(d, device=DEV)
        c.pages[at[:8, None], 1, (e // 32 * 1024 + e % 16 * 16 + e // 16 % 2 * 8)[None]] = 192
        c.scales.fill_(1.0)
        c.scales[:, 0] = bits * math.log(2.0) / (127 * 2.0 * d ** -0.5)
        open_ = torch.zeros((self.seqs, 1, 2, 32, d), dtype=dt, device=DEV)
        c.c = pi.KVCache(c.pages, c.scales, open_, c.table.expand(self.seqs, 1, nb).contiguous())
        self.lens, self.new, self.max_new = (self.tokens,) + (1,) * (self.seqs - 1), [new] + [1] * (self.seqs - 1), new
        self.start = np.concatenate(([0], np.cumsum(self.new)))
        self.ln = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.qs = torch.from_numpy(self.start.astype(np.int32)).to(DEV)
        self.q = torch.zeros((sum(self.new), heads, d), dtype=dt, device=DEV)
        self.q[:, :, 0] = 2.0
        self.at = at
