"""The attention side on the GPU against the float64 oracle (oracle/attention.py).

Tolerances, from the formulas (u = 2^-24, half a step of fp32; h = half a step of
the rows' type: 2^-11 fp16, 2^-24 fp32):
  * codes, scales, tables, lengths: equal; values read back: the fp32 product,
    rounded once, equal.
  * rope: the rounding h |y|, and for the angle (2^-26 of a turn), the sine's last
    bits, the norm and the two products 2^-20 of the largest |x w| scale in the head.
  * attention, with A = sum of weight * |v| and s = largest sum |q k| * scale of
    the row: the output's rounding h |out|; weights rounded to fp16 once,
    2^-11 A (two parts, 2^-22, for fp32), and below fp16's smallest step by 2^-31 of
    the largest, 2^-31 sum |v|; fp32 logits (sums of up to 256
    products of up to 2^-22 each, and an exponent as large), 2^-21 s A twice;
    the sums over n blocks, 2^-22 (8 + sqrt(n)) A.
  * weights of a block w: the logits' and sums' terms, and u times the score.
"""

import math

import numpy as np
import pytest
import torch

import activation_sparse_rank_amd as pi
from activation_sparse_rank_amd import _lib as L
from helpers import host, require_gpu
from oracle import attention as oa

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
f16, f32 = torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# ---- rope -----------------------------------------------------------------

def _freqs(rot, base=10000.0):
    i = np.arange(rot // 2)
    return base ** (-2.0 * i / rot) / (2 * np.pi)


def _check_rope(y, x, pos, freqs, layout, scale, w, eps, dt):
    ref = oa.rope(host(x), host(pos), freqs, layout, scale, None if w is None else host(w), eps)
    flat = oa.rope(host(x), np.zeros(len(pos)), freqs, layout, 1.0, None if w is None else host(w), eps)
    tol = HALF[dt] * np.abs(ref) + 2.0 ** -20 * max(1.0, scale) * np.abs(flat).max(-1, keepdims=True) + 2.0 ** -25 * (dt == f16)
    err = np.abs(host(y).astype(np.float64) - ref)
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-300)):.2f} of the tolerance"


@pytest.mark.parametrize("dt", [f16, f32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,n,h,hk,norm", [(128, 128, 1, 64, 8, False), (128, 64, 3, 5, 1, True), (64, 20, 37, 7, 7, True),
                                               (80, 80, 600, 3, 1, False), (256, 256, 2, 2, 2, True), (8, 2, 5, 1, 1, True)])
def test_rope(dt, layout, d, rot, n, h, hk, norm):
    g = torch.Generator(device=DEV).manual_seed(n * d + rot)
    qkv = torch.randn((n, (h + 2 * hk) * d), generator=g, device=DEV).to(dt)
    q, k = qkv[:, :h * d].unflatten(1, (h, d)), qkv[:, h * d:(h + hk) * d].unflatten(1, (hk, d))
    pos = torch.randint(-5, 1 << 21, (n,), generator=g, device=DEV).to(torch.int32)
    fr = _freqs(rot)
    wq = 1 + 0.3 * torch.randn(d, generator=g, device=DEV) if norm else None
    r = pi.Rope(torch.from_numpy(fr).to(DEV), d, layout, 1.3, wq, None, 1e-5)
    qo, ko = torch.empty((n, h, d), dtype=dt, device=DEV), torch.full((n, hk, d), 7.0, dtype=dt, device=DEV)
    x0 = qkv.clone()
    pi.qk_rope(r, q, k, pos, qo, ko)
    torch.cuda.synchronize()
    assert torch.equal(qkv, x0), "inputs changed"
    _check_rope(qo, q, pos, fr, layout, 1.3, wq, 1e-5, dt)
    _check_rope(ko, k, pos, fr, layout, 1.3, None, 1e-5, dt)
    # in place, on the strided views: the same bits, and the values untouched
    pi.qk_rope(r, q, k, pos)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, (h + hk) * d:], x0[:, (h + hk) * d:])


def test_rope_head_major_and_values_that_are_no_numbers():
    n, h, d = 9, 4, 64
    x = torch.randn((h, n, d), device=DEV).to(f16)
    x[1, 3, 5], x[2, 4, 0] = float("inf"), float("nan")
    q = x.transpose(0, 1)                                        # [n, h, d], head stride above the token's
    k = torch.randn((n, 1, d), device=DEV).to(f16)
    pos = torch.arange(n, dtype=torch.int32, device=DEV)
    fr = _freqs(d)
    r = pi.Rope(torch.from_numpy(fr).to(DEV), d)
    qo, ko = torch.empty((n, h, d), dtype=f16, device=DEV), torch.empty_like(k)
    pi.qk_rope(r, q, k, pos, qo, ko)
    bad = torch.zeros((n, h), dtype=torch.bool, device=DEV)
    bad[3, 1] = bad[4, 2] = True
    assert torch.isfinite(qo[~bad]).all() and not torch.isfinite(qo[3, 1]).all() and torch.isnan(qo[4, 2]).any()
    keep = ~bad.cpu().numpy()
    ref = oa.rope(np.where(keep[..., None], host(q), 0), host(pos), fr)
    err = np.abs(host(qo).astype(np.float64) - ref)[keep]
    assert (err <= 2.0 ** -11 * np.abs(ref)[keep] + 2.0 ** -17).all()


# ---- cache ----------------------------------------------------------------

class Cache:
    """A cache whose pages lie in no order, with host copies of all rows."""

    def __init__(self, seqs, hk, d, nb, dt, seed=0, score=False, spare=3, pages=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = pages or seqs * hk * nb + spare
        self.pages = torch.randint(0, 256, (n, 2, 32 * d), generator=g, device=DEV, dtype=torch.uint8)
        self.scales = torch.full((n, 2), float("nan"), device=DEV)
        self.open = torch.full((seqs, hk, 2, 32, d), float("nan"), dtype=dt, device=DEV)
        self.table = torch.randperm(n, generator=g, device=DEV)[:seqs * hk * nb].to(torch.int32).view(seqs, hk, nb)
        self.score = torch.rand((seqs, hk, nb), generator=g, device=DEV) if score else None
        self.seqs, self.hk, self.d, self.nb, self.dt = seqs, hk, d, nb, dt
        self.rows = [np.zeros((2, hk, 0, d)) for _ in range(seqs)]
        self.c = pi.KVCache(self.pages, self.scales, self.open, self.table, self.score)

    def append(self, k, v, new):
        """new[s] rows of k and v [n, hk, d] to sequence s; returns (lens, q_start)."""
        st = np.concatenate(([0], np.cumsum(new)))
        for s in range(self.seqs):
            part = np.stack([host(x[st[s]:st[s + 1]]).astype(np.float64).transpose(1, 0, 2) for x in (k, v)])
            self.rows[s] = np.concatenate((self.rows[s], part), 2)
        lens = torch.tensor([r.shape[2] for r in self.rows], dtype=torch.int32, device=DEV)
        qs = torch.from_numpy(st.astype(np.int32)).to(DEV)
        pi.kv_append(self.c, k, v, lens, q_start=qs, max_new=max(1, max(new)))
        return lens, qs

    def expected(self, s, h, b):
        """(page bytes, scales) of a block from the rows themselves."""
        got = [oa.quantise(self.rows[s][i, h, 32 * b:32 * b + 32]) for i in (0, 1)]
        return oa.to_page(got[0][0], got[1][0]), np.array([got[0][1], got[1][1]])

    def check(self):
        pages, scales, table = host(self.pages), host(self.scales), host(self.table)
        for s in range(self.seqs):
            n = self.rows[s].shape[2]
            for h in range(self.hk):
                for b in range((n + 31) // 32):
                    page, sc = self.expected(s, h, b)
                    at = table[s, h, b]
                    assert np.array_equal(scales[at], sc, equal_nan=True), (s, h, b)
                    assert np.array_equal(pages[at], page), (s, h, b, np.argwhere(pages[at] != page)[:3])

    def values(self, s, h):
        """Keys and values [tokens, d] that the device's pages hold."""
        table, n = host(self.table[s, h]), self.rows[s].shape[2]
        nb = (n + 31) // 32
        at = torch.from_numpy(table[:nb].astype(np.int64)).to(DEV)
        pages, scales = host(self.pages[at]), host(self.scales[at])
        kv = [oa.page_values(pages[b], scales[b], self.d) for b in range(nb)]
        if not kv:
            return np.zeros((0, self.d)), np.zeros((0, self.d))
        return np.concatenate([x[0] for x in kv])[:n], np.concatenate([x[1] for x in kv])[:n]


def _rows(n, hk, d, dt, seed, ties=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kv = torch.randn((n, 2 * hk * d), generator=g, device=DEV)
    if ties:                       # halves of the largest magnitude lie between two codes
        kv = (kv * 4).round().clamp_(-8, 8) / 4
    kv = kv.to(dt)
    return tuple(kv[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in (0, 1))


def _check_read(c, lens, qs, k_rows=None):
    n = int(qs[-1])
    out = [torch.zeros((n, c.hk, c.d), dtype=c.dt, device=DEV) for _ in range(2)]
    pi.kv_read(c.c, lens, out[0], out[1], q_start=qs, max_new=max(1, int((qs[1:] - qs[:-1]).max())))
    st, ln = qs.tolist(), lens.tolist()
    for s in range(c.seqs):
        new = st[s + 1] - st[s]
        for h in range(c.hk):
            for i in (0, 1):
                vals = []
                for b in range((ln[s] + 31) // 32):
                    codes, sc = oa.quantise(c.rows[s][i, h, 32 * b:32 * b + 32])
                    vals.append((codes.astype(np.float32) - 128) * sc)
                ref = np.concatenate(vals)[ln[s] - new:ln[s]] if vals else np.zeros((0, c.d))
                ref = ref.astype(np.float16) if c.dt == f16 else ref
                assert np.array_equal(host(out[i][st[s]:st[s + 1], h]), ref, equal_nan=True), (s, h, i)


@pytest.mark.parametrize("dt", [f16, f32])
@pytest.mark.parametrize("d,hk", [(64, 1), (128, 3)])
@pytest.mark.parametrize("ties", [False, True])
def test_append_and_read(dt, d, hk, ties):
    c = Cache(3, hk, d, 9, dt)
    # prompts, single tokens, a sequence without rows, block ends met and passed
    for i, new in enumerate([(31, 5, 0), (1, 1, 1), (1, 0, 30), (33, 90, 64), (1, 1, 1), (95, 1, 32)]):
        k, v = _rows(sum(new), hk, d, dt, i, ties)
        lens, qs = c.append(k, v, new)
        torch.cuda.synchronize()
        c.check()
        _check_read(c, lens, qs)
        for s in range(3):                                       # the open rows as they came
            n = c.rows[s].shape[2]
            if n % 32:
                ref = c.rows[s][:, :, n - n % 32:].transpose(1, 0, 2, 3)
                assert np.array_equal(host(c.open[s, :, :, :n % 32]).astype(np.float64), ref)


def test_append_extreme_values():
    c = Cache(1, 1, 64, 8, f32)
    k, v = _rows(200, 1, 64, f32, 5)
    k = k.clone()
    k[:32] *= 1e-42                                              # subnormal
    k[32:64] *= 1e37
    k[64:96] = 0
    k[100, 0, 3] = float("inf")
    k[130, 0, 3] = float("nan")
    lens, qs = c.append(k, v, (200,))
    torch.cuda.synchronize()
    c.check()
    _check_read(c, lens, qs)


def test_append_without_q_start_and_head_major_rows():
    c = Cache(2, 4, 64, 4, f16)
    x = torch.randn((2, 4, 2 * 40, 64), device=DEV).to(f16)      # [half, head, token, d]
    k, v = x[0].transpose(0, 1), x[1].transpose(0, 1)
    for s in range(2):
        c.rows[s] = host(x[:, :, 40 * s:40 * s + 40]).astype(np.float64)
    lens = torch.tensor([40, 40], dtype=torch.int32, device=DEV)
    pi.kv_append(c.c, k, v, lens)
    torch.cuda.synchronize()
    c.check()


def test_append_leaves_the_invalid_alone():
    c = Cache(3, 2, 64, 4, f16)
    k, v = _rows(30, 2, 64, f16, 1)
    c.append(k, v, (10, 10, 10))
    torch.cuda.synchronize()
    before = [t.clone() for t in (c.pages, c.scales, c.open)]
    qs = torch.tensor([0, 10, 20, 30], dtype=torch.int32, device=DEV)
    # lens below the rows, negative, beyond the table
    lens = torch.tensor([9, -1, 4 * 32 + 1], dtype=torch.int32, device=DEV)
    pi.kv_append(c.c, k, v, lens, q_start=qs, max_new=10)
    # rows outside [0, n_tok), backwards, more than max_new
    lens = torch.tensor([20, 20, 20], dtype=torch.int32, device=DEV)
    pi.kv_append(c.c, k, v, lens, q_start=torch.tensor([-10, 0, -5, 40], dtype=torch.int32, device=DEV), max_new=10)
    torch.cuda.synchronize()
    now = (c.pages, c.scales, c.open)
    # of the second call only rows [-10, 0) (outside), [0, -5) (backwards), [-5, 40): none is valid
    for a, b in zip(before, now):
        assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))
    out = [torch.zeros((30, 2, 64), dtype=f16, device=DEV) for _ in range(2)]
    pi.kv_read(c.c, torch.tensor([9, -1, 10], dtype=torch.int32, device=DEV), out[0], out[1], q_start=qs, max_new=10)
    assert torch.isnan(out[0][:20]).all() and torch.isnan(out[1][:20]).all() and torch.isfinite(out[0][20:]).all()
    # a bad page is not written, and reads as NaN
    c.table[0, 0, 0], c.table[1, 1, 0] = -1, c.pages.shape[0]
    lens = torch.tensor([10, 10, 10], dtype=torch.int32, device=DEV)
    pi.kv_append(c.c, k, v, lens, q_start=qs, max_new=10)
    pi.kv_read(c.c, lens, out[0], out[1], q_start=qs, max_new=10)
    assert torch.isnan(out[0][:10, 0]).all() and torch.isnan(out[1][10:20, 1]).all()
    assert torch.isfinite(out[0][:10, 1]).all() and torch.isfinite(out[0][20:]).all()


# ---- attention ------------------------------------------------------------

def _attend(c, q, lens, qs, max_q, score=False, ws=None, **kw):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    if ws is None:
        ws = pi.alloc_attend_workspace(c.c, q.shape[1], max_q, kw.get("max_len"), add_score=score)
    pi.attend(c.c, q, lens, out, q_start=qs, max_q=max_q, add_score=score, ws=ws, **kw)
    torch.cuda.synchronize()
    return out, ws


def _check_attend(c, q, out, lens, qs, scale, score0=None, score1=None, seqs=None):
    st, ln = qs.tolist(), lens.tolist()
    group = q.shape[1] // c.hk
    for s in (range(c.seqs) if seqs is None else seqs):
        new = st[s + 1] - st[s]
        for h in range(c.hk):
            k, v = c.values(s, h)
            k, v = k[:ln[s]], v[:ln[s]]
            qq = host(q[st[s]:st[s + 1], h * group:(h + 1) * group]).astype(np.float64).reshape(new * group, c.d)
            sees = np.repeat(ln[s] - new + 1 + np.arange(new), group)
            ref, w, mag, slog = oa.attend(qq, k, v, sees, scale)
            got = host(out[st[s]:st[s + 1], h * group:(h + 1) * group]).astype(np.float64).reshape(new * group, c.d)
            part = 2.0 ** -11 if c.dt == f16 else 2.0 ** -22
            nb = (ln[s] + 31) // 32
            rel = 2.0 ** -20 * slog[:, None] + 2.0 ** -22 * (8 + math.sqrt(nb))
            tol = HALF[c.dt] * np.abs(ref) + (part + rel) * mag + 2.0 ** -25 * (c.dt == f16)
            tol = tol + 2.0 ** -31 * np.abs(v).sum(0)
            err = np.abs(got - ref)
            assert (err <= tol).all(), (s, h, float(np.max(err / np.maximum(tol, 1e-300))))
            if score0 is not None:
                s0, s1 = host(score0[s, h]).astype(np.float64), host(score1[s, h]).astype(np.float64)
                pad = np.zeros((len(w), nb * 32))
                pad[:, :ln[s]] = w
                wb = pad.reshape(len(w), nb, 32).sum(2)
                tol = (wb * rel).sum(0) + 2.0 ** -23 * (s0[:nb] + wb.sum(0)) + 1e-30
                err = np.abs(s1[:nb] - (s0[:nb] + wb.sum(0)))
                assert (err <= tol).all(), (s, h, float(np.max(err / tol)))
                assert np.array_equal(s1[nb:], s0[nb:])


def _filled(seqs, hk, d, dt, lens, seed=0, score=False, slack=2):
    c = Cache(seqs, hk, d, (max(lens) + 31) // 32 + slack, dt, seed, score)
    k, v = _rows(sum(lens), hk, d, dt, seed + 100)
    c.append(k, v, lens)
    c.table[:, :, (max(lens) + 31) // 32:] = -1                  # never read past the length
    return c


CASES = [   # lens (with the call's rows), new rows, kv heads, group
    ((1,), (1,), 1, 1),
    ((33, 32, 1, 0), (1, 1, 1, 0), 2, 3),
    ((131,), (1,), 2, 8),
    ((700, 65), (1, 1), 1, 16),
    ((95, 40), (5, 40), 2, 7),
    ((3000,), (1,), 1, 8),
    ((2500,), (3,), 2, 16),
    ((300, 0, 129), (37, 0, 129), 1, 8),
    ((10, 3), (12, 3), 1, 2),                                    # more rows than tokens: the first see none
]


@pytest.mark.parametrize("dt", [f16, f32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_attend(dt, d, score, case):
    lens, new, hk, group = case
    c = _filled(len(lens), hk, d, dt, lens, score=score)
    n = sum(new)
    q = (torch.randn((n, hk * group, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(n)) * 2).to(dt)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.from_numpy(np.concatenate(([0], np.cumsum(new))).astype(np.int32)).to(DEV)
    s0 = c.score.clone() if score else None
    out, ws = _attend(c, q, ln, qs, max(new), score)
    _check_attend(c, q, out, ln, qs, d ** -0.5, s0, c.score)
    assert pi.read_flags(ws) == 0
    # the same bits again, from a used workspace
    s1 = c.score.clone() if score else None
    if score:
        c.score.copy_(s0)
    again, _ = _attend(c, q, ln, qs, max(new), score, ws)
    assert torch.equal(out, again) and (not score or torch.equal(s1, c.score))


@pytest.mark.parametrize("dt,d,hk,group,new,length", [(f16, 64, 4, 16, 300, 900), (f16, 128, 8, 8, 513, 600),
                                                      (f32, 64, 8, 4, 1100, 1100), (f32, 128, 16, 8, 130, 150)])
@pytest.mark.parametrize("score", [False, True])
def test_attend_prompt(dt, d, hk, group, new, length, score):
    """Enough rows that each wave has its own."""
    c = _filled(1, hk, d, dt, (length,), score=score)
    q = (torch.randn((new, hk * group, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)) * 2).to(dt)
    ln = torch.tensor([length], dtype=torch.int32, device=DEV)
    qs = torch.tensor([0, new], dtype=torch.int32, device=DEV)
    s0 = c.score.clone() if score else None
    out, _ = _attend(c, q, ln, qs, new, score)
    _check_attend(c, q, out, ln, qs, d ** -0.5, s0, c.score)


def _mixed(seqs, *long):
    """Long sequences among short ones, some of them empty."""
    lens = [(13 * i) % 150 if i % 5 else 0 for i in range(seqs)]
    for i, n in enumerate(long):
        lens[(7 * i + 3) % seqs] = n
    return tuple(lens)


SHARED = [  # lens, kv heads, group: few rows and more than 32 blocks to a split of the longest
    (_mixed(40, 4000, 2500), 2, 8),
    (_mixed(64, 4500), 1, 1),
    (_mixed(64, 2500, 2100, 1000), 2, 4),
    ((13000, 40, 9000), 7, 3),
    ((33000, 32999), 1, 3),
    ((0, 33000, 0), 1, 2),
    (_mixed(20, 9000, 5000, 700), 8, 2),                         # more pairs than splits: the long alone are split
    (_mixed(64, 9000, 2000), 6, 1),
]


@pytest.mark.parametrize("dt,d", [(f16, 128), (f16, 64), (f32, 64), (f32, 128)])
@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("case", SHARED, ids=[str(i) for i in range(len(SHARED))])
def test_attend_sequences_of_unlike_lengths(dt, d, score, case):
    """Sequences that share the workgroups by their lengths, some without rows, one invalid."""
    lens, hk, group = case
    c = _filled(len(lens), hk, d, dt, lens, score=score)
    new = [0 if i % 11 == 8 else (2 if n > 1 and i % 3 == 1 and group <= 8 else 1) for i, n in enumerate(lens)]
    n = sum(new)
    q = (torch.randn((n, hk * group, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(n)) * 2).to(dt)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.from_numpy(np.concatenate(([0], np.cumsum(new))).astype(np.int32)).to(DEV)
    s0 = c.score.clone() if score else None
    out, ws = _attend(c, q, ln, qs, max(new), score)
    s1 = c.score.clone() if score else None
    _check_attend(c, q, out, ln, qs, d ** -0.5, s0, s1, [s for s in range(len(lens)) if new[s]])
    assert pi.read_flags(ws) == 0
    if score:
        c.score.copy_(s0)
    ws[256:].fill_(255)                                          # a used workspace holds anything
    again, _ = _attend(c, q, ln, qs, max(new), score, ws)
    assert torch.equal(out, again) and (not score or torch.equal(s1, c.score))
    # the last sequence invalid: NaN in its rows, the others as they are
    if score:
        c.score.copy_(s0)
    ln[-1] = -1
    bad, _ = _attend(c, q, ln, qs, max(new), score, ws)
    assert pi.read_flags(ws) == L.PI_FLAG_KV_RANGE
    at = int(qs[-2])
    assert torch.isnan(bad[at:]).all()
    rest = [s for s in range(len(lens) - 1) if new[s]]
    _check_attend(c, q, bad, ln, qs, d ** -0.5, s0, c.score, rest)
    if score:
        assert torch.equal(c.score[-1], s0[-1])


@pytest.mark.parametrize("dt,d", [(f16, 128), (f16, 64), (f32, 64)])
@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("new,group", [(3, 7), (4, 8), (5, 8), (8, 8), (13, 5), (16, 8), (17, 8), (200, 2)])
def test_attend_a_few_tokens_over_long_contexts(dt, d, score, new, group):
    """Rows between one token's and a prompt's, ragged, one sequence with fewer of them than the others."""
    _few_tokens((2200, 2111, 700, 90), dt, d, score, new, group)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("new,group", [(3, 7), (5, 8), (13, 5)])
def test_attend_a_few_tokens_of_many_sequences(d, score, new, group):
    _few_tokens((900, 30, 880, 33, 64, 500, 1, 871, 95), f32, d, score, new, group)


@pytest.mark.parametrize("dt,d", [(f16, 64), (f16, 128), (f32, 64)])
def test_attend_prompts_of_many_sequences(dt, d):
    """More workgroups than run at once; whole prompts, and one that goes on from 50 tokens."""
    _few_tokens((350, 333, 400, 1, 350, 32, 347, 350, 350, 100, 350, 350), dt, d, False, 350, 4)


def _few_tokens(lens, dt, d, score, new, group):
    hk = 8
    c = _filled(len(lens), hk, d, dt, lens, score=score)
    rows = [min(new, x) for x in lens]
    rows[2] = 1
    n = sum(rows)
    q = (torch.randn((n, hk * group, d), device=DEV, generator=torch.Generator(device=DEV).manual_seed(n)) * 2).to(dt)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.from_numpy(np.concatenate(([0], np.cumsum(rows))).astype(np.int32)).to(DEV)
    s0 = c.score.clone() if score else None
    out, ws = _attend(c, q, ln, qs, new, score)
    _check_attend(c, q, out, ln, qs, d ** -0.5, s0, c.score)
    assert pi.read_flags(ws) == 0
    s1 = c.score.clone() if score else None
    if score:
        c.score.copy_(s0)
    again, _ = _attend(c, q, ln, qs, new, score, ws)
    assert torch.equal(out, again) and (not score or torch.equal(s1, c.score))


@pytest.mark.parametrize("dt", [f16, f32])
def test_attend_strided_rows_and_scale(dt):
    lens, hk, group, d = (200, 77), 2, 4, 64
    c = _filled(2, hk, d, dt, lens)
    big = torch.randn((5, (hk * group + 4) * d), device=DEV).to(dt)
    q = big[:, 2 * d:(2 + hk * group) * d].unflatten(1, (hk * group, d))
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.tensor([0, 4, 5], dtype=torch.int32, device=DEV)
    ref, _ = _attend(c, q, ln, qs, 4, scale=0.3)
    _check_attend(c, q, ref, ln, qs, 0.3)
    wide = torch.full((hk * group, 5, d), 7.0, dtype=dt, device=DEV)      # head-major output
    pi.attend(c.c, q, ln, wide.transpose(0, 1), q_start=qs, max_q=4, scale=0.3)
    assert torch.equal(wide.transpose(0, 1), ref)
    flat, _ = _attend(c, q, ln, qs, 4, scale=0.0)                # scale 0: the mean of what is seen
    _check_attend(c, q, flat, ln, qs, 0.0)


@pytest.mark.parametrize("dt", [f16, f32])
def test_attend_logits_far_apart_and_large_scales(dt):
    """Blocks whose scales differ by 2^40, logits in the hundreds that rise along the row."""
    lens, d = (40 * 32,), 64
    c = Cache(1, 1, d, 40, dt)
    k, v = _rows(lens[0], 1, d, dt, 9)
    c.append(k, v, lens)
    torch.cuda.synchronize()
    at = c.table[0, 0].long()
    c.scales[at, 0] *= torch.linspace(0.1, 20, 40, device=DEV)
    c.scales[at, 1] *= torch.exp2(torch.linspace(-20, 20 if dt == f32 else 8, 40, device=DEV))
    c.scales[at[7]] = 0
    q = torch.randn((1, 1, d), device=DEV).to(dt)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    out, _ = _attend(c, q, ln, qs, 1)
    _check_attend(c, q, out, ln, qs, d ** -0.5)


@pytest.mark.parametrize("new", [1, 40])
def test_attend_values_that_are_no_numbers(new):
    """A block with a NaN makes NaN of the rows that see a token of it, and of no others."""
    lens, hk, d = (160, 96), 2, 64
    c = Cache(2, hk, d, 8, f16)
    k, v = _rows(sum(lens), hk, d, f16, 2)
    v = v.clone()
    v[150, 1, 5] = float("inf")                                  # sequence 0, head 1, block 4 (tokens 128..159)
    c.append(k, v, lens)
    q = torch.randn((2 * new, 4, d), device=DEV).to(f16)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.tensor([0, new, 2 * new], dtype=torch.int32, device=DEV)
    out, ws = _attend(c, q, ln, qs, new)
    assert pi.read_flags(ws) == 0
    nan = torch.isnan(out)
    sees = 160 - new + 1 + torch.arange(new, device=DEV)
    hit = sees > 128
    assert nan[:new][hit][:, 2:].all() and not nan[:new][~hit].any()
    assert not nan[:new, :2].any() and not nan[new:].any()


def test_attend_bad_pages_and_invalid_sequences():
    lens, hk, d = (100, 100, 100), 2, 64
    c = _filled(3, hk, d, f16, lens, score=True)
    q = torch.randn((3, 4, d), device=DEV).to(f16)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.arange(4, dtype=torch.int32, device=DEV)
    good, ws = _attend(c, q, ln, qs, 1)
    c.table[0, 1, 2], c.table[1, 0, 0] = -7, 1 << 30
    out, ws = _attend(c, q, ln, qs, 1, ws=ws)
    assert pi.read_flags(ws) == L.PI_FLAG_KV_RANGE
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(out[1, :2]).all()
    assert torch.equal(out[0, :2], good[0, :2]) and torch.equal(out[1, 2:], good[1, 2:]) and torch.equal(out[2], good[2])
    # invalid: beyond max_len, negative, more rows than max_q; their score stays
    pi.clear_flags(ws)
    s0 = c.score.clone()
    bad = torch.tensor([129, -3, 100], dtype=torch.int32, device=DEV)
    out, ws = _attend(c, q, bad, qs, 1, True, max_len=128)
    assert pi.read_flags(ws) == L.PI_FLAG_KV_RANGE
    assert torch.isnan(out[:2]).all() and torch.equal(out[2], good[2])
    assert torch.equal(c.score[:2], s0[:2]) and not torch.equal(c.score[2], s0[2])
    out, ws = _attend(c, q, ln, torch.tensor([0, 2, 2, 9], dtype=torch.int32, device=DEV), 1)
    assert torch.isnan(out).all()


def test_attend_far_pages():
    """Pages beyond 4 GiB of the cache."""
    d, n_pages = 128, 600_000
    c = Cache(1, 2, d, 70, f16, score=True, pages=n_pages)
    far = torch.arange(140, dtype=torch.int32, device=DEV).view(1, 2, 70) * 4000 + 40_000
    assert int(far.max()) * 64 * d > 1 << 32
    c.table.copy_(far)
    lens = (70 * 32 - 3,)
    k, v = _rows(lens[0], 2, d, f16, 1)
    ln, qs = c.append(k, v, lens)
    _check_read(c, ln, qs)
    q = torch.randn((1, 16, d), device=DEV).to(f16)
    qs = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    s0 = c.score.clone()
    out, _ = _attend(c, q, ln, qs, 1, True)
    _check_attend(c, q, out, ln, qs, d ** -0.5, s0, c.score)


def test_attend_streams_and_graph():
    """On a stream of its own, and replayed from a graph with eager calls between."""
    lens, hk, d = (900, 333), 2, 128
    c = _filled(2, hk, d, f16, lens, score=True)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    xs = [torch.randn((2, 16, d), device=DEV).to(f16) for _ in range(3)]
    refs, scores = [], []
    zero = torch.zeros_like(c.score)
    for x in xs:
        c.score.copy_(zero)
        out, ws = _attend(c, x, ln, qs, 1, True)
        refs.append(out), scores.append(c.score.clone())
    stage, out = xs[0].clone(), torch.empty_like(xs[0])
    stream = torch.cuda.Stream()
    c.score.copy_(zero)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        pi.attend(c.c, stage, ln, out, q_start=qs, max_q=1, add_score=True, ws=ws)
    stream.synchronize()
    assert torch.equal(out, refs[0]) and torch.equal(c.score, scores[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pi.attend(c.c, stage, ln, out, q_start=qs, max_q=1, add_score=True, ws=ws)
    for rep in range(6):
        stage.copy_(xs[rep % 3])
        c.score.copy_(zero)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, refs[rep % 3]) and torch.equal(c.score, scores[rep % 3])
        eager, _ = _attend(c, xs[(rep + 1) % 3], ln, qs, 1, True, ws)
        assert torch.equal(eager, refs[(rep + 1) % 3])


def test_attend_huge_logits():
    """fp32 logits far below -1e30 are logits still.  (One block: between blocks
    the weights hold to half a step of the logits, which is 1e26 here.)"""
    d = 64
    c = Cache(1, 1, d, 3, f32)
    k, v = _rows(30, 1, d, f32, 4)
    c.append(torch.ones_like(k), v, (30,))                       # every key the same: equal weights
    q = torch.full((1, 1, d), -1e33, device=DEV)
    ln = torch.tensor([30], dtype=torch.int32, device=DEV)
    out, _ = _attend(c, q, ln, torch.tensor([0, 1], dtype=torch.int32, device=DEV), 1)
    _, vals = c.values(0, 0)
    assert np.abs(host(out)[0, 0] - vals.mean(0)).max() <= 2.0 ** -18 * np.abs(vals).max()


@pytest.mark.parametrize("how", ["object", "handle"])
def test_a_step_on_a_stream_of_its_own_and_in_a_graph(how):
    """Rotation, append, attention, eviction, in a row, on the stream that is
    given; then replayed from a graph with eager steps between, each replay
    against the eager step from the same state."""
    seqs, hk, group, d, keep, recent = 2, 2, 4, 64, 3, 1
    c = Cache(seqs, hk, d, 8, f16, score=True)
    k, v = _rows(150, hk, d, f16, 1)
    lens, _ = c.append(k, v, (90, 60))
    c.scales.nan_to_num_(nan=1.0)                                # spare pages: no NaN to compare
    c.open.nan_to_num_(nan=0.0)
    r = pi.Rope(torch.from_numpy(_freqs(d)).to(DEV), d)
    qkv = torch.empty((seqs, (group * hk + 2 * hk) * d), dtype=f16, device=DEV)
    q, kk, vv = (t.unflatten(1, (-1, d)) for t in qkv.split((group * hk * d, hk * d, hk * d), 1))
    pos = torch.tensor([90, 60], dtype=torch.int32, device=DEV)
    qs = torch.arange(seqs + 1, dtype=torch.int32, device=DEV)
    out = torch.zeros((seqs, group * hk, d), dtype=f16, device=DEV)
    held = torch.zeros_like(lens)
    now = lens + 1
    ws = pi.alloc_attend_workspace(c.c, group * hk, 1, add_score=True)
    xs = [torch.randn(qkv.shape, device=DEV).to(f16) for _ in range(3)]
    state = (c.pages, c.scales, c.open, c.table, c.score)
    first = [t.clone() for t in state]
    torch.cuda.synchronize()

    def step(s):
        pi.qk_rope(r, q, kk, pos, stream=s)
        pi.kv_append(c.c, kk, vv, now, q_start=qs, max_new=1, stream=s)
        pi.attend(c.c, q, now, out, q_start=qs, max_q=1, add_score=True, ws=ws, stream=s)
        pi.kv_evict(c.table, c.score, now, keep, recent, held, stream=s)

    def reset(i):
        for t, f in zip(state, first):
            t.copy_(f)
        qkv.copy_(xs[i])
        out.zero_(), held.zero_()
        torch.cuda.synchronize()

    def seen():
        torch.cuda.synchronize()
        return [t.clone() for t in (*state, qkv, out, held)]

    stream = torch.cuda.Stream()
    given = stream if how == "object" else stream.cuda_stream
    want = []
    for i in range(3):
        reset(i)
        step(None)
        want.append(seen())
        reset(i)
        step(given)
        assert all(torch.equal(a, b) for a, b in zip(seen(), want[i])), i
    reset(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(None)
    for rep in range(6):
        reset(rep % 3)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(seen(), want[rep % 3])), rep
        reset((rep + 1) % 3)
        step(None)
        assert all(torch.equal(a, b) for a, b in zip(seen(), want[(rep + 1) % 3])), rep
    assert pi.read_flags(ws) == 0


# ---- eviction -------------------------------------------------------------

@pytest.mark.parametrize("seqs,hk,n,keep,recent", [(1, 1, 1, 1, 1), (3, 2, 130, 96, 8), (2, 3, 1024, 40, 40), (2, 1, 4099, 2048, 32),
                                                   (1, 2, 9000, 8999, 1), (1, 1, 20000, 9000, 100)])
@pytest.mark.parametrize("kind", ["tail", "ties", "odd"])
def test_evict(seqs, hk, n, keep, recent, kind):
    g = torch.Generator(device=DEV).manual_seed(n)
    shape = (seqs, hk, n)
    table = torch.randperm(seqs * hk * n, generator=g, device=DEV).to(torch.int32).view(shape)
    if kind == "ties":
        score = torch.randint(0, 3, shape, generator=g, device=DEV).float()
    else:
        score = torch.exp(torch.randn(shape, generator=g, device=DEV) * 2)
    if kind == "odd":
        r = torch.rand(shape, generator=g, device=DEV)
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1.5, 1e-42)):
            score[(r > 0.1 * i) & (r < 0.1 * i + 0.05)] = x
    lens = torch.tensor([n * 32 - 5, 17, 0, 40 * 32][:seqs], dtype=torch.int32, device=DEV)
    want = [[oa.evict(host(table[s, h]), host(score[s, h]), int(lens[s]), keep, recent) for h in range(hk)]
            for s in range(seqs)]
    out = (torch.empty_like(table), torch.empty_like(score), torch.empty_like(lens))

    def check(t, sc, ln):
        torch.cuda.synchronize()
        for s in range(seqs):
            for h in range(hk):
                wt, ws, wl = want[s][h]
                assert np.array_equal(host(t[s, h]), wt), (s, h)
                assert np.array_equal(host(sc[s, h]), ws, equal_nan=True), (s, h)
                assert int(ln[s]) == wl

    pi.kv_evict(table, score, lens, keep, recent, out[2], out[0], out[1])
    check(*out)
    if n <= L.PI_KV_EVICT_IN_PLACE:
        pi.kv_evict(table, score, lens, keep, recent, out[2])
        check(table, score, out[2])
    else:
        with pytest.raises(pi.PiError):
            pi.kv_evict(table, score, lens, keep, recent, out[2])


def test_evict_then_attend():
    """A decode loop: append, attend with scores, evict; the cache stays whole."""
    hk, group, d, keep, recent = 2, 4, 64, 6, 2
    c = _filled(2, hk, d, f16, (310, 120), score=True, slack=4)
    # the table's spare slots name pages of their own again
    used = set(c.table[c.table >= 0].tolist())
    free = torch.tensor([p for p in range(c.pages.shape[0]) if p not in used], dtype=torch.int32, device=DEV)
    c.table[c.table < 0] = free[:int((c.table < 0).sum())]
    ln = torch.tensor([310, 120], dtype=torch.int32, device=DEV)
    qs = torch.arange(3, dtype=torch.int32, device=DEV)
    nxt = torch.empty_like(ln)
    for step in range(70):
        pi.kv_evict(c.table, c.score, ln, keep, recent, nxt)
        ln = nxt + 1
        k, v = _rows(2, hk, d, f16, 1000 + step)
        pi.kv_append(c.c, k, v, ln, q_start=qs, max_new=1)
        q = torch.randn((2, hk * group, d), device=DEV).to(f16)
        out, ws = _attend(c, q, ln, qs, 1, True)
        assert pi.read_flags(ws) == 0 and torch.isfinite(out).all()
        kk, vv = torch.empty((2, hk, d), dtype=f16, device=DEV), torch.empty((2, hk, d), dtype=f16, device=DEV)
        pi.kv_read(c.c, ln, kk, vv, q_start=qs, max_new=1)
        assert (kk - k).abs().max() < 0.05 and (vv - v).abs().max() < 0.05
    assert ln.max() <= keep * 32 + 1
    assert sorted(c.table.flatten().tolist()) == sorted(set(c.table.flatten().tolist()))
