"""CPU checks of the attention side's C ABI: bad arguments are rejected before
anything is launched.  No call here reaches a kernel launch."""

import ctypes

import pytest
import torch

from activation_sparse_rank_amd import _lib as L

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="fake-pointer validation tests run only on hosts without a GPU")

A, B, C, D = 0x100000, 0x10000000, 0x20000000, 0x30000000      # never dereferenced
ODD = 0x100004
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _rope(d=128, rot=128, layout=L.PI_ROPE_HALF, scale=1.0, eps=1e-6, freqs=A, qn=None, kn=None):
    return L.PiRope(d, rot, layout, scale, eps, freqs, qn, kn)


def test_rope_rejects(lib):
    def call(r=None, q=A, qt=1024, qh=128, h=8, k=B, kt=256, kh=128, hk=2, pos=A, n=4, dt=L.PI_F16, qo=C, ko=D,
             kot=256):
        r = _rope() if r is None else r
        return lib.pi_qk_rope(ctypes.byref(r), q, qt, qh, h, k, kt, kh, hk, pos, n, dt, qo, 1024, 128, ko, kot, 128,
                              None)

    assert lib.pi_qk_rope(None, A, 1024, 128, 8, B, 256, 128, 2, A, 4, L.PI_F16, C, 1024, 128, D, 256, 128,
                          None) == L.PI_E_NULL
    assert call(pos=None) == L.PI_E_NULL
    assert call(q=None) == L.PI_E_NULL
    assert call(ko=None) == L.PI_E_NULL
    assert call(_rope(freqs=None)) == L.PI_E_NULL
    assert call(dt=L.PI_Q4_0) == L.PI_E_DTYPE
    assert call(_rope(layout=2)) == L.PI_E_DTYPE
    for bad in (dict(d=12), dict(d=264), dict(rot=0), dict(rot=3), dict(rot=130)):
        assert call(_rope(**bad)) == L.PI_E_SHAPE, bad
    for bad in (dict(n=0), dict(h=-1), dict(h=0, hk=0), dict(qt=1020), dict(qh=64), dict(kt=100), dict(qt=512)):
        assert call(**bad) == L.PI_E_SHAPE, bad
    for bad in (dict(scale=NAN), dict(scale=INF), dict(eps=-1.0), dict(eps=NAN)):
        assert call(_rope(**bad)) == L.PI_E_RANGE, bad
    for bad in (dict(q=ODD), dict(ko=D + 8), dict(pos=A + 2)):
        assert call(**bad) == L.PI_E_ALIGN, bad
    assert call(_rope(freqs=A + 4)) == L.PI_E_ALIGN
    assert call(qo=A + 16) == L.PI_E_RANGE                      # overlaps q
    assert call(qo=A, qt=2048) == L.PI_E_RANGE                  # in place with another stride
    assert call(ko=A) == L.PI_E_RANGE                           # k's output over q
    assert call(ko=C) == L.PI_E_RANGE                           # both outputs in one place


def _cache(s=2, h=4, d=128, nb=16, pages=64, dt=L.PI_F16, p=A, sc=B, op=C, tb=D, score=None):
    return L.PiKVCache(s, h, d, nb, pages, dt, p, sc, op, tb, score)


BAD_CACHES = [(dict(dt=L.PI_Q4_0), L.PI_E_DTYPE), (dict(d=96), L.PI_E_SHAPE), (dict(s=0), L.PI_E_SHAPE),
              (dict(h=0), L.PI_E_SHAPE), (dict(nb=0), L.PI_E_SHAPE), (dict(nb=(1 << 24) + 1), L.PI_E_SHAPE),
              (dict(pages=0), L.PI_E_SHAPE), (dict(s=1 << 20, h=1 << 20), L.PI_E_SHAPE), (dict(p=None), L.PI_E_NULL),
              (dict(sc=None), L.PI_E_NULL), (dict(op=None), L.PI_E_NULL), (dict(tb=None), L.PI_E_NULL),
              (dict(p=ODD), L.PI_E_ALIGN), (dict(score=ODD), L.PI_E_ALIGN)]


def test_append_and_read_reject(lib):
    def append(c=None, k=A, kt=512, kh=128, v=B, n=4, lens=A, qs=A, mx=4):
        c = _cache() if c is None else c
        return lib.pi_kv_append(ctypes.byref(c), k, kt, kh, v, 512, 128, n, lens, qs, mx, None)

    def read(c=None, k=A, kt=512, kh=128, v=B, n=4, lens=A, qs=A, mx=4):
        c = _cache() if c is None else c
        return lib.pi_kv_read(ctypes.byref(c), lens, qs, mx, k, kt, kh, v, 512, 128, n, None)

    for call in (append, read):
        for bad, st in BAD_CACHES:
            assert call(_cache(**bad)) == st, bad
        for bad in (dict(k=None), dict(v=None), dict(lens=None)):
            assert call(**bad) == L.PI_E_NULL, bad
        for bad in (dict(n=0), dict(mx=0), dict(mx=16 * 32 + 1), dict(kt=511), dict(kh=100), dict(kt=256),
                    dict(qs=None, mx=3)):
            assert call(**bad) == L.PI_E_SHAPE, bad
        for bad in (dict(k=ODD), dict(lens=A + 1), dict(qs=A + 2)):
            assert call(**bad) == L.PI_E_ALIGN, bad
    assert lib.pi_kv_append(None, A, 512, 128, B, 512, 128, 4, A, A, 4, None) == L.PI_E_NULL


def test_attend_rejects(lib):
    def call(c=None, q=A, qt=2048, qh=128, h=16, n=4, lens=A, qs=A, mq=2, ml=512, scale=0.1, score=0, o=B, w=C,
             wsb=1 << 40):
        c = _cache() if c is None else c
        return lib.pi_attend(ctypes.byref(c), q, qt, qh, h, n, lens, qs, mq, ml, scale, score, o, 2048, 128, w, wsb,
                             None)

    for bad, st in BAD_CACHES:
        assert call(_cache(**bad)) == st, bad
    for bad in (dict(q=None), dict(o=None), dict(lens=None), dict(score=1)):
        assert call(**bad) == L.PI_E_NULL, bad
    for bad in (dict(h=0), dict(h=10), dict(n=0), dict(mq=0), dict(qt=100), dict(qh=64), dict(qs=None, mq=3)):
        assert call(**bad) == L.PI_E_SHAPE, bad
    for bad in (dict(ml=0), dict(ml=513), dict(scale=NAN), dict(scale=INF), dict(scale=-1.0), dict(o=A + 256)):
        assert call(**bad) == L.PI_E_RANGE, bad
    for bad in (dict(q=ODD), dict(o=B + 8), dict(lens=A + 2), dict(w=ODD)):
        assert call(**bad) == L.PI_E_ALIGN, bad
    assert call(w=None) == L.PI_E_WORKSPACE
    assert call(wsb=100) == L.PI_E_WORKSPACE


def test_attend_workspace(lib):
    def size(c=None, h=16, mq=1, ml=512, score=0):
        c = _cache() if c is None else c
        return lib.pi_attend_workspace_bytes(ctypes.byref(c), h, mq, ml, score)

    assert size() >= L.PI_WS_HEADER_BYTES
    assert size(score=1) >= size() + 2 * 16 * 16 * 4
    assert size(h=10) == size(mq=0) == size(ml=0) == size(ml=513) == size(_cache(d=96)) == 0
    big = _cache(s=1, nb=1 << 15)
    assert size(big, ml=1 << 20) > size(big, ml=512)


def test_evict_rejects(lib):
    def call(t=A, sc=B, lens=C, s=2, h=4, nb=16, keep=4, recent=1, to=D, so=D + (1 << 20), lo=C + 64):
        return lib.pi_kv_evict(t, sc, lens, s, h, nb, keep, recent, to, so, lo, None)

    for name in ("t", "sc", "lens", "to", "so", "lo"):
        assert call(**{name: None}) == L.PI_E_NULL, name
        assert call(**{name: A + 2}) == L.PI_E_ALIGN, name
    for bad in (dict(s=0), dict(h=0), dict(nb=0), dict(nb=(1 << 24) + 1)):
        assert call(**bad) == L.PI_E_SHAPE, bad
    for bad in (dict(recent=0), dict(recent=5), dict(keep=0), dict(to=A), dict(so=B + 4), dict(lo=C), dict(to=A + 16),
                dict(so=D), dict(lo=A), dict(t=A, to=A, so=B, nb=16385)):
        assert call(**bad) == L.PI_E_RANGE, bad
