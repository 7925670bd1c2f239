"""The attention oracle against hand-worked numbers and scalar loops (CPU)."""

import math

import numpy as np
import pytest

from oracle import attention as oa


def test_rope_quarter_turn():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0, 8.0]]])
    # a quarter turn per position: (a, b) -> (-b, a)
    half = oa.rope(x, [1], [0.25, 0.25], "half")
    assert np.allclose(half[0, 0], [-3, -4, 1, 2, 5, 6, 7, 8])
    inter = oa.rope(x, [1], [0.25, 0.25], "interleaved", scale=2.0)
    assert np.allclose(inter[0, 0], [-4, 2, -8, 6, 5, 6, 7, 8])
    assert np.allclose(oa.rope(x, [4], [0.25], "half"), x)


def test_rope_norm():
    x = np.array([[[3.0, 4.0, 0, 0, 0, 0, 0, 0]]])
    y = oa.rope(x, [0], [0.1], norm=np.full(8, 2.0), eps=0.0)
    assert np.allclose(y[0, 0, :2], np.array([3, 4]) * 2 / math.sqrt(25 / 8))


def test_quantise():
    codes, scale = oa.quantise(np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5]]))
    assert scale == np.float32(1.0)
    assert codes[0].tolist() == [255, 1, 128, 130, 130, 128]      # ties to even
    assert (codes[1:] == 128).all()
    codes, scale = oa.quantise(np.zeros((3, 4)))
    assert scale == 0 and (codes == 128).all()
    assert np.isnan(oa.quantise(np.array([[np.inf, 1.0]]))[1])


@pytest.mark.parametrize("d", [64, 128])
def test_page_order_is_a_permutation(d):
    t, e = np.arange(32)[:, None], np.arange(d)[None]
    for f in (oa.key_offset, oa.value_offset):
        assert sorted(f(t, e, d).ravel().tolist()) == list(range(32 * d))
    rng = np.random.default_rng(d)
    k, v = rng.integers(0, 256, (2, 32, d)).astype(np.uint8)
    kk, vv = oa.page_values(oa.to_page(k, v), (1.0, 2.0), d)
    assert (kk == k.astype(float) - 128).all() and (vv == 2 * (v.astype(float) - 128)).all()


def test_attend_scalar_loop():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 4)), rng.normal(size=(6, 4)), rng.normal(size=(6, 4))
    out, w, _, _ = oa.attend(q, k, v, [0, 2, 6], 0.5)
    assert (out[0] == 0).all() and (w[0] == 0).all()
    for i, n in ((1, 2), (2, 6)):
        e = [math.exp(0.5 * sum(q[i][x] * k[j][x] for x in range(4))) for j in range(n)]
        for x in range(4):
            assert math.isclose(out[i][x], sum(e[j] * v[j][x] for j in range(n)) / sum(e), rel_tol=1e-12)


def test_evict_worked():
    t, s, n = oa.evict([10, 11, 12, 13, 14, 15], [5, 1, 1, 9, 0, 7], 5 * 32 - 3, keep=3, recent=1)
    # blocks 0..4 held, 4 recent; of 0..3 the heaviest two are 3 and 0
    assert t.tolist() == [10, 13, 14, 11, 12, 15] and s.tolist() == [5, 9, 0, 0, 0, 7] and n == 3 * 32 - 3
