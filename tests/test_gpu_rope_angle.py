"""The cosines and sines that pi_qk_rope multiplies by: a pair (1, 0) becomes
(cos, sin), so fp32 outputs show them whole.

Tolerance: cosine and sine of an fp32 angle to 4 units in the last place (2^-21),
as much again for what fp32 leaves of the angle, and its square's share, 2^-44.
An angle rounded to fp32 is off by up to 2^-26 of a turn, 9e-8, which is far more
wherever the cosine or the sine is small."""

import numpy as np
import pytest
import torch

import activation_sparse_rank_amd as pi
from helpers import host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [0, 100000, (1 << 31) - 5000])
def test_angles(first):
    require_gpu()
    d, n = 128, 4096
    g = np.random.default_rng(first)
    freqs = np.concatenate((10000.0 ** (-np.arange(32) / 32) / (2 * np.pi), 0.25 + g.uniform(-1e-6, 1e-6, 16), 0.5 + g.uniform(-1e-6, 1e-6, 16)))
    pos = first + np.arange(n)
    x = torch.zeros((n, 1, d), device="cuda")
    x[:, :, :d // 2] = 1.0
    k = x.clone()
    r = pi.Rope(torch.from_numpy(freqs).cuda(), d)
    pi.qk_rope(r, x, k, torch.from_numpy(pos.astype(np.int32)).cuda())
    # turns exactly: the product of two doubles, in two parts
    hi = np.float64(np.float32(freqs))
    turns = (pos[:, None] * hi) % 1.0 + (pos[:, None] * (freqs - hi)) % 1.0
    turns -= np.rint(turns)
    eighth = np.rint(turns * 4)                                  # sines of small angles keep their bits
    small = 2 * np.pi * (turns - eighth / 4)
    c, s = np.cos(small), np.sin(small)
    q = eighth.astype(int) % 4
    ref = np.concatenate((np.choose(q, (c, -s, -c, s)), np.choose(q, (s, c, -s, -c))), 1)
    err = np.abs(host(x)[:, 0].astype(np.float64) - ref)
    # the angle itself: a product in 64 bits (2^-53 of up to 2^30 turns) and its reduction
    angle = 2 * np.pi * 2.0 ** -52 * np.abs(pos[:, None] * freqs)
    tol = 2.0 ** -20 * np.abs(ref) + 2.0 ** -44 + np.concatenate((angle, angle), 1)
    assert (err <= tol).all(), float((err / tol).max())
