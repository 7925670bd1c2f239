"""fp32 rows over long contexts: the sum of thousands of like weights.  Eight
tokens take the row; the others' weights are 2^-13 of theirs and their values
0, so the output is the heavy tokens' value times their share of the sum, and
off by what the sum is off.

Tolerance: additions of like terms do not average their roundings, 2^-24 each,
so a chain of n is off by up to n 2^-24; 64 blocks to a chain and n / 64 chains
for n blocks, beside the terms of test_gpu_attention."""

import pytest
import torch

from attention_helpers import Tail, f32
from helpers import host, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("d,new,heads", [(64, 1, 4), (128, 1, 4), (64, 5, 8), (128, 3, 8), (128, 5, 8), (64, 20, 8)])
def test_a_sum_of_like_weights(d, new, heads):
    call = Tail(f32, d, new, heads, bits=13.3)
    c = call.c
    e = torch.arange(d, device=c.pages.device)
    c.pages[:, 1] = 128
    c.pages[call.at[:8, None], 1, (e // 32 * 1024 + e % 16 * 16 + e // 16 % 2 * 8)[None]] = 192
    call.run()
    nb = call.tokens // 32
    for i in range(new):
        tail = (call.tokens - new + 1 + i - 8) * 2.0 ** -13.3
        ref = 64 * 8 / (8 + tail)
        err = abs(host(call.out[i]).astype(float) - ref).max() / ref
        # the logit: 13.3 ln 2, fp32 to 2^-20 of its size
        assert err <= 2.0 ** -20 * 13.3 * 0.7 + 2.0 ** -22 * 8 + 2.0 ** -24 * (64 + nb / 64), (i, err)
