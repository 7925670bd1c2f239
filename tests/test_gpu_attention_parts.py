"""Where fp16 rows' weights are held to 2^-22 (two fp16 parts): rows that see at
most 512 tokens, and calls of at most 32 rows to a kv head, whatever bounds the
call is given.  Values lie in pairs of v and -v with nearly equal weights, so
the output is small beside what is summed and a single fp16 part's rounding
(2^-12 of a weight) shows."""

import numpy as np
import pytest
import torch

from attention_helpers import Call, f16
from helpers import require_gpu
from test_gpu_attention import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


PARTS = {
    "prompt": (f16, 64, (300, 129), 60, 1, 8),
    "prompt, wide": (f16, 128, (500,), 60, 2, 8),
    "whole prompt": (f16, 64, (512,), 512, 2, 2),
    "whole prompt, wide": (f16, 128, (512, 100), 512, 2, 2),
    "prompts, many": (f16, 64, (500, 340, 350, 333, 64), 300, 8, 16),
    "prompts, waves": (f16, 128, (500,) * 2 + (60,) * 6, 5, 8, 8),
    "two tiles, wide": (f16, 128, (700, 90), 3, 2, 8),
    "two tiles, wide, split": (f16, 128, (3000,), 4, 1, 8),
    "one tile": (f16, 64, (700, 90), 1, 2, 8),
}


def _pairs(call):
    """Each odd token's values are those of the token before it, negated; keys small, so that weights are nearly equal."""
    c = call.c
    rows = [r.copy() for r in c.rows]
    for r in rows:
        n = r.shape[2]
        r[1][:, 1::2] = -r[1][:, :n - n % 2:2]
        r[0] *= 0.1
    k, v = (torch.from_numpy(np.concatenate([r[i].transpose(1, 0, 2) for r in rows])).to(DEV).to(call.dt) for i in (0, 1))
    c.rows = [np.zeros((2, call.hk, 0, call.d)) for _ in rows]
    table = c.table.clone()
    c.append(k, v, list(call.lens))
    assert torch.equal(table, c.table)


@pytest.mark.parametrize("slack", [0, 300])
@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("name", list(PARTS))
def test_weights_in_two_parts(name, score, slack):
    """The bound on the lengths is what the table holds: the call's longest, or 300 blocks above it."""
    call = Call(PARTS[name], score, seed=5, slack=slack)
    _pairs(call)
    call.run()
    call.check(two_parts=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bound", [3, 40, 400])
def test_weights_in_two_parts_by_the_rows_there_are(d, bound):
    """32 rows to a kv head at most, over 700 tokens, whatever the bound on them."""
    call = Call((f16, d, (700, 90), 3, 2, 8))
    _pairs(call)
    call.max_new = bound
    call.run()
    call.check(two_parts=True)


@pytest.mark.parametrize("d", [64, 128])
def test_the_first_rows_of_a_long_prompt(d):
    """Rows that see at most 512 tokens, of a prompt of 1500."""
    call = Call((f16, d, (1500,), 1500, 1, 4), seed=5)
    _pairs(call)
    call.run()
    call.check()
    # the first 512 rows, as the last of a sequence of 512
    call.lens, call.new = (512,), [512]
    call.start = np.array([0, 512])
    call.c.rows[0] = call.c.rows[0][:, :, :512]
    call.check(two_parts=True)
