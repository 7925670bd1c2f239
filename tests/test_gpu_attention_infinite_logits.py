"""Rows whose logits are all -infinity: their softmax is NaN, and no other row's is."""

import pytest
import torch

from attention_helpers import CALLS, Call
from helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_rows_of_minus_infinity(name, score):
    require_gpu()
    call = Call(CALLS[name], score)
    s = len(call.lens) - 1
    # the first element of the keys of the last sequence's first kv head: negative
    at = call.pages(s, 0)[:, None]
    slot = torch.arange(32, device=at.device)[None]
    call.c.pages[at, 0, slot // 16 * (call.d // 64) * 1024 + slot % 16 * 16] = 100
    hit = call.new[s] // 2 + int(call.start[s])                  # a token's second query head of that kv head
    head = min(1, call.group - 1)
    call.q[hit, head, 0] = float("inf")
    out = call.run()
    bad = torch.zeros(out.shape[:2], dtype=torch.bool, device=out.device)
    bad[hit, head] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()
    if score:
        new, rest = call.c.score[s, 0], call.c.score.clone()
        rest[s, 0] = 0
        assert torch.isnan(new[0]) and torch.isfinite(rest).all()
