"""Values next to fp32's largest: the output lies between them, so no sum on the
way to it may overflow."""

import pytest
import torch

from attention_helpers import CALLS, Call, f32
from helpers import require_gpu

pytestmark = pytest.mark.gpu

NAMES = [n for n in CALLS if CALLS[n][0] == f32]

@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("top", [1e31, 3e38])
@pytest.mark.parametrize("name", NAMES)
def test_large_values(name, top, score):
    call = Call(CALLS[name], score)
    c = call.c
    for s in range(len(call.lens)):
        for h in range(call.hk):
            at = call.pages(s, h)
            c.scales[at, 1] = top / 127 * torch.rand(len(at), generator=call.gen, device=at.device).clamp_(min=0.01)
    c.pages[:, 1].clamp_(min=1)                                  # codes 1 .. 255: magnitudes of 127 at most
    call.run()
    assert torch.isfinite(call.out).all()
    call.check()
    # and beside values next to nothing in another sequence
    at = call.pages(len(call.lens) - 1, 0)
    c.scales[at, 1] *= 2.0 ** -100 / top
    call.run()
    call.check()
