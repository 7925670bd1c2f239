"""Blocks whose value scale is 0: each of their values is 0 whatever the codes,
while their tokens keep their weights."""

import numpy as np
import pytest
import torch

from attention_helpers import CALLS, Call, f32
from helpers import host, require_gpu
from test_gpu_attention import DEV, Cache, _attend, _check_attend, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_blocks_of_value_scale_zero(name, score):
    call = Call(CALLS[name], score)
    for s in range(len(call.lens)):
        for h in range(call.hk):
            at = call.pages(s, h)
            call.c.scales[at[(s + h) % 3::3], 1] = 0.0           # codes as they were
    call.run()
    call.check()


@pytest.mark.parametrize("name", ["one tile", "fp32, one tile", "eight waves", "two groups"])
def test_zero_filled_pages(name):
    call = Call(CALLS[name])
    call.c.pages.zero_(), call.c.scales.zero_()
    out = call.run()
    assert torch.equal(out, torch.zeros_like(out))


def test_append_of_subnormal_rows_then_attend():
    """A largest magnitude of which a 127th is no fp32 number: scale 0 beside codes that are not 128."""
    n, d = 96, 64
    c = Cache(1, 1, d, 4, f32)
    k, v = _rows(n, 1, d, f32, 7)
    v = v.clone()
    v[32:64] = torch.randint(-40, 41, (32, 1, d), device=DEV) * 2.0 ** -149
    lens, _ = c.append(k, v, (n,))
    c.check()
    page = c.table[0, 0, 1]
    assert float(c.scales[page, 1]) == 0.0 and int((c.pages[page, 1] != 128).sum()) > 0
    q = torch.randn((1, 1, d), device=DEV)
    qs = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    out, _ = _attend(c, q, lens, qs, 1)
    _check_attend(c, q, out, lens, qs, d ** -0.5)
    assert np.isfinite(host(out)).all()
