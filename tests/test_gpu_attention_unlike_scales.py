"""Value scales of a sequence that lie far apart, beside a long flat tail of
small weights: a weight counts down to 2^-31 of the row's largest, whatever its
block's value scale.

The first token of each of the first eight blocks takes the row (eight, so that
each wave that shares the blocks with others meets one); every other token's
weight is 2^-21.6 of one of theirs, all together half a hundredth of the sum,
so a sum that loses them is off by ten times the weights' rounding (2^-11) and
twenty times what 4096 fp32 additions of like terms may round by."""

import pytest
import torch

from attention_helpers import CALLS, Call, Tail, f16, f32
from helpers import require_gpu
from test_gpu_attention import DEV

pytestmark = pytest.mark.gpu

# dtype, head size, new rows, query heads: a workgroup of k_attend with one or two tiles, of k_attend_many with two, four or eight waves
ROWS = [(f16, 64, 1, 4), (f16, 64, 3, 8), (f16, 128, 1, 8), (f16, 128, 3, 8), (f16, 64, 5, 8), (f16, 128, 5, 8),
        (f16, 128, 9, 8), (f16, 128, 17, 8), (f32, 64, 1, 4), (f32, 128, 1, 4), (f32, 64, 5, 8), (f32, 128, 5, 8)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("bits", [0, 2, 5, 9, 9.9, 12, 15, 23])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"{r[0]}-{r[1]}-{r[2] * r[3]}")
def test_a_tail_in_blocks_of_low_scale(rows, bits):
    """The heavy tokens' blocks have the large scale."""
    call = Tail(*rows)
    call.c.scales[call.at[8:], 1] = 2.0 ** -bits
    call.run()
    call.check(seqs=[0], alike=True)


@pytest.mark.parametrize("bits", [2, 5, 9, 9.9, 12, 15])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"{r[0]}-{r[1]}-{r[2] * r[3]}")
def test_a_row_in_blocks_of_low_scale(rows, bits):
    """Eight blocks of the large scale, whose weights are next to nothing; the row and its tail lie in the others."""
    call = Tail(*rows)
    c = call.c
    c.scales[:, 1] = 2.0 ** -bits
    big = call.at[8:16, None]
    c.scales[big, 1] = 1.0
    slot = torch.arange(32, device=DEV)[None]
    c.pages[big, 0, slot // 16 * (call.d // 64) * 1024 + slot % 16 * 16] = 1       # element 0 of their keys: -127
    call.run()
    call.check(seqs=[0], alike=True)


@pytest.mark.parametrize("score", [False, True])
@pytest.mark.parametrize("span", [30, 60, 100])
@pytest.mark.parametrize("name", list(CALLS))
def test_scales_that_span(name, span, score):
    """Value scales spread over 2^span (fp16 outputs hold 2^30 of them at most), in no order."""
    call = Call(CALLS[name], score)
    if call.dt == f16:
        span = min(span, 30)
    c = call.c
    for s in range(len(call.lens)):
        for h in range(call.hk):
            at = call.pages(s, h)
            e = torch.rand(len(at), generator=call.gen, device=at.device) * span - span * (0.5 if call.dt == f32 else 0.8)
            c.scales[at, 1] = torch.exp2(e) * 1.37
    call.run()
    call.check()
