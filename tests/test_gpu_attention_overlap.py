"""Parts of one buffer that lie side by side, each in the other's span, without a common byte."""

import pytest
import torch

import activation_sparse_rank_amd as pi
from helpers import require_gpu
from test_gpu_attention import DEV, _filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# a buffer's shape and its two parts [n_tok, heads, d]
PARTS = {
    "side by side in a token": lambda n, h, d: ((n, 2, h, d), lambda x: (x[:, 0], x[:, 1])),
    "head by head": lambda n, h, d: ((n, h, 2, d), lambda x: (x[:, :, 0], x[:, :, 1])),
    "head-major": lambda n, h, d: ((h, 2, n, d), lambda x: (x[:, 0].transpose(0, 1), x[:, 1].transpose(0, 1))),
    "token by token in a head": lambda n, h, d: ((h, n, 2, d), lambda x: (x[:, :, 0].transpose(0, 1), x[:, :, 1].transpose(0, 1))),
}


@pytest.mark.parametrize("name", list(PARTS))
def test_read_into_parts_of_a_buffer(name):
    lens, hk, d = (90, 40), 3, 64
    c = _filled(2, hk, d, torch.float16, lens)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    shape, parts = PARTS[name](20, hk, d)
    k, v = parts(torch.zeros(shape, dtype=torch.float16, device=DEV))
    want = [torch.zeros((20, hk, d), dtype=torch.float16, device=DEV) for _ in range(2)]
    pi.kv_read(c.c, ln, want[0], want[1])
    pi.kv_read(c.c, ln, k, v)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and not torch.equal(k, v)


@pytest.mark.parametrize("name", list(PARTS))
def test_attend_between_parts_of_a_buffer(name):
    lens, hk, d = (90, 40), 3, 64
    c = _filled(2, hk, d, torch.float16, lens)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    shape, parts = PARTS[name](4, 2 * hk, d)
    q, out = parts(torch.zeros(shape, dtype=torch.float16, device=DEV))
    q.copy_(torch.randn(q.shape, device=DEV))
    want = torch.zeros((4, 2 * hk, d), dtype=torch.float16, device=DEV)
    q0 = q.clone()
    pi.attend(c.c, q0, ln, want)
    pi.attend(c.c, q, ln, out)
    assert torch.equal(out, want) and torch.equal(q, q0)
    with pytest.raises(pi.PiError):
        pi.attend(c.c, q, ln, q)
