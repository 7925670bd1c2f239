"""Bounds that a caller leaves out, and sizes of 0."""

import numpy as np
import pytest
import torch

import activation_sparse_rank_amd as pi
from helpers import require_gpu
from test_gpu_attention import DEV, Cache, _check_read, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_append_and_read_without_a_bound():
    """More rows in all than one sequence's table row holds."""
    f16 = torch.float16
    new = (100, 120, 5, 128, 0, 77)
    c = Cache(len(new), 2, 64, 4, f16)
    k, v = _rows(sum(new), 2, 64, f16, 3)
    start = np.concatenate(([0], np.cumsum(new)))
    for s in range(len(new)):
        c.rows[s] = np.stack([x[start[s]:start[s + 1]].cpu().numpy().astype(np.float64).transpose(1, 0, 2) for x in (k, v)])
    lens = torch.tensor(new, dtype=torch.int32, device=DEV)
    qs = torch.from_numpy(start.astype(np.int32)).to(DEV)
    pi.kv_append(c.c, k, v, lens, q_start=qs)
    c.check()
    _check_read(c, lens, qs)
    out = [torch.zeros((sum(new), 2, 64), dtype=f16, device=DEV) for _ in range(2)]
    pi.kv_read(c.c, lens, out[0], out[1], q_start=qs)
    want = [torch.zeros_like(x) for x in out]
    pi.kv_read(c.c, lens, want[0], want[1], q_start=qs, max_new=128)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("seqs,heads,blocks,pages", [(0, 2, 4, 8), (2, 0, 4, 8), (2, 2, 0, 8), (2, 2, 4, 0)])
def test_caches_without_sequences_heads_blocks_or_pages(seqs, heads, blocks, pages):
    with pytest.raises(ValueError, match="must have"):
        pi.KVCache(torch.zeros((pages, 2, 2048), dtype=torch.uint8, device=DEV), torch.zeros((pages, 2), device=DEV),
                   torch.zeros((seqs, heads, 2, 32, 64), dtype=torch.float16, device=DEV),
                   torch.zeros((seqs, heads, blocks), dtype=torch.int32, device=DEV))
