"""CPU checks of the attention side's C ABI: rows that are written must not share
bytes with others; views side by side in one buffer do not.  No call that a test
expects to be refused reaches a kernel launch, and no call that is not is made."""

import ctypes

import pytest
import torch

from activation_sparse_rank_amd import _lib as L

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="fake-pointer validation tests run only on hosts without a GPU")

A, B, C, D = 0x100000, 0x10000000, 0x20000000, 0x30000000      # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _cache(h=4):
    return L.PiKVCache(2, h, 128, 16, 64, L.PI_F16, A, B, C, D, None)


@pytest.mark.parametrize("k,kt,kh,v,vt,vh", [
    (B, 512, 128, B, 512, 128),                                  # the same rows
    (B, 512, 128, B + 256, 512, 128),                            # a head further
    (B, 1024, 128, B + 768, 1024, 128),                          # interleaved, the last head shared
    (B, 512, 128, B + 1024, 1024, 128),                          # one token further, with another stride
    (B, 128, 512, B + 2048, 128, 512),                           # head-major, inside each other
])
def test_read_refuses_outputs_that_overlap(lib, k, kt, kh, v, vt, vh):
    c = _cache()
    assert lib.pi_kv_read(ctypes.byref(c), A, A, 4, k, kt, kh, v, vt, vh, 4, None) == L.PI_E_RANGE
