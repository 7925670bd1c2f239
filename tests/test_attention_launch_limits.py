"""CPU checks of the attention side's C ABI: sizes of which a launch could not
hold the threads (2^32 - 1) are refused before the first launch of the call.  No
call here reaches a kernel launch."""

import ctypes

import pytest
import torch

from activation_sparse_rank_amd import _lib as L

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="fake-pointer validation tests run only on hosts without a GPU")

A, B, C, D = 0x100000, 1 << 44, 1 << 45, 1 << 46      # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return L.load()


def _cache(s, h, d, nb, dt=L.PI_F16):
    return L.PiKVCache(s, h, d, nb, 64, dt, A, B, C, D, A)


def test_rope(lib):
    r = L.PiRope(128, 128, L.PI_ROPE_HALF, 1.0, 1e-6, A, None, None)
    n = 1 << 24                                                  # 256 threads a token
    st = lib.pi_qk_rope(ctypes.byref(r), B, 64 * 128, 128, 64, None, 0, 0, 0, A, n, L.PI_F16, D, 64 * 128, 128, None, 0, 0, None)
    assert st == L.PI_E_SHAPE


def test_append_and_read(lib):
    c = _cache(1 << 10, 1 << 3, 128, 1 << 12)
    rows = 65504                                                 # 2048 blocks of 2^13 kv heads, two halves of 256 threads each
    n = (1 << 10) * 4
    args = (B, 1024, 128, C, 1024, 128, n, A, A, rows, None)
    assert lib.pi_kv_append(ctypes.byref(c), *args) == L.PI_E_SHAPE
    assert lib.pi_kv_read(ctypes.byref(c), A, A, rows, B, 1024, 128, C, 1024, 128, n, None) == L.PI_E_SHAPE


@pytest.mark.parametrize("seqs,hk,group,new,length,score", [
    (2048, 1, 1, 64, 8192 * 32, 1),          # the join: a workgroup of 256 threads for each of 2^24 blocks
    (1 << 20, 8, 1, 33, 544, 0),             # k_attend_many: a workgroup of 512 threads for each of 2^23 kv heads
    (1 << 21, 4, 1, 1, 100, 0),              # k_attend: a workgroup of 512 threads for each of 2^23
])
def test_attend(lib, seqs, hk, group, new, length, score):
    c = _cache(seqs, hk, 64, (length + 31) // 32)
    assert lib.pi_attend_workspace_bytes(ctypes.byref(c), hk * group, new, length, score) == 0
    d, h = 64, hk * group
    st = lib.pi_attend(ctypes.byref(c), B, h * d, d, h, seqs, A, A, new, length, 0.1, score, C, h * d, d, D, 1 << 62, None)
    assert st == L.PI_E_SHAPE


@pytest.mark.parametrize("seqs,nb", [(1 << 22, 600), (1 << 23, 512), (1 << 26, 1)])
def test_evict(lib, seqs, nb):
    st = lib.pi_kv_evict(B, C, A, seqs, 1, nb, 1, 1, D, 1 << 47, 1 << 46 | 1 << 45, None)
    assert st == L.PI_E_SHAPE


def test_sizes_below_the_limit_have_a_workspace(lib):
    for seqs, hk, new, length, score in ((2047, 1, 64, 8191 * 32, 1), ((1 << 20) - 1, 8, 33, 544, 0), ((1 << 20) - 1, 8, 1, 100, 0)):
        c = _cache(seqs, hk, 64, (length + 31) // 32)
        assert lib.pi_attend_workspace_bytes(ctypes.byref(c), hk, new, length, score) > 0, (seqs, hk, new)
