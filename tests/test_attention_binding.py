"""CPU checks of the attention side's binding: what the C ABI cannot see is
refused before anything is launched (no GPU tensor is made here)."""

import ctypes

import pytest
import torch

from activation_sparse_rank_amd import _lib as L
from activation_sparse_rank_amd import attention as A
import activation_sparse_rank_amd as pi

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="refusals of CPU tensors, on hosts without a GPU")

H, F, I = torch.float16, torch.float32, torch.int32


def t(*shape, dtype=H):
    return torch.zeros(shape, dtype=dtype)


@pytest.fixture(scope="module")
def native():
    return A.load_native()


@pytest.fixture()
def rope():
    return L.PiRope(64, 64, L.PI_ROPE_HALF, 1.0, 1e-6, 0x1000, None, None)


@pytest.fixture()
def cache():
    return L.PiKVCache(2, 3, 64, 4, 10, L.PI_F16, 0x1000, 0x2000, 0x3000, 0x4000, None)


def test_descriptors_refuse_cpu_tensors():
    with pytest.raises(ValueError, match="GPU"):
        pi.Rope(torch.zeros(32, dtype=torch.float64), 64)
    with pytest.raises(ValueError, match="layout"):
        pi.Rope(torch.zeros(32, dtype=torch.float64), 64, layout="other")
    with pytest.raises(ValueError, match="GPU"):
        pi.KVCache(t(4, 2, 2048, dtype=torch.uint8), t(4, 2, dtype=F), t(1, 1, 2, 32, 64), t(1, 1, 4, dtype=I))


def test_rope_refuses(native, rope):
    a = ctypes.addressof(rope)

    def call(q=t(5, 4, 64), k=t(5, 2, 64), pos=t(5, dtype=I), qo=t(5, 4, 64), ko=t(5, 2, 64)):
        native.qk_rope(a, 0, q, k, pos, qo, ko, None)

    with pytest.raises(ValueError, match="q must live in GPU memory"):
        call()
    for bad, err in ((dict(q=[1]), TypeError), (dict(q=t(5, 4, 64, dtype=torch.bfloat16)), TypeError),
                     (dict(q=t(5, 4, 64, dtype=torch.int16)), TypeError)):
        with pytest.raises(err):
            call(**bad)
    with pytest.raises(TypeError, match="arguments"):
        native.qk_rope(a, 0)
    with pytest.raises(ValueError, match="descriptor"):
        native.qk_rope(0, 0, *[t(5, 4, 64)] * 5, None)


def test_cache_calls_refuse(native, cache):
    a = ctypes.addressof(cache)
    for f in (native.kv_append, native.kv_read):
        with pytest.raises(ValueError, match="GPU"):
            f(a, 0, t(4, 3, 64), t(4, 3, 64), t(2, dtype=I), None, None, None)
        with pytest.raises(TypeError, match="float16"):
            f(a, 0, t(4, 3, 64, dtype=F), t(4, 3, 64), t(2, dtype=I), None, None, None)
        with pytest.raises(TypeError, match="Tensor"):
            f(a, 0, None, t(4, 3, 64), t(2, dtype=I), None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        native.attend(a, 0, t(4, 6, 64), t(2, dtype=I), t(4, 6, 64), None, None, 64, 0.1, False,
                      t(999, dtype=torch.uint8), None)
    with pytest.raises(TypeError):
        native.attend(a, "0", t(4, 6, 64), t(2, dtype=I), t(4, 6, 64), None, None, 64, 0.1, False,
                      t(999, dtype=torch.uint8), None)


def test_evict_refuses():
    tab, sc, n = t(2, 3, 8, dtype=I), t(2, 3, 8, dtype=F), t(2, dtype=I)
    with pytest.raises(ValueError, match="table must live in GPU memory"):
        pi.kv_evict(tab, sc, n, 4, 1, n)
    with pytest.raises(ValueError, match="together"):
        pi.kv_evict(tab, sc, n, 4, 1, n, table_out=tab)
    with pytest.raises(TypeError):
        pi.kv_evict(None, sc, n, 4, 1, n)
