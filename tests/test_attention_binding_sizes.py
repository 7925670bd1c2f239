"""CPU checks of the attention side's binding: a descriptor without sequences is
refused before rows are divided by their number."""

import ctypes

import pytest
import torch

from activation_sparse_rank_amd import _lib as L
from activation_sparse_rank_amd import attention as A

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="refusals of CPU tensors, on hosts without a GPU")


@pytest.mark.parametrize("n", [0, -1])
def test_no_sequences(n):
    native = A.load_native()
    cache = L.PiKVCache(n, 3, 64, 4, 10, L.PI_F16, 0x1000, 0x2000, 0x3000, 0x4000, None)
    a = ctypes.addressof(cache)
    rows, lens = torch.zeros((4, 3, 64), dtype=torch.float16), torch.zeros(0, dtype=torch.int32)
    for f in (native.kv_append, native.kv_read):
        with pytest.raises(ValueError, match="sequences"):
            f(a, 0, rows, rows, lens, None, None, None)
    with pytest.raises(ValueError, match="sequences"):
        native.attend(a, 0, rows, lens, rows, None, None, 64, 0.1, False, torch.zeros(999, dtype=torch.uint8), None)
