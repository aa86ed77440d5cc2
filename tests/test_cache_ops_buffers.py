"""What the page operators' torch forms take as caches (no GPU is needed)."""
import ctypes

import pytest

import moe_token_dispatch_persistent_gb300 as mk

torch = pytest.importorskip("torch")


def test_caches_from_a_generator_are_held():
    mk._load_torch()
    caches = [torch.zeros((4, 2, 8)), torch.zeros((4, 3))]
    base, strides, sizes, n, held, pages = mk._page_buffers((t for t in caches), -1)
    assert n == 2 and pages == 4 and any(t is caches[0] for t in held) and any(t is caches[1] for t in held)
    words = ctypes.cast(base, ctypes.POINTER(ctypes.c_int64))
    assert list(words[:6]) == [caches[0].data_ptr(), caches[1].data_ptr(), 64, 12, 64, 12]
    assert strides == base + 16 and sizes == base + 32


def test_one_tensor_is_not_a_list_of_caches():
    mk._load_torch()
    with pytest.raises(ValueError, match="list"):
        mk._page_buffers(torch.zeros((4, 4, 8)), -1)
