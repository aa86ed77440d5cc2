"""The tensor forms: outputs when torch's internal allocation entry is missing or
does something else than it is used for, strides that say nothing."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk._load_torch()


def _raises(*a):
    raise TypeError("another signature")


@pytest.mark.parametrize("entry", [
    None,
    lambda shape, strides, dtype: torch.empty(shape, dtype=torch.float32, device="cuda"),     # another type
    lambda shape, strides, dtype: torch.empty([2 * n for n in shape], dtype=dtype, device="cuda"),  # another shape
    lambda shape, strides, dtype: torch.empty(shape[::-1], dtype=dtype, device="cuda").T,     # other strides
    lambda shape, strides, dtype: torch.empty(shape, dtype=dtype).pin_memory(),               # another device
    lambda *a: None,
    _raises,
], ids=["missing", "dtype", "shape", "strides", "device", "none", "raises"])
def test_outputs_whatever_the_internal_entry_does(entry, monkeypatch):
    x, w = torch.randn(6, 256, device="cuda").bfloat16(), torch.ones(256, device="cuda").bfloat16()
    want = mk.add_rmsnorm(x, w, e4m3=True)
    monkeypatch.setattr(torch._C._dynamo.guards, "_empty_strided_cuda", entry)
    mk._load_torch()
    got = mk.add_rmsnorm(x, w, e4m3=True)
    for name, dtype in (("out", torch.bfloat16), ("out8", torch.float8_e4m3fn), ("scale", torch.float32)):
        t = got[name]
        assert t.dtype == dtype and t.is_cuda and t.is_contiguous() and t.shape == want[name].shape
        assert torch.equal(t.view(torch.uint8), want[name].view(torch.uint8))


def test_strides_of_dimensions_of_one_do_not_matter():
    kv = torch.randn(4, 2, 1, 1, 64, device="cuda").bfloat16()
    k, v = kv[:, 0], kv[:, 1]
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    lens = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    want = mk.paged_attention(q, k, v, table, lens)
    odd = v.as_strided(v.shape, (v.stride(0), 999, 7, 1), v.storage_offset())
    for a, b in ((k, odd), (k.as_strided(k.shape, (k.stride(0), 13, 0, 1), k.storage_offset()), v)):
        got = mk.paged_attention(q, a, b, table, lens)
        assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    with pytest.raises(ValueError, match="strides"):
        mk.paged_attention(q, k, v.contiguous(), table, lens)
