"""mk_paged_attention_fp4 over one large page, as a cache that is not paged is
passed: places in it past 32 bits, of the values and of the scales."""
import math

import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()
    torch.cuda.empty_cache()


TAIL = 2 ** 18  # keys, more than a few warps' ranges


@pytest.mark.parametrize("D,head,more", [
    (64, 2 ** 27, 0), (128, 2 ** 26, 0), (256, 2 ** 25, 0),  # 2^32 bytes of values before the last keys
    (128, 2 ** 26, 8), (128, 2 ** 26, 1),                    # units of 8 keys; rows looked up one by one
    (256, 2 ** 28, 0),                                       # and of scales
])
def test_places_in_a_page_past_32_bits(D, head, more):
    """The last TAIL keys are zeros, all others -1 in every column against queries of 1: scores of 0 and -D, and
    e^-64 * 2^27 < 2^-65 * TAIL, so the output is the last keys' value, 3 * 2, to the last bit, and lse log TAIL
    (weights of 1 are exact, so are their sums; the logarithm is off by 2^-22 of itself and 2^-21)."""
    n = head + TAIL + more
    c = mk.fp4_cache(1, n, 1, D)
    for name, first, last in (("k_cache", 0xaa, 0), ("v_cache", 0x22, 0x55), ("k_scales", 0x38, 0x38), ("v_scales", 0x38, 0x40)):
        t = c[name].view(torch.uint8)
        t[:, :n - TAIL].fill_(first)
        t[:, n - TAIL:].fill_(last)
    q = torch.ones((1, 1, D), dtype=torch.bfloat16, device="cuda")
    got = mk.paged_attention_fp4(q, **c, block_table=torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                                 seq_lens=torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0)
    assert torch.all(got["out"] == 6)
    assert abs(got["lse"].item() - math.log(TAIL)) <= 2.0 ** -21 + 2.0 ** -22 * math.log(TAIL)
