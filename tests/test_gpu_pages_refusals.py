"""What mk_last_error_detail() says of a refused extension: the place in the list
of a wrong count, the page that is none, and how many pages are missing.  Exact."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_pages import Pool, i32  # noqa: E402

POOL_FULL, PAGE_INDEX, TOKEN_COUNT = 25, 26, 27


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()


def refused(p, seqs, counts, most):
    slots = mk.extend_sequences(*p.state(), i32(seqs), i32(counts), most, p.caches, p.page, check=False)
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    assert torch.all(slots == -1)
    o = mk.mk_last_error_detail()
    return o["site"], o["info"]


def test_what_is_wrong_with_an_entry():
    p = Pool(4, 3, 8, 4)
    p.extend([0, 1], [10, 5])
    assert refused(p, [0], [3], 3) == (POOL_FULL, 1)          # 13 tokens are 4 pages of a row of 3
    assert refused(p, [2, 0], [1, 2 ** 31 - 1], 2 ** 31 - 1) == (POOL_FULL, 2 ** 29)  # ceil((2^31 + 9) / 4) - 3
    assert refused(p, [1], [2], 1) == (TOKEN_COUNT, 0)
    assert refused(p, [2, 3, 1], [1, 0, -1], 1) == (TOKEN_COUNT, 2)
    assert refused(p, [3, 1, 0], [2, 2, 9], 1) == (TOKEN_COUNT, 0)  # the first of three
    p.check()
    p.lens[3] = -2
    assert refused(p, [0, 3], [1, 0], 1) == (TOKEN_COUNT, 1)
    p.lens[3] = 0
    p.table[1, 1] = 99
    assert refused(p, [1], [1], 1) == (PAGE_INDEX, 99)


def test_missing_pages():
    p = Pool(5, 4, 8, 4)
    p.extend([0, 1], [10, 5])
    assert refused(p, [2, 3], [12, 5], 12) == (POOL_FULL, 2)  # 5 of 3
    p.fork([1, 1], [2, 3])
    assert refused(p, [1, 2, 3, 4], [1, 1, 1, 8], 8) == (POOL_FULL, 1)  # two copies, two new ones, of 3
    p.check()


def test_missing_pages_counted_in_64_bits():
    state = (i32([[0]]), i32([0] * 3), i32([0] * 8))  # the table is never looked at
    counts = i32([2 ** 31 - 2] * 3)
    assert mk.mk_extend_sequences(*state, 3, 2 ** 31 - 1, 8, 1, i32([0, 1, 2]), counts, 3, 2 ** 31 - 2, None, []) == mk.MK_OK
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    assert mk.mk_last_error_detail()["site"] == POOL_FULL and mk.mk_last_error_detail()["info"] == 2 ** 31 - 1
    # rows of 2^30 - 1 pages of two tokens; two of them are in the middle of page 4
    table = torch.empty((3, 2 ** 30 - 1), dtype=torch.int32, device="cuda")
    table[:2, 0] = 4
    lens, refs = i32([1, 1, 0]), i32([0, 0, 0, 0, 2, 0, 0, 0])
    slots = mk.extend_sequences(table, lens, refs, i32([0, 1, 2]), i32([41, 1, 8]), 41, [], 2, check=False)
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT and torch.all(slots == -1)
    # 20 and a copy, none (it keeps the page), 4; 7 are free
    assert mk.mk_last_error_detail()["site"] == POOL_FULL and mk.mk_last_error_detail()["info"] == 18
    assert lens.tolist() == [1, 1, 0] and int(refs.sum()) == 2
