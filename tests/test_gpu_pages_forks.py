"""Forks of rows of any length: every column of every pair is read before it is
written, and the call's memory does not grow with the rows.  Exact, on the lists of
test_gpu_pages.py."""
import numpy as np
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_pages import Pool, i32  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()


# max_pages: a row of 8 columns and less, of several turns of the grid, of odd length
@pytest.mark.parametrize("max_pages", [1, 7, 8, 129, 1300, 5003])
@pytest.mark.parametrize("rows", [2, 32, 33, 200])
def test_permutations_chains_and_shared_parents(rows, max_pages):
    rng = np.random.default_rng(rows + max_pages)
    lens = rng.integers(0, max_pages + 1, rows)
    lens[0], lens[-1] = max_pages, 0
    p = Pool(rows, max_pages, int(lens.sum()) + 1, 1, caches=[])
    p.extend(list(range(rows)), lens.tolist())
    p.fork([(i + 1) % rows for i in range(rows)], list(range(rows)))  # a cycle: every child another's parent
    p.check()
    p.fork(rng.permutation(rows).tolist(), rng.permutation(rows).tolist())
    p.check()
    some = rng.permutation(rows)[:max(1, rows - 1)].tolist()
    p.fork(rng.integers(0, rows, len(some)).tolist(), some)
    p.check()
    assert mk.mk_get_status() == mk.MK_OK


@pytest.mark.parametrize("n", [3, 40])
def test_workspace_does_not_grow_with_the_rows(n):
    rows, max_pages = n + 1, 2 ** 21 + 5
    table = torch.full((rows, max_pages), -7, dtype=torch.int32, device="cuda")
    table[0, :3] = i32([4, 2, 9])
    lens, refs = torch.zeros(rows, dtype=torch.int32, device="cuda"), torch.zeros(12, dtype=torch.int32, device="cuda")
    lens[0] = 3
    refs[i32([4, 2, 9]).long()] = 1
    ws = torch.randint(0, 255, (256,), device="cuda", dtype=torch.uint8)  # 4 bytes a pair
    mk.fork_sequences(table, lens, refs, i32([0] * n), i32(list(range(1, rows))), 1, workspace=ws, ws_bytes=256)
    assert lens.tolist() == [3] * rows and refs[i32([4, 2, 9]).long()].tolist() == [rows] * 3 and int(refs.sum()) == 3 * rows
    assert torch.equal(table[:, :3], table[:1, :3].expand(rows, 3)) and torch.all(table[:, 3:] == -7)


def test_a_refused_fork_of_many_changes_nothing():
    p = Pool(60, 20, 400, 4, caches=[])
    p.extend(list(range(10)), [17] * 10)
    children = list(range(10, 55))
    for parents, kids in (([0] * 45, children[:-1] + [11]), ([0] * 44 + [60], children), ([-1] * 45, children)):
        mk.fork_sequences(*p.state(), i32(parents), i32(kids), 4, check=False)
        assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
        p.check()
    p.fork([i % 10 for i in range(45)], children)
    p.check()
