"""Pages of a pool against the same steps on lists: forks in any order, copies on
write, the lowest free pages first, compaction in place and beside, refused calls
that change nothing, buffers of any size and number.  Everything is whole numbers
or moved bytes, so all comparisons are exact."""
import numpy as np
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


class Model:
    """The pool on lists; contents[p] stands for what page p holds."""

    def __init__(self, rows, max_pages, pages, page):
        self.page, self.max_pages = page, max_pages
        self.table = [[-7] * max_pages for _ in range(rows)]
        self.lens = [0] * rows
        self.refs = [0] * pages
        self.contents = list(range(pages))

    def held(self, n):
        return -(-n // self.page)

    def fork(self, parents, children):
        table, lens = [list(r) for r in self.table], list(self.lens)
        for p, c in zip(parents, children):
            for j in range(self.held(lens[c])):
                self.refs[table[c][j]] -= 1
            for j in range(self.held(lens[p])):
                self.refs[table[p][j]] += 1
                self.table[c][j] = table[p][j]
            self.lens[c] = lens[p]

    def free(self, seqs):
        for s in seqs:
            for j in range(self.held(self.lens[s])):
                self.refs[self.table[s][j]] -= 1
            self.lens[s] = 0

    def extend(self, seqs, counts, most):
        free = [i for i, r in enumerate(self.refs) if r == 0]
        moves, slots = [], []
        for s, n in zip(seqs, counts):
            have, row = self.held(self.lens[s]), self.table[s]
            if n and self.lens[s] % self.page and self.refs[row[have - 1]] > 1:
                self.refs[row[have - 1]] -= 1
                moves.append((row[have - 1], free[0]))
                row[have - 1] = free.pop(0)
                self.refs[row[have - 1]] = 1
            for j in range(have, self.held(self.lens[s] + n)):
                row[j] = free.pop(0)
                self.refs[row[j]] = 1
            at = range(self.lens[s], self.lens[s] + n)
            slots.append([row[i // self.page] * self.page + i % self.page for i in at] + [-1] * (most - n))
            self.lens[s] += n
        self.move(moves)
        return slots

    def move(self, moves):
        for a, b in moves:
            self.contents[b] = self.contents[a]

    def compact(self):
        used = sum(r > 0 for r in self.refs)
        holes = [i for i in range(used) if self.refs[i] == 0]
        moves = list(zip([i for i in range(used, len(self.refs)) if self.refs[i] > 0], holes))
        to = dict(moves)
        for row, n in zip(self.table, self.lens):
            for j in range(self.held(n)):
                row[j] = to.get(row[j], row[j])
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.move(moves)


class Pool:
    """The same on the device, beside a model; the caches' pages hold numbers of their own."""

    def __init__(self, rows, max_pages, pages, page, caches=None):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.model = Model(rows, max_pages, pages, page)
        self.table = torch.full((rows, max_pages), -7, **i32)
        self.lens, self.refs = torch.zeros(rows, **i32), torch.zeros(pages, **i32)
        self.page = page
        self.caches = [torch.randint(0, 255, (pages, 4, 48), device="cuda", dtype=torch.uint8)] if caches is None else caches
        self.first = [c.clone() for c in self.caches]

    def state(self):
        return self.table, self.lens, self.refs

    def fork(self, parents, children):
        mk.fork_sequences(*self.state(), i32(parents), i32(children), self.page)
        self.model.fork(parents, children)

    def free(self, seqs):
        mk.free_sequences(*self.state(), i32(seqs), self.page)
        self.model.free(seqs)

    def extend(self, seqs, counts, most=None):
        most = max(counts, default=0) if most is None else most
        slots = mk.extend_sequences(*self.state(), i32(seqs), i32(counts), most, self.caches, self.page)
        want = self.model.extend(seqs, counts, most)
        assert slots.tolist() == want
        return slots

    def compact(self, in_place=False):
        where = dict(table_out=self.table, refs_out=self.refs) if in_place else {}
        before = [t.clone() for t in self.state()]
        o = mk.compact_pages(*self.state(), self.caches, self.page, **where)
        if not in_place:
            assert all(torch.equal(a, b) for a, b in zip(self.state(), before))
        self.table, self.refs = o["block_table"], o["refs"]
        self.model.compact()

    def check(self):
        m = self.model
        assert self.table.tolist() == m.table and self.lens.tolist() == m.lens and self.refs.tolist() == m.refs
        at = torch.tensor(m.contents, device="cuda")
        for c, first in zip(self.caches, self.first):
            assert torch.equal(c, first[at])


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_grow_fork_write_free():
    p = Pool(6, 5, 30, 4)
    p.extend([0, 3], [7, 4])
    p.check()
    p.fork([0, 0, 3], [1, 2, 4])
    p.check()
    p.extend([2, 0, 1, 4], [1, 1, 6, 0])  # three rows hold page 1: two copy it, the last keeps it
    p.check()
    p.free([0, 5, 3])
    p.check()
    p.extend([5, 0], [20, 1])
    p.check()


def test_forks_among_themselves():
    p = Pool(5, 6, 40, 8)
    p.extend([0, 1, 2, 3], [9, 20, 8, 33])
    for parents, children in (([1, 0], [0, 1]), ([1, 2, 3, 0], [0, 1, 2, 3]), ([2, 2, 2, 2, 2], [0, 1, 2, 3, 4]),
                              ([3, 4], [3, 0]), ([], [])):
        p.fork(parents, children)
        p.check()
        p.extend([0, 1], [1, 1])
        p.check()


@pytest.mark.parametrize("seed", range(6))
def test_any_order_of_steps(seed):
    rng = np.random.default_rng(seed)
    rows, page = int(rng.integers(2, 40)), int(rng.choice([1, 3, 8, 16]))
    p = Pool(rows, 12, rows * 12, page)
    for _ in range(25):
        some = rng.permutation(rows)[:rng.integers(0, rows + 1)].tolist()
        step = rng.integers(0, 5)
        if step == 0:
            p.fork(rng.integers(0, rows, len(some)).tolist(), some)
        elif step == 1:
            p.free(some[:len(some) // 2])
        elif step <= 3:
            room = [12 * page - p.model.lens[s] for s in some]
            counts = [int(rng.integers(0, min(r, 3 * page) + 1)) for r in room]
            p.extend(some, counts, most=max(counts, default=0) + int(rng.integers(0, 3)))
        else:
            p.compact(in_place=bool(rng.integers(0, 2)))
        p.check()


def test_many_sharers_and_rows():
    p = Pool(4096, 3, 9000, 16)
    p.extend([0], [20])
    p.fork([0] * 4095, list(range(1, 4096)))
    p.check()
    p.extend(list(range(4096)), [1] * 4096)
    p.check()
    p.free(list(range(0, 4096, 2)))
    p.compact()
    p.check()


@pytest.mark.parametrize("pages,free", [(70001, 90), (32768, 1), (8193, 60), (1025, 60), (31, 4)])
def test_lowest_free_pages_of_full_pools(pages, free):
    rng = np.random.default_rng(pages)
    p = Pool(3, 64, pages, 1, caches=[torch.arange(pages * 4, device="cuda", dtype=torch.int32).view(pages, 4)])
    where = rng.permutation(pages)[:free]
    p.refs.fill_(1)
    p.refs[torch.from_numpy(where).cuda()] = 0
    p.model.refs = p.refs.tolist()
    a = free // 3
    p.extend([2, 0], [a, free // 2])
    p.check()
    p.extend([1], [min(64, free - a - free // 2)])
    p.check()


def test_refused_lists_change_nothing():
    p = Pool(4, 3, 8, 4)
    p.extend([0, 1], [10, 5])
    for list_of in (lambda: mk.fork_sequences(*p.state(), i32([0, 0]), i32([2, 2]), 4, check=False),     # a child twice
                    lambda: mk.fork_sequences(*p.state(), i32([0]), i32([4]), 4, check=False),
                    lambda: mk.fork_sequences(*p.state(), i32([-1, 0]), i32([2, 3]), 4, check=False),
                    lambda: mk.free_sequences(*p.state(), i32([1, 0, 1]), 4, check=False),
                    lambda: mk.free_sequences(*p.state(), i32([2 ** 31 - 1]), 4, check=False)):
        list_of()
        assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
        p.check()
    for seqs, counts, most in (([0, 1, 0], [1, 1, 1], 1), ([9], [1], 1), ([0], [3], 3),   # twice; no row; its row is full
                               ([1], [2], 1), ([1], [-1], 1), ([2, 3], [12, 5], 12)):     # above most; below none; 3 pages free
        slots = mk.extend_sequences(*p.state(), i32(seqs), i32(counts), most, p.caches, 4, check=False)
        assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
        assert torch.all(slots == -1)
        p.check()
    with pytest.raises(mk.MkError):
        mk.free_sequences(*p.state(), i32([7]), 4)
    p.extend([2, 3], [4, 8])  # all that is left
    p.check()
    assert p.refs.min() == 1


def test_more_pages_than_32_bits_count_are_refused():
    # rows of 2^31 - 1 pages of one token each; their table is never looked at
    state = (i32([[0]]), i32([0] * 3), i32([0] * 8))
    before = [t.clone() for t in state]
    slots = torch.zeros((3, 1), dtype=torch.int64, device="cuda")
    counts = i32([2 ** 31 - 2] * 3)
    assert mk.mk_extend_sequences(*state, 3, 2 ** 31 - 1, 8, 1, i32([0, 1, 2]), counts, 3, 2 ** 31 - 2, None, []) == mk.MK_OK
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    assert all(torch.equal(a, b) for a, b in zip(state, before)) and slots.sum() == 0


def test_empty_pools_tables_and_lists():
    none = i32([])
    p = Pool(2, 0, 0, 4)
    p.caches = []
    p.extend([0], [0])
    p.fork([0], [1])
    p.free([0, 1])
    o = mk.compact_pages(*p.state(), [], 4)
    assert o["block_table"].shape == (2, 0) and o["refs"].shape == (0,)
    q = Pool(2, 3, 0, 4)
    assert mk.compact_pages(*q.state(), [], 4)["block_table"].tolist() == q.table.tolist()
    for pool in (p, q):
        mk.fork_sequences(*pool.state(), none, none, 4)
        mk.free_sequences(*pool.state(), none, 4)
        assert mk.extend_sequences(*pool.state(), none, none, 3, [], 4).shape == (0, 3)


def test_entries_that_are_no_pages_are_reported():
    p = Pool(3, 4, 10, 2)
    p.extend([0, 1], [6, 3])
    p.table[0, 1] = 10
    p.table[1, 0] = -3
    before = [t.clone() for t in p.state()]
    mk.fork_sequences(*p.state(), i32([0]), i32([2]), 2, check=False)
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    assert p.table[2].tolist() == [0, 10, 2, -7] and p.refs[:5].tolist() == [2, 1, 2, 1, 1]
    mk.free_sequences(*p.state(), i32([2, 1]), 2, check=False)
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    assert p.refs[:5].tolist() == [1, 1, 1, 1, 0]
    o = mk.compact_pages(*p.state(), p.caches, 2, check=False)
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    assert torch.equal(o["block_table"], p.table) and torch.equal(o["refs"], p.refs)
    assert torch.equal(before[0][0], p.table[0])
    assert mk.mk_get_status() == mk.MK_OK


@pytest.mark.parametrize("pages,used", [(1, 1), (1, 0), (1023, 500), (1024, 1024), (1025, 1), (40000, 20001), (300000, 7),
                                        (300000, 299990)])
def test_compaction_of_pools(pages, used):
    rng = np.random.default_rng(pages + used)
    p = Pool(3, max(1, -(-used // 2)), pages, 2, caches=[torch.arange(pages * 16, device="cuda", dtype=torch.int32).view(pages, 4, 4)])
    order = rng.permutation(pages)[:used]
    cut = used // 2
    for row, part in ((0, order[:cut]), (2, order[cut:])):
        p.table[row, :len(part)] = i32(part.tolist())
        p.model.table[row][:len(part)] = part.tolist()
        p.lens[row] = p.model.lens[row] = 2 * len(part)
    p.refs[torch.from_numpy(order).cuda()] = 1
    for i in order.tolist():
        p.model.refs[i] = 1
    p.compact(in_place=pages % 2 == 0)
    p.check()
    assert int((p.refs[:used] == 0).sum()) == 0


@pytest.mark.parametrize("shape,dtype", [((3,), torch.uint8), ((1,), torch.uint8), ((16385,), torch.uint8), ((2, 6), torch.uint8),
                                         ((8, 16, 128), torch.bfloat16), ((5, 7), torch.float32), ((70000, 5), torch.float32)])
def test_copies_of_any_size(shape, dtype):
    pages = 11
    whole = torch.randint(0, 255, (2, pages + 1, *shape), device="cuda").to(dtype)
    caches = [whole[0, 1:], whole[1, 1:]]
    strided = torch.randint(0, 255, (pages, 3, *shape), device="cuda").to(dtype)
    caches.append(strided[:, 1])
    if len(shape) > 1:
        caches.append(torch.randint(0, 255, (pages, shape[1], shape[0], *shape[2:]), device="cuda").to(dtype).transpose(1, 2))
    all_before = [whole.clone(), strided.clone()]
    want = [c.clone() for c in caches]
    src, dst = [0, 5, 5, 10], [1, 4, 9, 2]
    for w in want:
        w[dst] = w[src]
    mk.copy_pages(caches, i32(src), i32(dst))
    for c, w in zip(caches, want):
        assert torch.equal(c, w)
    assert torch.equal(whole[:, 0], all_before[0][:, 0]) and torch.equal(strided[:, ::2], all_before[1][:, ::2])
    mk.copy_pages(caches, i32([]), i32([]))
    mk.copy_pages([], i32([1]), i32([2]))
    mk.copy_pages(caches, i32([0, -1, 3]), i32([7, 1, pages]), check=False)
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    for w in want:
        w[7] = w[0]
    for c, w in zip(caches, want):
        assert torch.equal(c, w)


def test_more_buffers_than_one_launch_takes():
    n = 300
    caches = [torch.randint(0, 255, (6, 2, 24 + i % 5), device="cuda", dtype=torch.uint8) for i in range(n)]
    p = Pool(3, 2, 6, 4, caches=caches)
    p.extend([0], [6])
    p.fork([0, 0], [1, 2])
    p.extend([0, 1, 2], [1, 1, 1])
    p.check()
    p.free([0])
    p.compact()
    p.check()
    want = [c.clone() for c in caches]
    for w in want:
        w[5] = w[1]
    mk.copy_pages(caches, i32([1]), i32([5]))
    assert all(torch.equal(c, w) for c, w in zip(caches, want))


def test_offsets_past_32_bits():
    pages, size = 80, 2 ** 26 + 64
    c = torch.empty((pages, size), dtype=torch.uint8, device="cuda")
    c[3] = 5
    c[79].random_(0, 255)
    mk.copy_pages([c], i32([79, 3]), i32([70, 78]))
    assert torch.equal(c[70], c[79]) and torch.all(c[78] == 5)


def test_streams_and_workspace():
    p = Pool(8, 6, 60, 4)
    side = torch.cuda.Stream()
    ws = torch.randint(0, 255, (mk.mk_pages_workspace_size(6, 60, 8),), device="cuda", dtype=torch.uint8)
    seqs, counts = i32([0, 1]), i32([5, 9])
    torch.cuda.synchronize()
    slots = mk.extend_sequences(*p.state(), seqs, counts, 9, p.caches, 4, stream=side, workspace=ws, ws_bytes=ws.numel())
    assert slots.tolist() == p.model.extend([0, 1], [5, 9], 9)
    with pytest.raises(mk.MkError) as e:
        mk.fork_sequences(*p.state(), seqs, counts, 4, workspace=ws, ws_bytes=64)
    assert e.value.status == mk.MK_ERR_WORKSPACE
    p.check()


def test_captured_steps_replay():
    p = Pool(9, 8, 200, 4)
    p.extend([0], [6])
    children, parents, ones = i32(list(range(1, 9))), i32([0] * 8), i32([1] * 8)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())

    def step():
        mk.fork_sequences(*p.state(), parents, children, 4, check=False)
        return mk.extend_sequences(*p.state(), children, ones, 1, p.caches, 4, check=False)

    with torch.cuda.stream(stream):
        step()  # allocates what the library keeps for this stream
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            slots = step()
    p.model.fork([0] * 8, list(range(1, 9)))
    p.model.extend(list(range(1, 9)), [1] * 8, 1)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        p.model.fork([0] * 8, list(range(1, 9)))
        assert slots.tolist() == p.model.extend(list(range(1, 9)), [1] * 8, 1)
        p.check()
    assert mk.mk_get_status() == mk.MK_OK
