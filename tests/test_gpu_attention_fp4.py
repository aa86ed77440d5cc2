"""mk_paged_attention_fp4 against the softmax in 64 bits: head layouts, page
sizes from one key up, lengths around tiles and pages, strided caches, factors,
sequences without keys, garbage in every place that must not be read, faults
that the kernel's own checks turn into a status.

Tolerances.  A score is a sum of D exact products in fp32: off by at most
2^-20 * scale * sum |q_i k_i| (16 steps of 2^-24); a query column 2^-28 of its
head's largest or less loses 2^-39 of that largest in fp16.  Together ds.  A
weight e^(s - m) is then off by 2 ds of itself (its own score and the maximum),
the exponential by 2^-21, and the sums over at most 6000 keys by 2^-16: together
less than 2 ds + 2^-15 of the weight, once in the sum of values and once in the
denominator.  In the sum of values it is rounded to fp16: 2^-11 of it, and
2^-35 of the largest weight where that is more.  Rounding the output adds 2^-8 of
it; lse is off by ds plus 2^-15, and 2^-22 of itself."""
import numpy as np
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()


def values_of(codes, scales):
    """Rows [..,D] in 64 bits of codes [..,D/2] and scales [..,D/16]."""
    steps = torch.tensor(STEPS + [-x for x in STEPS], dtype=torch.float64, device="cuda")
    x = torch.stack([steps[(codes & 15).long()], steps[(codes >> 4).long()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scales.double()[..., None]).flatten(-2)


class Case:
    """Random q and caches; pages given out in random order, the rest of the pool and of the table garbage."""

    def __init__(self, lens, Hq, Hkv, D, page, seed=0, layout="heads", q_pad=0, spare=3, factors=False):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lens)
        need = [-(-n // page) for n in lens]
        most, pages = max(max(need), 1) + 2, sum(need) + spare
        table = rng.integers(-2 ** 31, 2 ** 31 - 1, (B, most)).astype(np.int32)  # never read past a sequence's pages
        order = rng.permutation(pages)
        at = 0
        used = torch.zeros((pages, page), dtype=torch.bool)
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        for b, n in enumerate(lens):
            for j in range(need[b]):
                used[table[b, j], :min(page, n - j * page)] = True
        junk = ~used.cuda()

        def rows(cols):
            shape = {"tokens": (pages, 2, page, Hkv, cols), "heads": (pages, 2, Hkv, page, cols)}[layout]
            t = torch.zeros(shape, dtype=torch.uint8, device="cuda")
            return t if layout == "tokens" else t.transpose(2, 3)

        codes, scales = rows(D // 2), rows(D // 16)
        codes.copy_(torch.randint(0, 256, codes.shape, generator=gen, device="cuda", dtype=torch.uint8))
        s = 0.25 * torch.exp(0.7 * torch.randn(scales.shape, generator=gen, device="cuda"))
        scales.copy_(s.to(torch.float8_e4m3fn).view(torch.uint8))
        scales.view(torch.uint8)[:, 0][junk] = 0x7f  # NaN
        scales.view(torch.uint8)[:, 1][junk] = 0xff
        scales = scales.view(torch.float8_e4m3fn)
        self.cache = dict(k_cache=codes[:, 0], v_cache=codes[:, 1], k_scales=scales[:, 0], v_scales=scales[:, 1])
        self.factors = {n: torch.exp(0.5 * torch.randn(Hkv, generator=gen, device="cuda"))
                        for n in ("k_factor", "v_factor")} if factors else {}
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        buf = (1.5 * torch.randn((B, Hq * D + q_pad), generator=gen, device="cuda")).bfloat16()
        self.q = buf[:, :Hq * D].unflatten(1, (Hq, D))
        self.scale = D ** -0.5
        self.page = page

    def run(self, **kw):
        return mk.paged_attention_fp4(self.q, block_table=self.table, seq_lens=self.lens, **self.cache, **self.factors, **kw)

    def rows(self, name, b, n):
        """[n, Hkv, D] of sequence b in 64 bits."""
        pages = self.table[b, :-(-n // self.page)].long()
        scales = self.cache[name + "_scales"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)
        x = values_of(self.cache[name + "_cache"][pages], scales).flatten(0, 1)[:n]
        f = self.factors.get(name + "_factor")
        return x if f is None else x * f.double()[:, None]

    def check(self, o, scale=None):
        scale = self.scale if scale is None else scale
        B, Hq, D = self.q.shape
        Hkv = self.cache["k_cache"].shape[2]
        G = Hq // Hkv
        for b, n in enumerate(self.lens.tolist()):
            out, lse = o["out"][b].double(), o["lse"][b].double()
            if n == 0:
                assert torch.all(out == 0) and torch.all(lse == -float("inf"))
                continue
            k, v = (self.rows(x, b, n).repeat_interleave(G, 1) for x in "kv")  # [n, Hq, D]
            q = self.q[b].double()
            s = torch.einsum("hd,nhd->hn", q, k) * scale
            ds = 2.0 ** -20 * torch.einsum("hd,nhd->hn", q.abs(), k.abs()).amax(1, keepdim=True)
            ds = abs(scale) * (ds + 2.0 ** -39 * q.abs().amax(1, keepdim=True) * k.abs().sum(2).amax(0)[:, None])
            p = torch.softmax(s, 1)
            want = torch.einsum("hn,nhd->hd", p, v)
            spread = torch.einsum("hn,nhd->hd", p, v.abs())
            tol = 2.0 ** -8 * want.abs() + (4 * ds + 2.0 ** -14 + 2.0 ** -11) * spread + 2.0 ** -35 * v.abs().sum(0)
            assert torch.all((out - want).abs() <= tol), f"sequence {b} of {n} keys"
            ref = torch.logsumexp(s, 1)
            assert torch.all((lse - ref).abs() <= ds[:, 0] + 2.0 ** -15 + 2.0 ** -22 * ref.abs())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 12), (32, 8), (15, 3), (16, 1), (24, 1), (40, 2), (128, 8), (9, 1)])
def test_head_layouts(D, Hq, Hkv):
    c = Case([0, 1, 15, 16, 17, 31, 32, 33, 130, 1029], Hq, Hkv, D, 16, seed=D + Hq, factors=Hq == 15)
    c.check(c.run())


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 256])
def test_page_sizes(page):
    c = Case([5, page, page + 1, 3 * page - 1, 700, 0, 2 * page], 8, 2, 128, page, seed=page, factors=True)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("page,layout", [(1, "heads"), (3, "heads"), (8, "heads"), (8, "tokens"), (24, "heads"), (32, "heads"),
                                         (48, "heads"), (96, "tokens")])
def test_page_sizes_of_other_heads(D, page, layout):
    c = Case([5, page, page + 1, 3 * page - 1, 700, 0, 2 * page], 20, 2, D, page, seed=page, layout=layout)
    c.check(c.run())


@pytest.mark.parametrize("lens", [[1], [16], [127], [128], [129], [5000], [0], [0, 0, 0], [5999, 1], [1, 5999],
                                  [33] * 300], ids=str)
@pytest.mark.parametrize("Hkv", [1, 4])
def test_lengths(lens, Hkv):
    c = Case(lens, 4, Hkv, 64, 16, seed=len(lens) + lens[0])
    c.check(c.run())


def test_most_sequences():
    rng = np.random.default_rng(5)
    c = Case([int(n) for n in rng.integers(0, 4, 4096)], 2, 1, 64, 2, seed=6)
    c.check(c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("layout,q_pad", [("tokens", 0), ("heads", 0), ("tokens", 2048), ("heads", 8)])
def test_strides(layout, q_pad, D):
    c = Case([100, 0, 513], 16, 4, D, 32, seed=q_pad, layout=layout, q_pad=q_pad)
    c.check(c.run())


def test_scale():
    c = Case([300, 64], 8, 2, 128, 16, seed=1)
    for scale in (0.0, -0.05, 1.0):
        c.check(c.run(scale=scale), scale)


@pytest.mark.parametrize("by", [2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100])
def test_queries_of_any_size(by):
    # a power of two taken from the queries to the scale
    c = Case([300, 64], 8, 2, 128, 16, seed=1)
    want = c.run()
    c.q = (c.q.double() * by).bfloat16()
    o = c.run(scale=c.scale / by)
    for n in ("out", "lse"):
        assert torch.equal(o[n], want[n])
    c.q = c.q.clone()
    c.q[0, 0, :64] *= 2.0 ** -9  # columns of very different size in a head
    c.q[0, 1, 1:] *= 2.0 ** -24
    c.check(c.run(scale=c.scale / by), c.scale / by)


def test_growing_and_falling_scores():
    # the largest score comes first, last, or grows with every key: the weights' reference moves along
    for sign, axis in ((1, "grow"), (-1, "grow"), (1, "last"), (1, "first")):
        c = Case([999], 8, 1, 64, 16, seed=2)
        n = 999
        at = torch.arange(n, device="cuda")
        level = {"grow": at * 126 // n, "last": (at == n - 1) * 126, "first": (at == 0) * 126}[axis]
        pages, token = c.table[0, at // 16].long(), at % 16
        s = c.cache["k_scales"].view(torch.uint8)
        s[pages, token, 0] = level.to(torch.uint8)[:, None]
        codes = c.cache["k_cache"]
        codes[pages, token, 0] = 0x22  # all ones
        c.q = (sign * (1 + torch.rand_like(c.q.float()))).bfloat16()
        for scale in (0.01, 0.125):
            c.check(c.run(scale=scale), scale)


def test_repeatable_whatever_ran_before_and_on_another_stream():
    c = Case([1000, 3, 0, 2500], 32, 8, 128, 16, seed=3)
    other = Case([4000, 77], 64, 2, 64, 8, seed=4)
    a = c.run()
    other.check(other.run())
    b = c.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    d = c.run(stream=side, check=False)
    ws = torch.zeros(mk.mk_paged_attention_fp4_workspace_size(4, 32, 8), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    e = [c.run(workspace=ws, ws_bytes=ws.numel()) for _ in range(3)][-1]
    assert mk.mk_get_status(side) == mk.MK_OK
    c.check(a)
    for o in (b, d, e):
        assert torch.equal(a["out"], o["out"]) and torch.equal(a["lse"], o["lse"])


def test_workspace_and_empty_batch():
    c = Case([10], 4, 4, 64, 16)
    ws = torch.zeros(1024, dtype=torch.uint8, device="cuda")
    with pytest.raises(mk.MkError) as e:
        c.run(workspace=ws, ws_bytes=ws.numel())
    assert e.value.status == mk.MK_ERR_WORKSPACE
    o = mk.paged_attention_fp4(c.q[:0], block_table=c.table[:0], seq_lens=c.lens[:0], **c.cache)
    assert o["out"].shape == (0, 4, 64) and o["lse"].shape == (0, 4)


def test_tables_and_pools_without_pages():
    q = torch.randn((3, 8, 64), device="cuda").bfloat16()
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    for pages in (0, 4):
        z = mk.fp4_cache(pages, 16, 2, 64)
        o = mk.paged_attention_fp4(q, block_table=torch.zeros((3, 0), dtype=torch.int32, device="cuda"), seq_lens=lens, **z)
        assert torch.all(o["out"] == 0) and torch.all(o["lse"] == -float("inf"))


def test_offsets_past_32_bits():
    # a pool of more than 2^32 bytes, with the sequence in its last pages
    page, Hkv, D = 64, 8, 128
    c = Case([700], 16, Hkv, D, page, seed=7)
    n = c.table.shape[1] - 2
    pages = 2 ** 32 // (page * Hkv * D // 2) + 20
    last = torch.arange(pages - n, pages, device="cuda", dtype=torch.int32)
    big = {}
    for name, t in c.cache.items():
        big[name] = torch.empty((pages, *t.shape[1:]), dtype=torch.uint8, device="cuda")
        big[name][last.long()] = t.view(torch.uint8)[c.table[0, :n].long()]
        big[name] = big[name].view(t.dtype)
    c.cache = big
    c.table[0, :n] = last
    c.check(c.run())


def test_bad_pages_and_lengths_are_reported():
    c = Case([100, 40], 8, 2, 64, 16, seed=8)
    good = c.run()
    pages = c.cache["k_cache"].shape[0]
    for where, value in (((0, 2), -1), ((0, 2), pages), ((1, 0), 2 ** 31 - 1)):
        table = c.table.clone()
        table[where] = value
        mk.paged_attention_fp4(c.q, block_table=table, seq_lens=c.lens, check=False, **c.cache)
        assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
        assert mk.mk_last_error_detail()["info"] == value
    table = c.table.clamp(0, pages - 1)  # the whole table holds pages: the clamped length may read them
    for n in (-5, table.shape[1] * 16 + 1):
        lens = torch.tensor([n, 40], dtype=torch.int32, device="cuda")
        o = mk.paged_attention_fp4(c.q, block_table=table, seq_lens=lens, check=False, **c.cache)
        assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
        assert torch.equal(o["out"][1], good["out"][1])
    assert mk.mk_get_status() == mk.MK_OK
    assert torch.equal(c.run()["out"], good["out"])


def test_values_that_are_not_finite():
    c = Case([40, 40], 8, 2, 64, 16, seed=9)
    good = c.run()
    page = int(c.table[0, 1])
    c.cache["v_scales"].view(torch.uint8)[page, 3, 1, 2] = 0x7f  # NaN: 16 columns of one head's values
    o = c.run()["out"]
    assert torch.all(torch.isnan(o[0, 4:, 32:48]))
    o[0, 4:, 32:48] = good["out"][0, 4:, 32:48]
    assert torch.equal(o, good["out"])
    c.cache["v_scales"].view(torch.uint8)[page, 3, 1, 2] = 0x20
    good = c.run()
    c.q = c.q.clone()
    c.q[1, 2, 7], c.q[1, 6, 9] = float("nan"), float("inf")
    o = c.run()
    for n in ("out", "lse"):
        assert torch.all(torch.isnan(o[n][1, 2]))
        assert torch.all(torch.isnan(o[n][1, 6]))
        o[n][1, 2], o[n][1, 6] = good[n][1, 2], good[n][1, 6]
        assert torch.equal(o[n], good[n])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,per_kv", [(200, 17), (160, 32), (90, 33), (200, 24), (80, 64)])
def test_more_than_16_heads_and_many_sequences(B, per_kv, D):
    lens = [(i * 37) % 150 for i in range(B)]
    lens[-1], lens[B // 2] = 2000, 0
    c = Case(lens, 2 * per_kv, 2, D, 16, seed=B + per_kv)
    c.check(c.run())


@pytest.mark.parametrize("D,page", [(64, 16), (64, 8), (64, 1), (128, 16), (256, 16)])
def test_longest_sequence(D, page):
    """2^31 - 32 keys, all of them of one page, with scores of -D: a key behind the last one, whose
    score would be 0, would outweigh them all.  All weights are the same number near 2^10, so a sum of 2^18 of
    them in a lane is off by no more than that number's distance from 2^10, 2^-16 of it."""
    n = 2 ** 31 - 32
    c = mk.fp4_cache(1, page, 1, D)
    for x in ("k_cache", "v_cache"):
        c[x].fill_(0x22)  # ones
    for x in ("k_scales", "v_scales"):
        c[x].view(torch.uint8).fill_(0x38)  # of 1
    q = -torch.ones((1, 1, D), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, n // page), dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = mk.paged_attention_fp4(q, **c, block_table=table, seq_lens=lens, scale=1.0)
    assert (got["out"] == 1).all()
    want = np.log(float(n)) - D
    assert abs(got["lse"].item() - want) <= 2.0 ** -15 + 2.0 ** -22 * abs(want)
