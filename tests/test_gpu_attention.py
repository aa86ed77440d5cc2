"""mk_paged_attention against the softmax in 64 bits: head layouts, page sizes
from one key up, lengths around tiles and pages, strided caches, sequences
without keys, garbage in every place that must not be read, faults that the
kernel's own checks turn into a status.

Tolerances.  A score is a sum of D products in fp32: off by at most
ds = 2^-20 * scale * sum |q_i k_i| (16 steps of 2^-24).  A weight e^(s - m) is
then off by 2 ds of itself (its own score and the maximum), the exponential by
2^-21, its two-part bf16 form by 2^-17, and the sums over at most 6000 keys by
2^-16: together less than 2 ds + 2^-15 of the weight, once in the sum of
values and once in the denominator.  Rounding the output adds 2^-8 of it; lse
is off by ds plus 2^-15, and 2^-22 of itself."""
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


class Case:
    """Random q and caches; pages given out in random order, the rest of the pool and of the table garbage."""

    def __init__(self, lens, Hq, Hkv, D, page, seed=0, layout="tokens", q_pad=0, spare=3):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lens)
        need = [-(-n // page) for n in lens]
        most, pages = max(max(need), 1) + 2, sum(need) + spare
        shape = {"tokens": (pages, 2, page, Hkv, D), "heads": (pages, 2, Hkv, page, D)}[layout]
        kv = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
        if layout == "heads":
            kv = kv.transpose(2, 3)
        self.k, self.v = kv[:, 0], kv[:, 1]
        table = rng.integers(-2 ** 31, 2 ** 31 - 1, (B, most)).astype(np.int32)  # never read past a sequence's pages
        order = rng.permutation(pages)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        used = torch.zeros((pages, page), dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(need[b]):
                used[table[b, j], :min(page, n - j * page)] = True
        junk = ~used.cuda()
        self.k[junk] = float("nan")
        self.v[junk] = float("inf")
        self.table = torch.from_numpy(table).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        buf = (1.5 * torch.randn((B, Hq * D + q_pad), generator=gen, device="cuda")).bfloat16()
        self.q = buf[:, :Hq * D].view(B, Hq, D) if q_pad == 0 else buf[:, :Hq * D].unflatten(1, (Hq, D))
        self.scale = D ** -0.5
        self.page = page

    def run(self, **kw):
        return mk.paged_attention(self.q, self.k, self.v, self.table, self.lens, **kw)

    def check(self, o, scale=None):
        scale = self.scale if scale is None else scale
        B, Hq, D = self.q.shape
        Hkv = self.k.shape[2]
        G = Hq // Hkv
        for b, n in enumerate(self.lens.tolist()):
            out, lse = o["out"][b].double(), o["lse"][b].double()
            if n == 0:
                assert torch.all(out == 0) and torch.all(lse == -float("inf"))
                continue
            pages = self.table[b, :-(-n // self.page)].long()
            k = self.k[pages].flatten(0, 1)[:n].double().repeat_interleave(G, 1)  # [n, Hq, D]
            v = self.v[pages].flatten(0, 1)[:n].double().repeat_interleave(G, 1)
            q = self.q[b].double()
            s = torch.einsum("hd,nhd->hn", q, k) * scale
            ds = 2.0 ** -20 * abs(scale) * torch.einsum("hd,nhd->hn", q.abs(), k.abs()).amax(1, keepdim=True)
            p = torch.softmax(s, 1)
            want = torch.einsum("hn,nhd->hd", p, v)
            spread = torch.einsum("hn,nhd->hd", p, v.abs())
            tol = 2.0 ** -8 * want.abs() + 2 * (2 * ds + 2.0 ** -15) * spread
            assert torch.all((out - want).abs() <= tol), f"sequence {b} of {n} keys"
            ref = torch.logsumexp(s, 1)
            assert torch.all((lse - ref).abs() <= ds[:, 0] + 2.0 ** -15 + 2.0 ** -22 * ref.abs())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 12), (32, 8), (15, 3), (16, 1), (24, 1), (40, 2), (128, 8)])
def test_head_layouts(D, Hq, Hkv):
    c = Case([0, 1, 15, 16, 17, 130, 1029], Hq, Hkv, D, 16, seed=D + Hq)
    c.check(c.run())


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 256])
def test_page_sizes(page):
    c = Case([5, page, page + 1, 3 * page - 1, 700, 0, 2 * page], 8, 2, 128, page, seed=page)
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


@pytest.mark.parametrize("layout,q_pad", [("tokens", 0), ("heads", 0), ("tokens", 2048), ("heads", 6)])
def test_strides(layout, q_pad):
    c = Case([100, 0, 513], 16, 4, 128, 32, seed=q_pad, layout=layout, q_pad=q_pad)
    c.check(c.run())


def test_scale():
    c = Case([300, 64], 8, 2, 128, 16, seed=1)
    for scale in (0.0, -0.05, 1.0):
        c.check(c.run(scale=scale), scale)


def test_large_scores_keep_the_largest():
    # one score far above the rest: the others' weights vanish, nothing overflows
    c = Case([400], 4, 1, 64, 16, seed=2)
    page, token = int(c.table[0, 7]), 5
    c.k[page, token, 0] = c.q[0, 2].float().mul(200).bfloat16()
    o = c.run()
    assert torch.all(torch.isfinite(o["out"].float())) and torch.all(torch.isfinite(o["lse"]))
    want = c.v[page, token, 0].float()
    assert torch.all((o["out"][0, 2].float() - want).abs() <= 2.0 ** -8 * want.abs())


def test_repeatable_whatever_ran_before_and_on_another_stream():
    c = Case([1000, 3, 0, 2500], 32, 8, 128, 16, seed=3)
    other = Case([4000, 77], 64, 2, 64, 8, seed=4)
    a = c.run()
    other.check(other.run())
    b = c.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    d = c.run(stream=side, check=False)
    ws = torch.zeros(mk.mk_paged_attention_workspace_size(4, 32, 8), dtype=torch.uint8, device="cuda")
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
    o = mk.paged_attention(c.q[:0], c.k, c.v, c.table[:0], c.lens[:0])
    assert o["out"].shape == (0, 4, 64) and o["lse"].shape == (0, 4)


def test_offsets_past_32_bits():
    # a pool of more than 2^32 elements, with the sequence in its last pages
    page, Hkv, D = 64, 8, 128
    pages = 2 ** 32 // (2 * page * Hkv * D) + 20
    kv = torch.empty((pages, 2, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    c = Case([700], 16, Hkv, D, page, seed=7)
    n = c.table.shape[1] - 2
    last = torch.arange(pages - n, pages, device="cuda", dtype=torch.int32)
    kv[last.long(), 0] = c.k[c.table[0, :n].long()]
    kv[last.long(), 1] = c.v[c.table[0, :n].long()]
    c.k, c.v = kv[:, 0], kv[:, 1]
    c.table[0, :n] = last
    c.check(c.run())


def test_bad_pages_and_lengths_are_reported():
    c = Case([100, 40], 8, 2, 64, 16, seed=8)
    good = c.run()
    for where, value in (((0, 2), -1), ((0, 2), c.k.shape[0]), ((1, 0), 2 ** 31 - 1)):
        table = c.table.clone()
        table[where] = value
        mk.paged_attention(c.q, c.k, c.v, table, c.lens, check=False)
        assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
        assert mk.mk_last_error_detail()["info"] == value
    table = c.table.clamp(0, c.k.shape[0] - 1)  # the whole table holds pages: the clamped length may read them
    for n in (-5, table.shape[1] * 16 + 1):
        lens = torch.tensor([n, 40], dtype=torch.int32, device="cuda")
        o = mk.paged_attention(c.q, c.k, c.v, table, lens, check=False)
        assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
        assert torch.equal(o["out"][1], good["out"][1])
    assert mk.mk_get_status() == mk.MK_OK
    assert torch.equal(c.run()["out"], good["out"])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,per_kv", [(200, 17), (160, 32), (90, 33), (200, 24), (80, 64)])
def test_more_than_16_heads_and_many_sequences(B, per_kv, D):
    lens = [(i * 37) % 150 for i in range(B)]
    lens[-1], lens[B // 2] = 2000, 0
    c = Case(lens, 2 * per_kv, 2, D, 16, seed=B + per_kv)
    c.check(c.run())
