"""The cache's operators together, as the example runs them: rows grow, fork,
write to shared pages, are freed, the pool is compacted, eagerly and from a CUDA
graph; and each of them beside other streams, threads and graphs.

Every row's cached keys and values, read through its table, are those that were
put there, and its attention is that over what is cached, in 64 bits.
Tolerances: a bf16 key is off by 2^-8 of itself and 2^-17 of its pair (see
test_gpu_qk_norm_rope.py); a 4-bit one by half the largest step, a scale, which
is amax / 6 and 2^-4 of that, and what limits it to 6 scales, 2^-4 of amax at
most; the attention by 2^-8 of itself and 2^-9 of the weighted |v|, more than
the sum of its own errors at these lengths (see test_gpu_attention_fp4.py)."""
import importlib
import os
import sys
import threading

import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    yield importlib.import_module("shared_prompts")
    sys.path.pop(0)
    mk.mk_release_workspace()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def unpack(codes):
    steps = torch.tensor(STEPS + [-x for x in STEPS], dtype=torch.float64, device="cuda")
    return torch.stack([steps[(codes & 15).long()], steps[(codes >> 4).long()]], -1).flatten(-2)


class Followed:
    """An attention whose rows are followed: the keys and values that each should hold."""

    def __init__(self, ex, z, seed):
        self.a, self.z = ex.Attention(z, seed), z
        self.keys = [[] for _ in range(z.rows)]
        self.values = [[] for _ in range(z.rows)]

    def held(self, row):
        a, n = self.a, int(self.a.lens[row])
        pages = a.table[row, :-(-n // self.z.page)].long()

        def part(name):
            t = a.cache[name + "_cache"][pages].flatten(0, 1)[:n]
            if not self.z.fp4:
                return t.double()
            s = a.cache[name + "_scales"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double().flatten(0, 1)[:n]
            return (unpack(t).unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)

        return part("k"), part("v")

    def step(self, x, live):
        a, z = self.a, self.z
        before = a.lens.tolist()
        out = a.step(x, live)
        assert mk.mk_get_status() == mk.MK_OK
        q, k, v = (t.unflatten(1, (-1, z.D)).double() for t in (x @ a.w_qkv).split([z.Hq * z.D, z.Hkv * z.D, z.Hkv * z.D], 1))
        angle = torch.tensor(before, dtype=torch.float64, device="cuda")[:, None, None] * a.inv_freq.double()

        def turned(y, w):
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            c, d = y.chunk(2, -1)
            return torch.cat([c * angle.cos() - d * angle.sin(), d * angle.cos() + c * angle.sin()], -1)

        q, k = turned(q, a.q_weight), turned(k, a.k_weight)
        for row in torch.nonzero(live)[:, 0].tolist():
            self.keys[row] = self.keys[row] + [k[row]]
            self.values[row] = self.values[row] + [v[row]]
        att = torch.zeros((z.rows, z.Hq, z.D), dtype=torch.float64, device="cuda")
        spread = torch.zeros_like(att)
        G = z.Hq // z.Hkv
        for row in range(z.rows):
            n = len(self.keys[row])
            assert int(a.lens[row]) == n
            if n == 0:
                continue
            hk, hv = self.held(row)
            for got, want in ((hk, torch.stack(self.keys[row])), (hv, torch.stack(self.values[row]))):
                off = (got - want).abs()
                if z.fp4:
                    top = want.unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
                    assert torch.all(off <= top * (1 + 2.0 ** -4) / 6 + 2.0 ** -10)
                else:
                    pair = want.abs() + want.roll(z.D // 2, -1).abs()
                    assert torch.all(off <= 2.0 ** -8 * want.abs() + 2.0 ** -17 * pair)
            qr = q[row].bfloat16().double()
            s = torch.einsum("hd,nhd->hn", qr, hk.repeat_interleave(G, 1)) * z.D ** -0.5
            p = torch.softmax(s, 1)
            att[row] = torch.einsum("hn,nhd->hd", p, hv.repeat_interleave(G, 1))
            spread[row] = torch.einsum("hn,nhd->hd", p, hv.repeat_interleave(G, 1).abs())
        # through the output's projection: the rows' errors add up by their norms at most
        want = att.flatten(1) @ a.w_o.double()
        tol = (2.0 ** -8 * att.abs() + 2.0 ** -9 * spread + 2.0 ** -7 * spread).flatten(1).norm(dim=1) * a.w_o.double().norm(dim=0).max()
        assert torch.all((out.double() - want).norm(dim=1) <= (tol * z.H ** 0.5) + 2.0 ** -8 * want.norm(dim=1))
        return out

    def fork(self, parents, children):
        self.a.fork(i32(parents), i32(children))
        keys, values = list(self.keys), list(self.values)
        for p, c in zip(parents, children):
            self.keys[c], self.values[c] = keys[p], values[p]

    def free(self, rows):
        self.a.free(i32(rows))
        for r in rows:
            self.keys[r], self.values[r] = [], []


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "fp4"])
@pytest.mark.parametrize("page,D", [(4, 64), (1, 64), (8, 128), (16, 64)])
def test_prompts_completions_and_compaction(ex, fp4, page, D):
    z = ex.Sizes(H=256, Hq=8, Hkv=2, D=D, page=page, pages=160, rows=7, longest=40, fp4=fp4)
    f = Followed(ex, z, seed=page + D)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def step(live):
        f.step(torch.randn((z.rows, z.H), generator=gen, device="cuda").bfloat16(), i32(live))

    for _ in range(6):
        step([1, 1, 0, 0, 0, 0, 0])
    f.fork([0, 0, 1], [2, 3, 4])
    step([0, 1, 1, 1, 0, 1, 0])
    step([1, 1, 1, 1, 1, 1, 1])
    f.fork([2, 3], [3, 2])  # one another's
    step([1, 1, 1, 1, 0, 0, 1])
    f.free([0, 4])
    f.a.compact()
    used = int((f.a.refs > 0).sum())
    assert torch.all(f.a.refs[:used] > 0) and torch.all(f.a.refs[used:] == 0)
    for _ in range(3):
        step([1, 1, 1, 1, 0, 1, 1])
    f.free([0, 1, 2, 3, 4, 5, 6])
    assert torch.all(f.a.refs == 0)
    step([0, 0, 0, 1, 0, 0, 0])
    assert mk.mk_get_status() == mk.MK_OK


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "fp4"])
def test_graph_replays_the_same_steps(ex, fp4):
    z = ex.Sizes(H=256, Hq=8, Hkv=2, D=64, page=4, pages=80, rows=5, longest=40, fp4=fp4)
    one, two = ex.Attention(z, 1), ex.Attention(z, 1)
    x, live = torch.randn(5, z.H, device="cuda").bfloat16(), i32([1, 1, 0, 1, 1])
    for a in (one, two):
        a.step(x, live)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        two.step(x, live)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = two.step(x, live)
    torch.cuda.synchronize()
    one.step(x, live)
    for _ in range(6):
        want = one.step(x, live)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out)
    assert torch.equal(one.lens, two.lens) and torch.equal(one.table, two.table) and torch.equal(one.refs, two.refs)
    for n in one.cache:
        assert torch.equal(one.cache[n].view(torch.uint8), two.cache[n].view(torch.uint8))
    assert mk.mk_get_status() == mk.MK_OK


# ------------------------------------------------ streams, threads, graphs --

LONG = 100_000_000  # clocks of a busy stream: 50 ms


def _rand(*shape, seed):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def _rope():
    x = _rand(500, 24 * 128, seed=1).bfloat16()
    q, k, v = (t.unflatten(1, (-1, 128)) for t in x.split([16 * 128, 4 * 128, 4 * 128], 1))
    pos, inv = torch.arange(500, dtype=torch.int32, device="cuda"), _rand(64, seed=2).abs()
    return [q, k, pos, inv], lambda t, **kw: mk.qk_norm_rope(*t, check=False, **kw)["q"]


def _attention4(B=64, n=300, Hq=16, Hkv=4, D=128):
    z = mk.fp4_cache(B * -(-n // 16), 16, Hkv, D)
    for i, t in enumerate(z.values()):
        t.view(torch.uint8).copy_(torch.randint(0, 90, t.shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda"))
    table = torch.arange(B * -(-n // 16), dtype=torch.int32, device="cuda").view(B, -1)
    t = [_rand(B, Hq, D, seed=3).bfloat16(), *z.values(), table, torch.full((B,), n, dtype=torch.int32, device="cuda")]
    return t, lambda t, **kw: mk.paged_attention_fp4(*t, check=False, **kw)["out"]


def _compact():
    refs = (_rand(5000, seed=4) > 0).to(torch.int32)
    table = torch.nonzero(refs)[:, 0].to(torch.int32)[None].contiguous()
    lens = i32([table.shape[1] * 2])
    return [table, lens, refs], lambda t, **kw: mk.compact_pages(*t, [], 2, check=False, **kw)["block_table"]


CASES = [_rope, _attention4, _compact]


def _bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("case", CASES)
def test_outputs_have_no_earlier_work_pending(case, form):
    tensors, run = case()
    side = torch.cuda.Stream()
    given = side if form == "stream" else side.cuda_stream
    want = run(tensors)
    run(tensors, stream=given)  # the stream's workspace
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.empty_like(want)
    torch.cuda._sleep(LONG)
    old.fill_(7)  # when the other stream has long been done
    del old
    out = run(tensors, stream=given)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(_bits(out), _bits(want))


@pytest.mark.parametrize("case", CASES)
def test_inputs_stay_while_the_call_runs(case):
    tensors, run = case()
    side = torch.cuda.Stream()
    want = run(tensors)
    run(tensors, stream=side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    shapes = [(t.shape, t.dtype) for t in tensors]
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    out = run(tensors, stream=side)
    tensors.clear()
    others = [torch.zeros(s, dtype=torch.uint8 if d is torch.float8_e4m3fn else d, device="cuda") for s, d in shapes]
    torch.cuda.synchronize()
    assert torch.equal(_bits(out), _bits(want)) and len(others) == len(shapes)


@pytest.mark.parametrize("case", CASES)
def test_refuses_tensors_of_a_device_that_is_not_current(case, monkeypatch):
    tensors, run = case()
    run(tensors)
    monkeypatch.setattr(mk, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        run(tensors)


def test_capture_does_not_grow_the_workspace():
    mk.mk_release_workspace()
    tensors, run = _attention4(3, 40, 8, 2, 64)
    ws = torch.zeros(mk.mk_paged_attention_fp4_workspace_size(3, 8, 2), dtype=torch.uint8, device="cuda")
    pool, compact = _compact()
    torch.cuda.synchronize()
    graph, stream, seen = torch.cuda.CUDAGraph(), torch.cuda.Stream(), []
    with torch.cuda.graph(graph, stream=stream):
        for t, f in ((tensors, run), (pool, compact)):
            try:
                f(t)
            except mk.MkError as e:
                seen.append(e.status)
        out = run(tensors, workspace=ws, ws_bytes=ws.numel())
    graph.replay()
    torch.cuda.synchronize()
    assert seen == [mk.MK_ERR_WORKSPACE] * 2
    assert torch.equal(out, run(tensors))


def test_threads_on_one_stream_and_calls_beside_a_graph():
    runs = [_attention4(), _attention4(4000, 20, 16, 16, 64), _attention4(2, 5000, 32, 8, 128), _compact(), _rope()]
    want = [run(t) for t, run in runs]
    torch.cuda.synchronize()
    mk.mk_release_workspace()
    seen, errors = [[] for _ in runs], []

    def work(first):
        try:
            for _ in range(4):
                for i in range(len(runs)):
                    at = (first + i * (1 + first % 2)) % len(runs)
                    seen[at].append(runs[at][1](runs[at][0]))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and mk.mk_get_status() == mk.MK_OK
    for outs, w in zip(seen, want):
        assert outs and all(torch.equal(o, w) for o in outs)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    (t, run), (big, run_big) = runs[2], runs[1]
    with torch.cuda.stream(side):
        run(t)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = run(t)
    torch.cuda.synchronize()
    for turn in range(10):
        with torch.cuda.stream(other):
            graph.replay()
        with torch.cuda.stream(side):
            eager = run(t)
            if turn == 5:
                eager_big = run_big(big)  # grows the stream's workspace
        torch.cuda.synchronize()
        assert torch.equal(captured, want[2]) and torch.equal(eager, want[2])
    assert torch.equal(eager_big, want[1]) and mk.mk_get_status() == mk.MK_OK
