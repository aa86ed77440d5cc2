"""The library's workspaces under the decode-step operators on a GPU: several
host threads on one stream, and calls beside a graph that holds captured ones.
What they share is counters and partial sums, so any overlap shows in the bits."""
import threading

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


def _rand(*shape, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda")


def _ffn(T, H, F, E, k, seed):
    x, logits = _rand(T, H, seed=seed).bfloat16(), _rand(T, E, seed=seed + 1)
    w = [(_rand(E, a, b, seed=seed + 2 + i) * a ** -0.5).bfloat16() for i, (a, b) in enumerate(((H, F), (H, F), (F, H)))]
    return lambda **kw: mk.moe_ffn_decode(x, logits, *w, k, check=False, **kw)["out"]


def _attention(B, n, Hq, Hkv, D, seed):
    page, per = 16, -(-n // 16)
    kv = _rand(B * per, 2, page, Hkv, D, seed=seed).bfloat16()
    q = _rand(B, Hq, D, seed=seed + 1).bfloat16()
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    return lambda **kw: mk.paged_attention(q, kv[:, 0], kv[:, 1], table, lens, check=False, **kw)["out"]


def test_threads_on_one_stream():
    # workspaces of 3 MB to 600 MB, in another order in every thread
    runs = [_ffn(2, 128, 128, 4, 2, 1), _ffn(128, 128, 8192, 8, 8, 10), _attention(3, 500, 8, 2, 64, 20),
            _ffn(128, 128, 32768, 8, 8, 30), _attention(4000, 20, 16, 16, 64, 40)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    mk.mk_release_workspace()
    seen, errors = [[] for _ in runs], []

    def work(first):
        try:
            for turn in range(4):
                for i in range(len(runs)):
                    at = (first + i * (1 + first % 2)) % len(runs)
                    seen[at].append(runs[at]())
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


@pytest.mark.parametrize("make,larger", [
    (lambda: _ffn(17, 512, 640, 16, 4, 1), lambda: _ffn(128, 128, 32768, 8, 8, 30)),
    (lambda: _attention(5, 3000, 32, 8, 128, 2), lambda: _attention(4000, 20, 16, 16, 64, 40)),
], ids=["ffn", "attention"])
def test_calls_beside_a_replayed_graph(make, larger):
    run, big = make(), larger()
    want, want_big = run(), big()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = run()
    torch.cuda.synchronize()
    for turn in range(20):
        with torch.cuda.stream(other):
            graph.replay()
        with torch.cuda.stream(side):
            eager = run()
            if turn == 10:
                eager_big = big()  # grows the stream's workspace
        torch.cuda.synchronize()
        assert torch.equal(captured, want) and torch.equal(eager, want)
    assert torch.equal(eager_big, want_big) and mk.mk_get_status() == mk.MK_OK
