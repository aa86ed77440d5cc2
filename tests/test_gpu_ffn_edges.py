"""mk_moe_ffn_decode at the edges of its own plan: blocks of h that several warps
complete, experts that are chosen but masked.  Layers, reference and tolerances are those of
test_gpu_ffn_decode.py."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk
from test_gpu_ffn_decode import Layer

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


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,H,F,E,k", [(50, 256, 512, 3, 2), (60, 2048, 1024, 2, 2), (128, 1024, 2048, 8, 4)])
def test_rows_completed_by_several_warps_are_seen(T, H, F, E, k, fp8):
    # one to many pieces of h; the blocks' rows are published by the last of three warps
    layer = Layer(T, H, F, E, k, fp8, seed=T + F)
    outs = [layer.run(check=False) for _ in range(100)]
    assert mk.mk_get_status() == mk.MK_OK
    layer.check(outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,H,F", [(1, 1024, 1024), (5, 256, 384), (40, 256, 384), (128, 256, 256)])
def test_masked_experts_are_not_used(T, H, F, fp8):
    # fewer live experts than k: the others' weights may hold anything
    gen = torch.Generator().manual_seed(T)
    E, k, live = 12, 4, [3, 7, 8]
    logits = torch.full((T, E), -float("inf"))
    logits[:, live] = torch.randn((T, len(live)), generator=gen)
    if T > 1:
        logits[1] = -float("inf")          # no expert at all
        logits[2, [3, 7]] = -float("inf")  # one
    logits[0, 8] = -200.0                  # a gate that is 0 in 32 bits, of an expert that is used
    layer = Layer(T, H, F, E, k, fp8, seed=T, logits=logits)
    want = layer.run()
    layer.check(want)
    dead = [e for e in range(E) if e not in live]
    for w in (layer.W1, layer.W3, layer.W2):
        w.view(torch.uint8)[dead] = 0x7f if fp8 else 0xff  # NaN
    out = layer.run()
    assert torch.equal(out, want)
    if T > 1:
        assert torch.all(out[1] == 0)


@pytest.mark.parametrize("T", [1, 9, 100])
def test_every_expert_masked(T):
    layer = Layer(T, 256, 320, 8, 2, seed=1, logits=torch.full((T, 8), -float("inf")))
    for w in (layer.W1, layer.W3, layer.W2):
        w.fill_(float("nan"))
    for _ in range(3):
        assert torch.all(layer.run() == 0)
