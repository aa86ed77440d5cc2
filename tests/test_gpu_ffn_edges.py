"""mk_moe_ffn_decode at the edges of its own plan: blocks of h that several warps
complete, experts that are chosen but masked.  Layers, reference and tolerances are those of
test_gpu_ffn_decode.py."""
import math

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


@pytest.mark.parametrize("T", [3, 40])
def test_infinite_weights_of_the_second_half(T):
    # h enters the product in two parts: both have its sign
    layer = Layer(T, 256, 320, 1, 1, seed=T)
    want = layer.run()
    x = layer.x.double()
    a = x @ layer.W1[0].double()
    h = a * torch.sigmoid(a) * (x @ layer.W3[0].double())
    layer.W2[0, 37, 100], layer.W2[0, 250, 9], layer.W2[0, 11, 200] = float("inf"), -float("inf"), float("nan")
    out = layer.run()
    rest = [c for c in range(256) if c not in (100, 9, 200)]
    assert torch.equal(out[:, rest], want[:, rest])
    assert torch.equal(out[:, 100].double(), torch.sign(h[:, 37]) * float("inf"))
    assert torch.equal(out[:, 9].double(), torch.sign(h[:, 250]) * -float("inf"))
    assert torch.all(torch.isnan(out[:, 200]))


def test_hidden_values_next_to_the_largest():
    # h between the largest bf16 and the largest 32-bit value is finite, and times a small weight so is the output
    layer = Layer(2, 64, 64, 1, 1, seed=3)
    for w in (layer.W1, layer.W3, layer.W2):
        w.zero_()
    layer.x.zero_()
    layer.x[:, 0] = 1.0
    layer.x[:, 1] = 2.0 ** -9
    big = 2.0 ** 65 * (2 - 2.0 ** -7)
    layer.W1[0, 0, 5], layer.W1[0, 1, 5] = big, 2.0 ** 65 * 2.5
    layer.W3[0, 0, 5] = 2.0 ** 62
    layer.W2[0, 5, 7] = 2.0 ** -100
    h = (big + 2.0 ** -9 * 2.0 ** 65 * 2.5) * 2.0 ** 62
    assert (2 - 2.0 ** -8) * 2.0 ** 127 < h < (2 - 2.0 ** -23) * 2.0 ** 127  # nearest in bf16 is infinity
    out = layer.run().double()
    assert torch.all((out[:, 7] - h * 2.0 ** -100).abs() <= 2.0 ** -8 * h * 2.0 ** -100)
    assert torch.all(out[:, [c for c in range(64) if c != 7]] == 0)


@pytest.mark.parametrize("a", [-88.0, -80.0, -20.0])
@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_large_denominators_of_the_gate(fp8, a):
    # 1 + e^-a is up to 2^127: silu(a) is tiny, its product with a large second factor is not
    layer = Layer(3, 128, 128, 1, 1, fp8, seed=5)
    layer.x, layer.W1, layer.W3, layer.W2 = (torch.zeros(s, device="cuda") for s in ((3, 128), *[(1, 128, 128)] * 3))
    layer.x[:, 0] = 1.0
    layer.W1[0, 0, 0], layer.W3[0, 0, 0], layer.W2[0, 0, 0] = 2 * a, 1.0, 1.0
    scale = {"W1": 0.5, "W3": 2.0 ** 120, "W2": 1.0}
    for n, s in scale.items():
        w = getattr(layer, n)
        setattr(layer, n, w.to(torch.float8_e4m3fn) if fp8 else (w * s).bfloat16())
        layer.scales[n + "_scale"] = torch.full((1, 1, 1), s, device="cuda")
    layer.x = layer.x.to(torch.float8_e4m3fn) if fp8 else layer.x.bfloat16()
    layer.scales = {**layer.scales, "x_scale": torch.ones(3, 1, device="cuda")} if fp8 else {}
    h = a / (1 + math.exp(-a)) * 2.0 ** 120
    out = layer.run()[:, 0].double()
    # the largest h of its group is 448 in 8 bits: its e4m3 value is exact up to the scale's own rounding
    assert torch.all((out - h).abs() <= (2.0 ** -8 + 2.0 ** -14) * abs(h))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [14, 15, 16, 17])
def test_every_cta_routes_or_they_share(T, fp8):
    # a CTA has 15 warps: up to 15 tokens each routes all of them, with more they divide them
    layer = Layer(T, 256, 384, 9, 3, fp8, seed=T)
    layer.check(layer.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 3, 4, 5, 16, 17, 48, 49, 63, 64, 65, 68, 127, 128])
def test_rows_of_an_expert(rows, fp8):
    # 64 rows are multiplied together, an expert with more is taken in parts; rows are loaded in fours and single ones
    T = max(rows, 70)
    logits = torch.zeros((T, 5))
    logits[:rows, 2], logits[rows:, 4] = 3.0, 3.0
    layer = Layer(T, 256, 384, 5, 1, fp8, seed=rows, logits=logits)
    layer.check(layer.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_workspace_ready(fp8):
    # a count of pieces that is never reached: the first block of h is not published, the
    # products of W2 wait for it within their limit (2 s) and every warp of every CTA ends
    layer = Layer(20, 512, 1024, 8, 2, fp8, seed=1)
    want = layer.run()
    bytes_ = mk.mk_moe_ffn_decode_workspace_size(20, 512, 1024, 8, 2, mk.MK_WEIGHT_E4M3 if fp8 else mk.MK_WEIGHT_BF16)
    ws = torch.zeros(bytes_ // 4, dtype=torch.int32, device="cuda")
    first_count = 64 + 256 + 1024 // 64  # after the control words and the parts' counters
    ws[first_count] = 1000
    layer.run(workspace=ws, ws_bytes=bytes_, check=False)
    assert mk.mk_get_status() == mk.MK_ERR_TIMEOUT
    assert mk.mk_last_error_detail()["site"] == 4  # waiting for a part's h
    assert mk.mk_get_status() == mk.MK_OK  # reading the status cleared it
    assert not torch.any(ws[:first_count + 4096])  # every counter is 0 again
    for _ in range(2):
        assert torch.equal(layer.run(workspace=ws, ws_bytes=bytes_), want)
    layer.check(want)
