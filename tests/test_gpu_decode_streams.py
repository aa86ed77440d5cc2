"""Memory of the decode-step operators' tensor forms when they run on another
stream than the current one: what they allocate has no earlier work pending on
it, and what they read or write is not handed out while they run."""
import pytest
import torch

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

LONG = 100_000_000  # clocks of a busy stream: 50 ms


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _rand(*shape, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def _norm():
    x, w = _rand(512, 4096, seed=1), _rand(4096, seed=2)
    return [x, w], lambda t, **kw: mk.add_rmsnorm(t[0], t[1], check=False, **kw)["out"]


def _attention():
    B, pages = 64, 128
    q, k, v = _rand(B, 64, 256, seed=3), _rand(pages, 16, 4, 256, seed=4), _rand(pages, 16, 4, 256, seed=5)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, 2)
    lens = torch.full((B,), 29, dtype=torch.int32, device="cuda")
    return [q, k, v, table, lens], lambda t, **kw: mk.paged_attention(*t, check=False, **kw)["out"]


def _ffn():
    x, w1, w3, w2 = _rand(128, 8192, seed=6), *(_rand(4, a, b, seed=s) for a, b, s in
                                                ((8192, 64, 7), (8192, 64, 8), (64, 8192, 9)))
    logits = _rand(128, 4, seed=10).float()
    return [x, logits, w1, w3, w2], lambda t, **kw: mk.moe_ffn_decode(*t, 2, check=False, **kw)["out"]


def _side(form):
    s = torch.cuda.Stream()
    return s, s if form == "stream" else s.cuda_stream


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("case", [_norm, _attention, _ffn])
def test_outputs_have_no_earlier_work_pending(case, form):
    tensors, run = case()
    side, given = _side(form)
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


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("case", [_norm, _attention, _ffn])
def test_inputs_stay_while_the_call_runs(case, form):
    tensors, run = case()
    side, given = _side(form)
    want = run(tensors)
    run(tensors, stream=given)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    shapes = [(t.shape, t.dtype) for t in tensors]
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    out = run(tensors, stream=given)
    tensors.clear()
    others = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes]  # where the inputs were, if they could
    torch.cuda.synchronize()
    assert torch.equal(_bits(out), _bits(want)) and len(others) == len(shapes)


@pytest.mark.parametrize("case", [_norm, _attention, _ffn])
def test_outputs_stay_while_the_current_stream_uses_them(case):
    tensors, run = case()
    side = torch.cuda.Stream()
    want = run(tensors)
    run(tensors, stream=side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out = run(tensors, stream=side)
    side.synchronize()
    torch.cuda._sleep(LONG)
    seen = out.clone()  # on the current stream, after the other has gone on
    shape = out.shape
    del out
    with torch.cuda.stream(side):
        other = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(_bits(seen), _bits(want)) and other.shape == shape


@pytest.mark.parametrize("case", [_norm, _attention, _ffn])
def test_refuses_tensors_of_a_device_that_is_not_current(case, monkeypatch):
    # the kernel would run on the current device, with the other's addresses
    tensors, run = case()
    run(tensors)
    monkeypatch.setattr(mk, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        run(tensors)
