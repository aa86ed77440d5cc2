"""The example's decode step: several steps of a block against the same step in
64 bits, eager and replayed from a CUDA graph.

Tolerance.  Both sides round to bf16 at the same places (two norms, the
projections, the attention, the residual, the experts' output), from values
that differ by the rounding before; each of the seven roundings is off by 2^-8
of a value at most, 2^-9 on average, and the norms keep relative errors as they
are.  Seven in a row stay below 7 * 2^-8 of the result's norm."""
import importlib
import os
import sys

import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 7 * 2.0 ** -8


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    yield importlib.import_module("decode_step")
    sys.path.pop(0)
    mk.mk_release_workspace()


def _b(v):
    return v.float().bfloat16().double()


def _norm(v, w):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * w.double()


class Plain:
    """The same block in 64 bits on the CPU, rounding where the example's tensors are bf16 (or e4m3)."""

    def __init__(self, block):
        self.block, self.z = block, block.z
        self.k = [torch.empty((0, block.z.Hkv, block.z.D), dtype=torch.float64) for _ in range(block.batch)]
        self.v = [t.clone() for t in self.k]
        self.cpu = {n: getattr(block, n).double().cpu() for n in ("w_in", "w_post", "w_qkv", "w_o", "w_router")}

    def weight(self, name, e):
        x = self.block.experts
        w = x[name][e].double().cpu()
        if self.z.fp8:
            s = x[name + "_scale"][e].double().cpu()
            w = w * s.repeat_interleave(128, 0).repeat_interleave(128, 1)
        return w

    def q8(self, v):
        g = v.view(v.shape[0], -1, 128)
        s = g.abs().amax(2, keepdim=True) / 448
        return ((g / s).to(torch.float8_e4m3fn).double() * s).view_as(v)

    def step(self, x, residual):
        z, c = self.z, self.cpu
        stream = x + residual
        qkv = _b(_b(_norm(stream, c["w_in"])) @ c["w_qkv"])
        stream = _b(stream)
        q, k, v = qkv.split([z.Hq * z.D, z.Hkv * z.D, z.Hkv * z.D], dim=1)
        att = torch.empty_like(q)
        for b in range(x.shape[0]):
            self.k[b] = torch.cat([self.k[b], k[b].view(1, z.Hkv, z.D)])
            self.v[b] = torch.cat([self.v[b], v[b].view(1, z.Hkv, z.D)])
            G = z.Hq // z.Hkv
            kk, vv = self.k[b].repeat_interleave(G, 1), self.v[b].repeat_interleave(G, 1)
            s = torch.einsum("hd,nhd->hn", q[b].view(z.Hq, z.D), kk) * z.D ** -0.5
            att[b] = torch.einsum("hn,nhd->hd", torch.softmax(s, 1), vv).flatten()
        y = _b(_b(att) @ c["w_o"]) + stream
        n = _norm(y, c["w_post"])
        logits = _b(n) @ c["w_router"]
        xe = self.q8(n) if z.fp8 else _b(n)
        out = torch.zeros_like(x)
        top, chosen = torch.topk(logits, z.k, dim=1)
        gate = torch.softmax(top, 1)
        for b in range(x.shape[0]):
            for j in range(z.k):
                e = int(chosen[b, j])
                a = xe[b] @ self.weight("W1", e)
                h = a * torch.sigmoid(a) * (xe[b] @ self.weight("W3", e))
                if z.fp8:
                    h = self.q8(h[None])[0]
                out[b] += gate[b, j] * (h @ self.weight("W2", e))
        return _b(out), _b(y), logits


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_steps(ex, fp8):
    z = ex.Sizes(H=256, Hq=8, Hkv=2, D=64, F=256, E=8, k=2, page=4, fp8=fp8)
    block = ex.Block(z, 5, 16, seed=1)
    plain = Plain(block)
    gen = torch.Generator().manual_seed(2)
    for _ in range(6):
        x, r = (torch.randn((5, z.H), generator=gen).bfloat16() for _ in range(2))
        out, stream = block.step(x.cuda(), r.cuda())
        want, want_stream, logits = plain.step(x.double(), r.double())
        assert mk.mk_get_status() == mk.MK_OK
        assert (stream.double().cpu() - want_stream).norm() <= TOL * want_stream.norm()
        # rows whose k-th and next logit are too close to tell apart may take other experts
        best = logits.sort(1, descending=True).values
        clear = best[:, z.k - 1] - best[:, z.k] > 0.05
        err = (out.double().cpu() - want)[clear].norm() / want[clear].norm()
        # 8 bits: a value next to a boundary may round to the other side, one step of 2^-3
        assert clear.sum() >= 2 and err <= (TOL if not fp8 else 2.0 ** -4)


def test_graph_replays_the_same_steps(ex):
    z = ex.Sizes(H=256, Hq=8, Hkv=2, D=64, F=384, E=16, k=4, page=16)
    x = torch.randn((7, z.H), device="cuda").bfloat16()
    r = torch.randn((7, z.H), device="cuda").bfloat16()
    one, two = ex.Block(z, 7, 64, seed=3), ex.Block(z, 7, 64, seed=3)
    graph, out = ex.capture(two, x, r)
    for _ in range(5):
        want = one.step(x, r)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert torch.equal(one.lens, two.lens) and torch.equal(one.cache, two.cache)
    assert mk.mk_get_status() == mk.MK_OK


def test_capture_does_not_grow_the_workspace():
    mk.mk_release_workspace()
    q = torch.randn((1, 4, 64), device="cuda").bfloat16()
    kv = torch.randn((2, 2, 16, 4, 64), device="cuda").bfloat16()
    k, v = kv[:, 0], kv[:, 1]
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    ws = torch.zeros(mk.mk_paged_attention_workspace_size(1, 4, 4), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph, stream, seen = torch.cuda.CUDAGraph(), torch.cuda.Stream(), []
    with torch.cuda.graph(graph, stream=stream):
        try:
            mk.paged_attention(q, k, v, table, lens, check=False)
        except mk.MkError as e:
            seen.append(e.status)
        out = mk.paged_attention(q, k, v, table, lens, workspace=ws, ws_bytes=ws.numel(), check=False)
    graph.replay()
    torch.cuda.synchronize()
    assert seen == [mk.MK_ERR_WORKSPACE]
    want = mk.paged_attention(q, k, v, table, lens)
    assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])
