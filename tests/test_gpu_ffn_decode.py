"""mk_moe_ffn_decode against the layer's formulas in 64 bits: token counts from
one to 128, odd expert counts, sizes that end inside a tile, skewed, masked
and equal logits, both weight types; repeatable bits; workspaces.

Tolerances, relative to a[t,c] = sum_j gate_j sum_f |h| |W2| and, through h, to
the same kind of bound of the first products.  fp32 sums of H <= 8192 terms in
groups inside the tensor core are off by less than 2^-14 of their sum of
magnitudes at the very worst and about 2^-20 in fact; the bounds below allow
2^-16.  16 bits: h as two bf16 values keeps 2^-16 of h.  8 bits: h is rounded
to e4m3; the kernel's h differs from the exact one by the above, so a value
next to a rounding boundary may go to the other side: the reference rounds h
itself and allows that one step (2^-3 of the value) where its own h lies within
2^-14 of a boundary.  The output's rounding adds 2^-8 of the value."""
import numpy as np
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()


def _blocks(s):
    return s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


def _to_e4m3(gen, rows, cols, E):
    w = torch.randn((E, rows, cols), generator=gen, device="cuda") * rows ** -0.5
    s = w.view(E, rows // 128, 128, cols // 128, 128).abs().amax((2, 4)) / 448
    s = s * (0.5 + torch.rand(s.shape, generator=gen, device="cuda"))  # no block fills its range exactly
    return (w / s.repeat_interleave(128, 1).repeat_interleave(128, 2)).clamp(-448, 448).to(torch.float8_e4m3fn), s


class Layer:
    def __init__(self, T, H, F, E, k, fp8=False, seed=0, logits=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.F, self.E, self.k, self.fp8 = T, H, F, E, k, fp8
        x = torch.randn((T, H), generator=gen, device="cuda")
        self.logits = torch.randn((T, E), generator=gen, device="cuda") if logits is None else logits.cuda()
        self.scales = {}
        if fp8:
            o = mk.add_rmsnorm(x.bfloat16(), torch.ones(H, device="cuda").bfloat16(), bf16=False, e4m3=True)
            self.x, self.scales["x_scale"] = o["out8"], o["scale"]
            for n, r, c in (("W1", H, F), ("W3", H, F), ("W2", F, H)):
                w, self.scales[n + "_scale"] = _to_e4m3(gen, r, c, E)
                setattr(self, n, w)
        else:
            self.x = x.bfloat16()
            for n, r, c in (("W1", H, F), ("W3", H, F), ("W2", F, H)):
                w = torch.randn((E, r, c), generator=gen, device="cuda") * r ** -0.5
                setattr(self, n, w.bfloat16())

    def run(self, **kw):
        return mk.moe_ffn_decode(self.x, self.logits, self.W1, self.W3, self.W2, self.k, **self.scales, **kw)["out"]

    def matrix(self, n, e):
        w = getattr(self, n)[e].double()
        return w * _blocks(self.scales[n + "_scale"][e]) if self.fp8 else w

    def check(self, out):
        assert out.shape == (self.T, self.H) and out.dtype == torch.bfloat16
        x = self.x.double()
        if self.fp8:
            x = x * self.scales["x_scale"].double().repeat_interleave(128, 1)
        want = torch.zeros((self.T, self.H), dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        l = self.logits.cpu().numpy()
        chosen = np.argsort(-l.astype(np.float64), axis=1, kind="stable")[:, :self.k]  # ties: lower expert first
        for e in np.unique(chosen):
            t, j = np.nonzero(chosen == e)
            v = l[t[:, None], chosen[t]].astype(np.float64)
            top = v[:, :1]
            w = np.where(v > -np.inf, np.exp(v - np.where(np.isinf(top), 0, top)), 0.0)
            s = w.sum(1, keepdims=True)
            gate = torch.from_numpy((w / np.where(s == 0, 1, s))[np.arange(len(t)), j]).cuda()[:, None]
            rows = torch.from_numpy(t).cuda()
            w1, w3, w2 = (self.matrix(n, int(e)) for n in ("W1", "W3", "W2"))
            a, b = x[rows] @ w1, x[rows] @ w3
            ea, eb = 2.0 ** -16 * (x[rows].abs() @ w1.abs()), 2.0 ** -16 * (x[rows].abs() @ w3.abs())
            h = a * torch.sigmoid(a) * b
            # |silu'| <= 1.1 and |silu(a)| <= |a|
            eh = 1.1 * ea * b.abs() + a.abs() * eb + ea * eb * 1.1 + 2.0 ** -16 * h.abs()
            if self.fp8:
                g = h.view(len(t), -1, 128)
                amax = g.abs().amax(2, keepdim=True)
                sc = torch.where(amax < 2.0 ** -100, torch.ones_like(amax), amax / 448)
                q = (g / sc).to(torch.float8_e4m3fn).double() * sc
                lo = ((g.abs() * (1 - 2.0 ** -14) - eh.view_as(g)).clamp(min=0) / sc).to(torch.float8_e4m3fn).double()
                hi = ((g.abs() * (1 + 2.0 ** -14) + eh.view_as(g)) / sc).clamp(max=448).to(torch.float8_e4m3fn).double()
                h = q.view_as(h)
                # the step to the other side of a boundary, and the scale's own error
                eh = ((hi - lo) * sc + 2.0 ** -14 * q.abs()).view_as(h)
            want.index_add_(0, rows, gate * (h @ w2))
            tol.index_add_(0, rows, gate * (eh @ w2.abs() + 2.0 ** -16 * (h.abs() @ w2.abs())))
        tol = tol + 2.0 ** -8 * want.abs() + 2.0 ** -20 * want.abs()
        bad = (out.double() - want).abs() > tol
        assert not torch.any(bad), f"{int(bad.sum())} of {bad.numel()} values off"
        # the bound above is for the worst case: on the whole the output is as good as its rounding
        err = (out.double() - want).norm() / want.norm().clamp(min=1e-300)
        assert err <= (2.0 ** -8 if not self.fp8 else 2.0 ** -7)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 2, 11, 12, 40, 128])
@pytest.mark.parametrize("E,k", [(1, 1), (7, 3), (64, 8)])
def test_tokens_and_experts(T, E, k, fp8):
    layer = Layer(T, 256, 384, E, k, fp8, seed=T + E)
    layer.check(layer.run())


@pytest.mark.parametrize("H,F", [(64, 64), (64, 1024), (1024, 64), (192, 320), (320, 192), (2112, 704), (704, 2112)])
def test_sizes_16(H, F):
    layer = Layer(5, H, F, 6, 2, seed=H + F)
    layer.check(layer.run())


@pytest.mark.parametrize("H,F", [(128, 128), (128, 1024), (1024, 128), (384, 640), (640, 384), (2176, 768)])
def test_sizes_8(H, F):
    layer = Layer(5, H, F, 6, 2, True, seed=H + F)
    layer.check(layer.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T", [3, 128])
def test_every_token_to_one_expert(T, fp8):
    logits = torch.zeros((T, 32))
    logits[:, 17] = 5
    layer = Layer(T, 256, 256, 32, 1, fp8, logits=logits)
    layer.check(layer.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_equal_masked_and_signed_zero_logits(fp8):
    logits = torch.randn((20, 40), generator=torch.Generator().manual_seed(3))
    logits[0] = 0                       # all equal: the lowest experts
    logits[1] = -INF                    # nothing left: gates 0, output 0
    logits[2] = -INF
    logits[2, 33] = 1                   # fewer live experts than k
    logits[3] = -0.0
    logits[3, 20:] = 0.0                # -0 and 0 are equal
    logits[4] = torch.finfo(torch.float32).min
    logits[5, 10] = torch.finfo(torch.float32).max
    logits[6:, 5:30] = -INF
    layer = Layer(20, 128, 256, 40, 4, fp8, logits=logits)
    out = layer.run()
    assert torch.all(out[1] == 0)
    layer.check(out)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_most_experts(fp8):
    layer = Layer(100, 128, 128, 256, 8, fp8, seed=9)
    layer.check(layer.run())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
def test_large_layer(fp8):
    layer = Layer(9, 4096, 1536, 24, 4, fp8, seed=10)
    layer.check(layer.run())


def test_repeatable_whatever_ran_before_and_on_another_stream():
    one, two = Layer(17, 512, 640, 16, 4, seed=11), Layer(100, 256, 256, 8, 2, True, seed=12)
    a, b = one.run(), two.run()
    need = max(mk.mk_moe_ffn_decode_workspace_size(17, 512, 640, 16, 4, mk.MK_WEIGHT_BF16),
               mk.mk_moe_ffn_decode_workspace_size(100, 256, 256, 8, 2, mk.MK_WEIGHT_E4M3))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(one.run(workspace=ws, ws_bytes=need), a)
        assert torch.equal(two.run(workspace=ws, ws_bytes=need), b)
        assert torch.equal(one.run(), a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    c = one.run(stream=side, check=False)
    assert mk.mk_get_status(side) == mk.MK_OK and torch.equal(a, c)
    one.check(a)
    two.check(b)


def test_no_tokens_and_small_workspace():
    layer = Layer(4, 128, 128, 4, 2)
    assert mk.moe_ffn_decode(layer.x[:0], layer.logits[:0], layer.W1, layer.W3, layer.W2, 2)["out"].shape == (0, 128)
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    with pytest.raises(mk.MkError) as e:
        layer.run(workspace=ws, ws_bytes=ws.numel())
    assert e.value.status == mk.MK_ERR_WORKSPACE


def test_agrees_with_the_dispatch_path():
    # the same routing and the same SwiGLU as the gated dispatch, completed by hand
    layer = Layer(30, 256, 512, 16, 4, seed=13)
    o = mk.moe_gated(layer.x, layer.logits, layer.W1, layer.W3, 4, cfg=mk.make_config(out_dtype=mk.MK_OUT_F32))
    off = o["expert_offsets"].tolist()
    y = torch.empty((120, 256), dtype=torch.float64, device="cuda")
    for e in range(16):
        y[off[e]:off[e + 1]] = o["y_sorted"][off[e]:off[e + 1]].double() @ layer.W2[e].double()
    want = torch.zeros((30, 256), dtype=torch.float64, device="cuda")
    want.index_add_(0, o["src_index"].long() // 4, o["gate_w"].double()[:, None] * y)
    # both are fp32 sums; the dispatch path uses the fast exponential
    assert (layer.run().double() - want).abs().max() <= 2.0 ** -8 * want.abs().max() + 1e-4


def test_offsets_past_32_bits():
    # weights of more than 2^31 elements a matrix; only the last experts are used, and only they are set
    E, H, F = 230, 4096, 2560
    logits = torch.full((3, E), -5.0)
    logits[:, E - 4:] = torch.randn((3, 4), generator=torch.Generator().manual_seed(1))
    small = Layer(3, H, F, 4, 3, seed=14, logits=logits[:, E - 4:].contiguous())
    W1, W3, W2 = (torch.empty((E, *w.shape[1:]), dtype=torch.bfloat16, device="cuda") for w in (small.W1, small.W3, small.W2))
    for big, w in ((W1, small.W1), (W3, small.W3), (W2, small.W2)):
        big[E - 4:] = w
    out = mk.moe_ffn_decode(small.x, logits.cuda(), W1, W3, W2, 3)["out"]
    assert torch.equal(out, small.run())


def test_hidden_values_past_the_16_bit_range_are_infinite():
    # h[:, 0] overflows for the first two tokens; the third's are zeros
    layer = Layer(3, 128, 192, 1, 1, seed=13)
    layer.x[:2], layer.x[2] = 1.0, 0.0
    layer.W1[0, :, 0], layer.W3[0, :, 0] = 1e20, 1e20
    layer.W2[0, 0, 5] = 0.25
    out = layer.run().float()
    assert torch.equal(out[:2], torch.sign(layer.W2[0, 0].float()).expand(2, -1) * INF) and torch.all(out[2] == 0)
