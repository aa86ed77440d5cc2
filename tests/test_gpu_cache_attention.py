"""The run of test_gpu_cache_run.py with the attention's own output held to what is
cached, value by value: the projection behind it is the identity, so a step returns
that output, and the queries are those that the step's rotation gave.

Tolerances are those of test_gpu_attention.py and test_gpu_attention_fp4.py: with
ds = 2^-20 * scale * max_j sum |q_i k_ij| (4 bits: and 2^-39 of the largest query
column times sum |k|), 2^-8 of the output and 4 ds + 2^-14 of the weighted |v|;
in 4 bits 2^-11 of that besides, the weights' rounding, and 2^-35 * sum |v|.  A
last key that was left out, or counted twice, has to lie outside of them."""
import importlib
import os
import sys

import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_cache_run import Followed, i32  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


class Exact(Followed):
    def __init__(self, ex, z, seed, monkeypatch):
        super().__init__(ex, z, seed)
        self.a.w_o = torch.eye(z.H, device="cuda").bfloat16()
        rotate = mk.qk_norm_rope

        def recorded(*args, **kw):
            o = rotate(*args, **kw)
            self.q = o["q"]
            return o

        monkeypatch.setattr(mk, "qk_norm_rope", recorded)
        self.seen = 0  # rows whose last key was told apart

    def want(self, q, k, v):
        """The attention of q [Hq,D] over k and v [n,Hkv,D] in 64 bits, and how far it may be off."""
        z = self.z
        G, scale = z.Hq // z.Hkv, z.D ** -0.5
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        s = torch.einsum("hd,nhd->hn", q, k) * scale
        ds = 2.0 ** -20 * torch.einsum("hd,nhd->hn", q.abs(), k.abs()).amax(1, keepdim=True)
        if z.fp4:
            ds = ds + 2.0 ** -39 * q.abs().amax(1, keepdim=True) * k.abs().sum(2).amax(0)[:, None]
        p = torch.softmax(s, 1)
        out, spread = (torch.einsum("hn,nhd->hd", p, x) for x in (v, v.abs()))
        tol = 2.0 ** -8 * out.abs() + (4 * scale * ds + 2.0 ** -14 + (2.0 ** -11 if z.fp4 else 0)) * spread
        return out, tol + (2.0 ** -35 * v.abs().sum(0) if z.fp4 else 0)

    def step(self, x, live):
        out = super().step(x, live)
        for row in range(self.z.rows):
            got, n = out[row].double().view(self.z.Hq, self.z.D), len(self.keys[row])
            if n == 0:
                assert torch.all(got == 0)
                continue
            q, (k, v) = self.q[row].double(), self.held(row)
            want, tol = self.want(q, k, v)
            assert torch.all((got - want).abs() <= tol), f"row {row} of {n} keys"
            if n > 1:
                for wrong in (slice(0, n - 1), list(range(n)) + [n - 1]):
                    want, tol = self.want(q, k[wrong], v[wrong])
                    assert not torch.all((got - want).abs() <= tol), f"row {row} of {n} keys"
                    self.seen += 1
        return out


@pytest.mark.parametrize("fp4", [False, True], ids=["bf16", "fp4"])
@pytest.mark.parametrize("page,D,Hkv", [(4, 64, 2), (1, 64, 8), (8, 128, 2), (16, 64, 1)])
def test_steps_forks_and_compaction(ex, monkeypatch, fp4, page, D, Hkv):
    z = ex.Sizes(H=8 * D, Hq=8, Hkv=Hkv, D=D, page=page, pages=220, rows=7, longest=48, fp4=fp4)
    f = Exact(ex, z, page + D, monkeypatch)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def step(live):
        f.step(torch.randn((z.rows, z.H), generator=gen, device="cuda").bfloat16(), i32(live))

    for _ in range(page + 1):
        step([1, 1, 0, 0, 0, 0, 0])
    f.fork([0, 0, 1], [2, 3, 4])
    step([0, 1, 1, 1, 0, 1, 0])
    step([1, 1, 1, 1, 1, 1, 1])
    f.fork([2, 3, 0], [3, 2, 6])  # two of them one another's
    step([1, 1, 1, 1, 0, 0, 1])
    f.free([0, 4])
    f.a.compact()
    for _ in range(3):
        step([1, 1, 1, 1, 0, 1, 1])
    assert f.seen >= 74 and mk.mk_get_status() == mk.MK_OK  # 4 + 10 + 12 + 14 + 34 with pages of one key
