"""mk_qk_norm_rope into caches in every form: neighbouring pairs as well as halves,
part of the columns rotated, small and odd heads, several axes, strided heads.
References and tolerances are those of test_gpu_qk_norm_rope.py."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_qk_norm_rope import Case, check_fp4, slots_for, unpack  # noqa: E402

SIZES = [(16, 16), (32, 32), (32, 16), (48, 48), (64, 64), (64, 32), (80, 80), (80, 48), (128, 128), (128, 64), (128, 0),
         (192, 192), (256, 256), (256, 64)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()


def cases(D, rot, interleaved):
    yield Case(75, 6, 3, D, rot, interleaved=interleaved, seed=D + rot)
    yield Case(1, 10, 5, D, rot, interleaved=interleaved, seed=D + rot + 1, layout="heads")
    yield Case(40, 4, 4, D, rot, interleaved=interleaved, seed=D + rot + 2, axes=3, layout="heads")
    yield Case(33, 2, 1, D, rot, interleaved=interleaved, seed=D + rot + 3, norm=False, layout="apart")


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("D,rot", SIZES)
def test_bf16_pages(D, rot, interleaved):
    for page, c in zip((16, 7, 1, 24), cases(D, rot, interleaved)):
        pages = -(-c.T // page) + 2
        both = torch.randn((pages, 2, page, c.Hkv, D), device="cuda").bfloat16()
        want = both.clone()
        slots = slots_for(c.T, pages, page, c.T)
        o = c.run(v=c.v, slots=slots, k_cache=both[:, 0], v_cache=both[:, 1], keep=True)
        c.check(o["q"], c.q, c.qw)
        c.check(o["k"], c.k, c.kw)
        rows = torch.nonzero(slots >= 0)[:, 0]
        at = slots[rows] // page, slots[rows] % page
        want[at[0], 0, at[1]], want[at[0], 1, at[1]] = o["k"][rows], c.v[rows]
        assert torch.equal(both, want)  # what was returned, and nothing else


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("D,rot", SIZES)
def test_4_bit_pages(D, rot, interleaved):
    for page, c in zip((16, 7, 1, 24), cases(D, rot, interleaved)):
        pages = -(-c.T // page) + 2
        z = mk.fp4_cache(pages, page, c.Hkv, D)
        for t in z.values():
            t.view(torch.uint8).random_(0, 120)
        before = {n: t.clone() for n, t in z.items()}
        f = {n: torch.exp(torch.randn(c.Hkv, device="cuda")) for n in ("k_factor", "v_factor")} if c.T % 2 else {}
        slots = slots_for(c.T, pages, page, c.T)
        o = c.run(v=c.v, slots=slots, keep=True, **z, **f)
        c.check(o["q"], c.q, c.qw)
        k, tol = c.want(c.k, c.kw)
        rows = torch.nonzero(slots >= 0)[:, 0]
        at = slots[rows] // page, slots[rows] % page
        for name, y, t in (("k", k, tol), ("v", c.v.double(), 0 * tol)):
            held = f.get(name + "_factor", torch.ones(c.Hkv, device="cuda")).double()[:, None]
            codes, scales = z[name + "_cache"][at], z[name + "_scales"].view(torch.uint8)[at].view(torch.float8_e4m3fn)
            check_fp4(codes, scales, (y / held)[rows], (t / held + 2.0 ** -23 * (y / held).abs())[rows])
            value = (unpack(codes).unflatten(-1, (-1, 16)) * scales.double()[..., None]).flatten(-2) * held
            assert torch.all((o[name][rows].double() - value).abs() <= 2.0 ** -8 * value.abs() * (1 + 2.0 ** -20))
            for part in ("_cache", "_scales"):  # nothing else was written
                was, now = (d[name + part].view(torch.uint8).clone() for d in (before, z))
                was[at] = 0
                now[at] = 0
                assert torch.equal(was, now)
