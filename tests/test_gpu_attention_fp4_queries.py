"""mk_paged_attention_fp4 with queries at the lower end of bf16, which a scale near
the upper end of fp32 makes count.  Cases, references and tolerances are those of
test_gpu_attention_fp4.py: subnormal values, whole multiples of 2^-133, keep all
their bits when they are moved into fp16's range."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_attention_fp4 import Case  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()


def subnormal(shape, seed):
    """bf16 values of -127 .. 127 times 2^-133, by their bits."""
    n = torch.randint(-127, 128, shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    return (n.abs() | (n < 0).int() * 0x8000).to(torch.int16).view(torch.bfloat16), n


@pytest.mark.parametrize("D,Hq", [(64, 8), (128, 8), (128, 32), (256, 8)])
def test_subnormal_queries(D, Hq):
    c = Case([300, 64, 0, 1], Hq, 2, D, 16, seed=D, factors=True)
    q, n = subnormal((4, Hq, D), D)
    assert torch.equal(q.double(), n.double() * 2.0 ** -133)
    for scale in (2.0 ** 124, -(2.0 ** 125)):
        c.q = q
        o = c.run(scale=scale)
        c.check(o, scale)
        # the same numbers as normal ones: the same scores, to the last bit
        c.q = (n.double() * 2.0 ** -33).bfloat16()
        same = c.run(scale=scale * 2.0 ** -100)
        assert torch.equal(o["lse"], same["lse"]) and torch.equal(o["out"], same["out"])


@pytest.mark.parametrize("exponent", [-126, -119, -113, -112, -111])
def test_largest_column_at_the_lower_end(exponent):
    c = Case([300, 64], 8, 2, 128, 16, seed=1)
    q, _ = subnormal((2, 8, 128), 3)
    q[:, :, 5] = 1.5 * 2.0 ** exponent  # beside subnormal ones
    q[:, 3] = 0
    c.q = q
    scale = 2.0 ** (-exponent - 1)
    c.check(c.run(scale=scale), scale)


def test_a_key_whose_scale_is_nan():
    c = Case([40, 40], 8, 2, 64, 16, seed=9)
    good = c.run()
    c.cache["k_scales"].view(torch.uint8)[int(c.table[0, 1]), 3, 1, 2] = 0x7f
    o = c.run()
    for n in ("out", "lse"):
        assert torch.all(torch.isnan(o[n][0, 4:]))
        o[n][0, 4:] = good[n][0, 4:]
        assert torch.equal(o[n], good[n])
