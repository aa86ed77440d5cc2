"""Sines and cosines of mk_qk_norm_rope by themselves: pairs (1, 0) turn into
(cos, sin), so small angles, and angles next to a quarter of a turn, show how many
bits of their own they keep.

Tolerances.  A frequency f is held as turns in steps of 2^-64, off by (1 + f/2) of
them: of 2^-36 or more that is 2^-25 of the angle.  What is left of a quarter turn
is exact before it is rounded to 24 bits (2^-24), the functions are off by 2^-22,
so a sine is known to 2^-21 of itself, taken as 2^-20.  Where the angle is far, its
distance from the nearest quarter turn is off by the angle's own error: 2^-62 of a
turn for each position, at frequencies up to 4.  Rounding to bf16: 2^-8."""
import math

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


def turned(inv, positions, interleaved):
    """(cos, sin) [T, rot/2] of every position and frequency."""
    half, T = inv.numel(), positions.numel()
    q = torch.zeros((T, 1, 2 * half), dtype=torch.bfloat16, device="cuda")
    ia, ib = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, half), slice(half, None))
    q[..., ia] = 1
    o = mk.qk_norm_rope(q, q, positions, inv, interleaved=interleaved)
    assert torch.equal(o["q"], o["k"])
    return o["q"][:, 0, ia].double(), o["q"][:, 0, ib].double()


def check(got, want, known):
    assert torch.all((got - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs() + known)


@pytest.mark.parametrize("interleaved", [False, True])
def test_small_angles(interleaved):
    # theta 10^6 over 128 columns, and the smallest frequencies that keep their bits
    inv = torch.cat([1e6 ** (-torch.arange(0, 112, 2, dtype=torch.float64) / 112), 2.0 ** -torch.arange(20.0, 36, 2).double()])
    inv = inv.float().cuda()
    pos = torch.tensor([0, 1, 2, -1, -3, 100, 4097], dtype=torch.int32, device="cuda")
    cosine, sine = turned(inv, pos, interleaved)
    angle = pos.double()[:, None] * inv.double()
    known = 2 * math.pi * 2.0 ** -62 * pos.double().abs()[:, None]
    check(cosine, angle.cos(), known)
    check(sine, angle.sin(), known)


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_next_to_quarter_turns(interleaved):
    # the fp32 numbers next to pi / 2, pi, 3 pi / 2 and 2 pi over small whole numbers, times these:
    # products that 64 bits hold exactly, 10^-7 from a quarter turn
    inv, pos = [], torch.tensor([1, -1, 2, 3, 5, 7, 12, -16, 60, 420], dtype=torch.int32, device="cuda")
    for n in (1, 2, 3, 4, 5, 6, 7, 8):
        inv += [math.pi / 2 / n, math.pi / 3 / n]
    inv = torch.tensor(inv, dtype=torch.float64).float().cuda()
    cosine, sine = turned(inv, pos, interleaved)
    angle = pos.double()[:, None] * inv.double()
    known = 2 * math.pi * 2.0 ** -62 * pos.double().abs()[:, None]
    check(cosine, angle.cos(), known)
    check(sine, angle.sin(), known)
    assert int((cosine.abs() < 1e-5).sum()) > 10 and int((sine.abs() < 1e-5).sum()) > 20
