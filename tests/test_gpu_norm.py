"""mk_add_rmsnorm against its formulas in 64 bits: widths that fill no vector,
group or warp, strided and misaligned rows, every choice of outputs, rows of
zeros, NaN and infinities, the residual updated in place.

Tolerances.  bf16 keeps 8 significant bits: rounding is off by at most 2^-8
of the value (half a step of 2^-7 at 1).  e4m3 keeps 4: at most 2^-4 of the value, or half its smallest
step (2^-10, times the scale).  Before the rounding the fp32 arithmetic is
off by less than 2e-5 of the value: the sum of squares adds at most 40 terms
in a row (32-bit rounding 2^-24 each, halved by the square root), and the
root, the two products and the divisions add a few 2^-23."""
import numpy as np
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

FP32 = 2e-5
BF16 = 2.0 ** -8 + FP32
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()


def _rows(T, H, seed, stride=None, offset=0):
    """bf16 [T,H] on the device with `stride` elements between rows, `offset` elements into its buffer."""
    stride = stride or H
    buf = torch.from_numpy(np.random.default_rng(seed).standard_normal(offset + max(T, 1) * stride)).bfloat16().cuda()
    return torch.as_strided(buf, (T, H), (stride, 1), offset)


def _reference(x, residual, weight, eps=EPS):
    z = x.double().cpu() + (residual.double().cpu() if residual is not None else 0)
    y = z / torch.sqrt((z * z).sum(1, keepdim=True) / z.shape[1] + eps) * weight.double().cpu()
    return z, y


def _close(got, want, rel):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = torch.isfinite(want)
    assert torch.all((got - want)[ok].abs() <= rel * want[ok].abs() + 1e-37)


def _check_e4m3(o, y):
    T, H = y.shape
    scale = o["scale"].double().cpu()
    assert scale.shape == (T, -(-H // 128))
    padded = torch.nn.functional.pad(y, (0, -H % 128)).view(T, -1, 128)
    amax = padded.abs().amax(2)
    want = torch.where(amax < 2.0 ** -100, torch.ones_like(amax), amax / 448)
    assert torch.all((scale - want).abs() <= FP32 * want)
    got = o["out8"].float().double().cpu()
    assert torch.all(got.abs() <= 448)
    s = scale.repeat_interleave(128, 1)[:, :H]
    assert torch.all((got * s - y).abs() <= (2.0 ** -4 + FP32) * y.abs() + 2.0 ** -10 * s)


def _run_and_check(x, weight, residual, bf16=True, e4m3=True, **kw):
    z, y = _reference(x, residual, weight)
    o = mk.add_rmsnorm(x, weight, residual=residual, eps=EPS, bf16=bf16, e4m3=e4m3, **kw)
    assert set(o) == ({"out"} if bf16 else set()) | ({"out8", "scale"} if e4m3 else set()) | (
        {"residual"} if residual is not None else set())
    if bf16:
        _close(o["out"], y, BF16)
    if e4m3:
        _check_e4m3(o, y)
    if residual is not None:
        _close(o["residual"], z, BF16)
    return o


@pytest.mark.parametrize("H", [1, 7, 8, 127, 128, 129, 256, 264, 1001, 4096, 7168, 8200, 20000, 32768])
@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("with_residual", [False, True])
def test_widths(T, H, with_residual):
    x, w = _rows(T, H, 1), _rows(1, H, 2)[0]
    _run_and_check(x, w, _rows(T, H, 3) if with_residual else None)


@pytest.mark.parametrize("bf16,e4m3", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("H", [1000, 1001])
def test_choice_of_outputs(H, bf16, e4m3):
    _run_and_check(_rows(9, H, 4), _rows(1, H, 5)[0], _rows(9, H, 6), bf16=bf16, e4m3=e4m3)


@pytest.mark.parametrize("x_stride,r_stride,x_off,r_off", [
    (1024, 2048, 0, 0),   # a slice of a wider row, vectors still aligned
    (1004, 1000, 0, 0),   # strides that are no multiple of a vector
    (1000, 1000, 1, 0),   # rows that start two bytes off
    (1000, 1000, 0, 4),
])
def test_strides_and_alignment(x_stride, r_stride, x_off, r_off):
    x, r = _rows(33, 1000, 7, x_stride, x_off), _rows(33, 1000, 8, r_stride, r_off)
    plain = mk.add_rmsnorm(x.contiguous(), _rows(1, 1000, 9)[0], residual=r.contiguous(), e4m3=True)
    o = _run_and_check(x, _rows(1, 1000, 9)[0], r)
    # the scalar and the vector form sum in another order: the same up to that
    _close(o["out"], plain["out"].double().cpu(), 2 * BF16)


def test_residual_in_place_and_repeatable():
    x, r, w = _rows(70, 2048, 10), _rows(70, 2048, 11), _rows(1, 2048, 12)[0]
    a = _run_and_check(x, w, r)
    mine = r.clone()
    b = mk.add_rmsnorm(x, w, residual=mine, eps=EPS, e4m3=True, residual_out=mine)
    assert b["residual"].data_ptr() == mine.data_ptr()
    for name in a:
        assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name


@pytest.mark.parametrize("H", [512, 515])
def test_zero_nan_and_infinite_rows(H):
    x, w = _rows(6, H, 13), _rows(1, H, 14)[0]
    x[1] = 0
    x[2, H // 2] = float("nan")
    x[3, 0] = float("inf")
    x[4] *= 1e-30  # mean of squares far below eps
    o = mk.add_rmsnorm(x, w, eps=EPS, e4m3=True)
    out, out8 = o["out"].float().cpu(), o["out8"].float().cpu()
    assert torch.all(out[1] == 0) and torch.all(out8[1] == 0) and torch.all(o["scale"][1] == 1)
    assert torch.all(torch.isnan(out[2])) and torch.all(torch.isnan(out8[2])) and torch.all(torch.isnan(o["scale"][2]))
    assert torch.isnan(out[3, 0]) and torch.all(out[3, 1:] == 0)
    assert torch.isnan(o["scale"][3, 0]) and torch.all(o["scale"][3, 1:] == 1) and torch.all(out8[3, 128:] == 0)
    _, y = _reference(x, None, w)
    rest = [0, 1, 4, 5]
    _close(o["out"][rest], y[rest], BF16)


def test_tiny_groups_get_scale_one():
    x = torch.full((1, 256), 2.0 ** -60).bfloat16().cuda()
    w = torch.ones(256).bfloat16().cuda()
    w[128:] = 2.0 ** -55
    o = mk.add_rmsnorm(x, w, eps=1.0, e4m3=True)  # y = 2^-60 and 2^-115
    assert o["scale"][0, 0].item() == pytest.approx(2.0 ** -60 / 448, rel=FP32) and o["scale"][0, 1].item() == 1.0
    assert torch.all(o["out8"].float()[0, :128] == 448) and torch.all(o["out8"].float()[0, 128:] == 0)


def test_no_rows_and_another_stream():
    w = _rows(1, 640, 15)[0]
    o = mk.add_rmsnorm(_rows(0, 640, 16), w, e4m3=True)
    assert o["out"].shape == (0, 640) and o["scale"].shape == (0, 5)
    x, r = _rows(40, 640, 17), _rows(40, 640, 18)
    here = mk.add_rmsnorm(x, w, residual=r, e4m3=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    there = mk.add_rmsnorm(x, w, residual=r, e4m3=True, stream=side, check=False)
    assert mk.mk_get_status(side) == mk.MK_OK
    for name in here:
        assert torch.equal(here[name].view(torch.uint8), there[name].view(torch.uint8)), name


def test_offsets_past_32_bits():
    # rows 2^30 elements apart, and more than 2^31 elements of output
    x, r, w = _rows(3, 72, 19), _rows(3, 72, 20), _rows(1, 72, 21)[0]
    far = torch.empty(2 * (2 ** 30 + 8) + 72, dtype=torch.bfloat16, device="cuda").as_strided((3, 72), (2 ** 30 + 8, 1))
    far.copy_(x)
    o, want = mk.add_rmsnorm(far, w, residual=r, e4m3=True), mk.add_rmsnorm(x, w, residual=r, e4m3=True)
    for name in o:
        assert torch.equal(o[name].view(torch.uint8), want[name].view(torch.uint8)), name
    del far
    T, H = 2 ** 31 // 32768 + 9, 32768
    big = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    tail = _rows(5, H, 22)
    big[-5:] = tail
    w = _rows(1, H, 23)[0]
    o, want = mk.add_rmsnorm(big, w, residual=big, e4m3=True), mk.add_rmsnorm(tail, w, residual=tail, e4m3=True)
    for name in o:
        assert torch.equal(o[name][-5:].view(torch.uint8), want[name].view(torch.uint8)), name
    assert torch.all(o["out"][:-5:4096] == 0)


@pytest.mark.parametrize("H", [32768, 32767])  # 16-byte accesses, and single elements
def test_8_bit_values_are_of_the_quotient(H):
    # x = +-1 and eps = 0 make y the weights themselves, so the stored scale and
    # e4m3(y / scale) are known: every significand of a group's largest value
    # against every significand, in four binades
    m = 1 + torch.arange(128, dtype=torch.float64) / 128
    w = m[:, None].repeat(1, 128).repeat_interleave(4, 0)  # 512 groups: the largest value, and
    for i in range(4):
        w[i::4, 1:] = m[1:] * 2.0 ** (-1 - i)              # the others below it
    x = torch.ones((3, H)).bfloat16()
    x[1] = -1
    for half in (w[:256], w[256:]):
        weight = half.reshape(-1)[:H].bfloat16().cuda()
        o = mk.add_rmsnorm(x.cuda(), weight, eps=0.0, e4m3=True)
        assert torch.equal(o["out"].cpu(), x * weight.cpu())
        y = torch.zeros(32768)
        y[:H] = weight.float().cpu()
        scale = y.view(256, 128).amax(1) / 448
        want = (y.view(256, 128) / scale[:, None]).to(torch.float8_e4m3fn).float().view(-1)[:H]
        assert torch.equal(o["scale"].cpu(), scale.expand(3, -1))
        assert torch.equal(o["out8"].float().cpu(), want * x.float())
