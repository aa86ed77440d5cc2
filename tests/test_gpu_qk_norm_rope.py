"""mk_qk_norm_rope against norm and rotation in 64 bits: head sizes and layouts,
pairs, axes, far and negative positions, partial rotation, strided inputs, both
kinds of cache, padding, slots outside the pool, values that are not finite.

Tolerances.  x * rstd * w in fp32: the sum of squares is off by 2^-20 of itself
at most (16 additions and products in a lane's chain and the shuffles), its root
and reciprocal by half of that and 2^-22, the two products by 2^-23: together
less than 2^-19.  Sine and cosine are off by 2^-22 (half a unit of the function,
2^-25 turns of the angle's rounding, 2^-32 of its cut), the two products and the
sum by 2^-23: a rotated value by less than 2^-18 * (|a| + |b|).  The output's
rounding adds half a step, 2^-8 of it at most.  In 4 bits the kernel's y may
lie on the other side of the middle of two steps: the bytes and scales are held
to those of the nearest y within that tolerance, see `check_fp4`."""
import numpy as np
import pytest

import moe_token_dispatch_persistent_gb300 as mk

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

EPS = 1e-6
STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()


class Case:
    def __init__(self, T, Hq, Hkv, D, rot=None, axes=1, interleaved=False, norm=True, layout="packed", positions=None,
                 seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.T, self.Hq, self.Hkv, self.D = T, Hq, Hkv, D
        self.rot = rot = D if rot is None else rot
        self.interleaved = interleaved
        if layout == "packed":
            x = randn(T, (Hq + 2 * Hkv) * D).bfloat16()
            self.q, self.k, self.v = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
        elif layout == "apart":
            self.q, self.k, self.v = (randn(T, h, D).bfloat16() for h in (Hq, Hkv, Hkv))
        else:  # heads outside, with a gap
            self.q, self.k, self.v = (randn(h, T, D + 8).bfloat16()[:, :, :D].transpose(0, 1) for h in (Hq, Hkv, Hkv))
        self.qw, self.kw = ((1 + 0.2 * randn(D)).bfloat16() if norm else None for _ in range(2))
        self.inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()
        if positions is None:
            positions = torch.randint(0, 200000, (axes, T), generator=gen, device="cuda")
        self.pos = positions.to(torch.int32).view(axes, T)
        self.axis = None if axes == 1 else [(i * 7) % axes for i in range(rot // 2)]

    def run(self, **kw):
        pos = self.pos if self.axis is not None else self.pos[0]
        return mk.qk_norm_rope(self.q, self.k, pos, self.inv, q_weight=self.qw, k_weight=self.kw, eps=EPS,
                               interleaved=self.interleaved, pair_axis=self.axis, **kw)

    def want(self, x, weight):
        """The rotated rows in 64 bits and how far fp32 may be off."""
        x = x.double()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()
        axis = torch.tensor(self.axis or [0] * (self.rot // 2), device="cuda", dtype=torch.int64)
        angle = (self.pos.double()[axis].T * self.inv.double())[:, None]
        h = self.rot // 2
        ia, ib = ((slice(0, self.rot, 2), slice(1, self.rot, 2)) if self.interleaved
                  else (slice(0, h), slice(h, self.rot)))
        a, b = x[..., ia].clone(), x[..., ib].clone()
        tol = 2.0 ** -18 * x.abs()
        x[..., ia], x[..., ib] = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
        tol[..., ia] = tol[..., ib] = 2.0 ** -18 * (a.abs() + b.abs())
        return x, tol

    def check(self, got, x, weight):
        want, tol = self.want(x, weight)
        off = (got.double() - want).abs()
        assert torch.all(off <= tol + 2.0 ** -8 * (want.abs() + tol)), float((off - tol).max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(16, 16), (32, 32), (48, 32), (64, 64), (64, 32), (80, 80), (96, 48), (112, 112),
                                   (128, 128), (128, 64), (128, 16), (192, 192), (256, 256), (256, 64), (128, 0)])
def test_head_sizes(D, rot, interleaved):
    c = Case(37, 6, 2, D, rot, interleaved=interleaved, seed=D + rot)
    o = c.run()
    assert set(o) == {"q", "k"}
    c.check(o["q"], c.q, c.qw)
    c.check(o["k"], c.k, c.kw)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (2, 5, 5), (300, 15, 3), (1, 128, 8), (3, 7, 1), (5000, 4, 1),
                                      (0, 4, 2), (40000, 1, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_layouts(T, Hq, Hkv, D):
    for layout in ("packed", "apart", "heads"):
        c = Case(T, Hq, Hkv, D, layout=layout, seed=T + Hq)
        o = c.run()
        assert o["q"].shape == (T, Hq, D) and o["k"].shape == (T, Hkv, D)
        c.check(o["q"], c.q, c.qw)
        c.check(o["k"], c.k, c.kw)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_axes(axes, interleaved):
    c = Case(77, 4, 2, 128, 96, axes=axes, interleaved=interleaved, seed=axes)
    o = c.run()
    c.check(o["q"], c.q, c.qw)
    c.check(o["k"], c.k, c.kw)


def test_far_and_negative_positions():
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 20 + 1, 131071, -77777, 2 ** 30], device="cuda")
    c = Case(len(pos), 4, 2, 128, positions=pos, seed=3)
    # beside the usual ones frequencies above one, tiny ones and none at all
    c.inv[:8] = torch.tensor([3.25, 1.0, 100.5, 1e-30, 0.0, 2.0 ** -149, -0.37, 6.2831855], device="cuda")
    o = c.run()
    # 2^-53 of a product of 2^31 * 100 in the 64-bit form, below 2^-15
    want, tol = c.want(c.q, c.qw)
    far = (o["q"].double() - want).abs() - tol - 2.0 ** -8 * (want.abs() + tol)
    assert torch.all(far <= 2.0 ** -15 * 8)
    near = [0, 1, 2, 5, 6, 7]
    assert torch.all(far[near] <= 2.0 ** -22)


@pytest.mark.parametrize("interleaved", [False, True])
def test_without_norm_and_with_one_of_them(interleaved):
    c = Case(21, 4, 2, 64, norm=False, interleaved=interleaved, seed=5)
    o = c.run()
    c.check(o["q"], c.q, None)
    c.check(o["k"], c.k, None)
    c.kw = torch.full((64,), 0.5, device="cuda").bfloat16()
    o = c.run()
    c.check(o["q"], c.q, None)
    c.check(o["k"], c.k, c.kw)


def slots_for(T, pages, page, seed, holes=True):
    rng = np.random.default_rng(seed)
    s = rng.permutation(pages * page)[:T].astype(np.int64)
    if holes and T > 3:
        s[rng.integers(0, T, max(1, T // 9))] = -1
        s[0] = -2 ** 40
    return torch.from_numpy(s).cuda()


@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("T,Hq,Hkv,D,page", [(1, 32, 8, 128, 16), (50, 12, 12, 64, 1), (333, 5, 1, 256, 24), (9, 4, 2, 80, 7)])
def test_bf16_cache(T, Hq, Hkv, D, page, layout):
    c = Case(T, Hq, Hkv, D, seed=T)
    pages = -(-T // page) + 2
    shape = (pages, 2, page, Hkv, D) if layout == "tokens" else (pages, 2, Hkv, page, D)
    kv = torch.randn(shape, device="cuda").bfloat16()
    both = kv if layout == "tokens" else kv.transpose(2, 3)
    before = both.clone()
    slots = slots_for(T, pages, page, T)
    o = c.run(v=c.v, slots=slots, k_cache=both[:, 0], v_cache=both[:, 1], keep=True)
    plain = c.run()
    assert torch.equal(o["q"], plain["q"]) and torch.equal(o["k"], plain["k"])
    c.check(o["q"], c.q, c.qw)
    rows = torch.nonzero(slots >= 0)[:, 0]
    at = slots[rows] // page, slots[rows] % page
    before[at[0], 0, at[1]] = plain["k"][rows]
    before[at[0], 1, at[1]] = c.v[rows]
    assert torch.equal(both, before)  # nothing else was written


def unpack(codes):
    steps = torch.tensor(STEPS + [-x for x in STEPS], dtype=torch.float64, device="cuda")
    return torch.stack([steps[(codes & 15).long()], steps[(codes >> 4).long()]], -1).flatten(-2)


def check_fp4(codes, scales, y, tol):
    """Codes [..,D/2] and scales [..,D/16] of y [..,D] known within tol: a scale
    is the e4m3 value nearest to some max |y| / 6, a value the step nearest to
    some y / scale."""
    g, t = y.unflatten(-1, (-1, 16)), tol.unflatten(-1, (-1, 16))
    s = scales.double()
    top = g.abs().amax(-1) / 6
    slack = t.amax(-1) / 6 + 2.0 ** -23 * top
    e4m3 = torch.arange(1, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    near = (top[..., None].clamp(max=448) - e4m3).abs().amin(-1)
    assert torch.all((s - top.clamp(max=448)).abs() <= near + slack)
    x = unpack(codes).unflatten(-1, (-1, 16))
    steps = torch.tensor(STEPS, dtype=torch.float64, device="cuda")
    m = (g.abs() / s[..., None]).clamp(max=6)
    best = (m[..., None] - steps).abs().amin(-1)
    signed = g / s[..., None]
    off = (x - signed.clamp(-6, 6)).abs()
    assert torch.all(off <= best + t / s[..., None] + 2.0 ** -22 * m)


@pytest.mark.parametrize("factors", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,page,norm", [(1, 32, 8, 128, 16, True), (70, 12, 12, 64, 8, True), (200, 5, 1, 256, 24, False),
                                                 (9, 4, 2, 80, 7, True), (3000, 2, 2, 128, 64, True)])
def test_fp4_cache(T, Hq, Hkv, D, page, norm, factors):
    c = Case(T, Hq, Hkv, D, seed=T, norm=norm)
    c.v = c.v * torch.exp(2 * torch.randn(Hkv, D, device="cuda")).bfloat16()
    pages = -(-T // page) + 2
    z = mk.fp4_cache(pages, page, Hkv, D)
    for t in z.values():
        t.view(torch.uint8).random_(0, 120)
    before = {n: t.clone() for n, t in z.items()}
    f = {n: torch.exp(torch.randn(Hkv, device="cuda")) for n in ("k_factor", "v_factor")} if factors else {}
    slots = slots_for(T, pages, page, T)
    o = c.run(v=c.v, slots=slots, keep=True, **z, **f)
    c.check(o["q"], c.q, c.qw)
    k, tol = c.want(c.k, c.kw)
    rows = torch.nonzero(slots >= 0)[:, 0]
    at = slots[rows] // page, slots[rows] % page
    for name, y, t in (("k", k, tol), ("v", c.v.double(), 0 * tol)):
        factor = f.get(name + "_factor", torch.ones(Hkv, device="cuda"))
        held = factor.double()[:, None]
        codes, scales = z[name + "_cache"][at], z[name + "_scales"].view(torch.uint8)[at].view(torch.float8_e4m3fn)
        check_fp4(codes, scales, (y / held)[rows], (t / held + 2.0 ** -23 * (y / held).abs())[rows])
        value = (unpack(codes).unflatten(-1, (-1, 16)) * scales.double()[..., None]).flatten(-2) * held
        assert torch.all((o[name][rows].double() - value).abs() <= 2.0 ** -8 * value.abs() * (1 + 2.0 ** -20))
        for part in ("_cache", "_scales"):  # nothing else was written
            was, now = (d[name + part].view(torch.uint8).clone() for d in (before, z))
            was[at] = 0
            now[at] = 0
            assert torch.equal(was, now)


def test_fp4_values_are_those_of_the_definition():
    # values whose quotients are steps, middles and next to them; a head each of zeros, tiny, huge and signed values
    D, Hkv = 64, 6
    v = torch.zeros((1, Hkv, D))
    mids = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, 0])
    v[0, 0] = mids.repeat(4) * torch.tensor([1, 0.5, 2, 0.0625]).repeat_interleave(16)
    v[0, 1] = 2.0 ** -20
    v[0, 2] = 3e38
    v[0, 3, ::16] = 1.0
    v[0, 4] = torch.linspace(-1, 1, D)
    v = v.bfloat16().cuda()
    c = Case(1, 1, Hkv, D, seed=1)
    z = mk.fp4_cache(1, 1, Hkv, D)
    mk.qk_norm_rope(c.q, c.k, c.pos[0], c.inv, v=v, slots=torch.zeros(1, dtype=torch.int64, device="cuda"), **z)
    codes, scales = z["v_cache"][0, 0], z["v_scales"][0, 0].float()
    g = v[0].float().unflatten(-1, (-1, 16))
    want_scale = (g.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    assert torch.equal(scales, want_scale)
    m = (g / want_scale[..., None]).abs()
    code = (m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    assert torch.equal(unpack(codes), (torch.tensor(STEPS, device="cuda")[code] * torch.sign(g)).flatten(-2).double())


def test_fp4_nan_and_infinity():
    c = Case(2, 2, 2, 64, norm=False, seed=2)
    c.v = c.v.clone()
    c.v[0, 0, 3] = float("nan")
    c.v[0, 1, 20] = -float("inf")
    z = mk.fp4_cache(1, 2, 2, 64)
    o = c.run(v=c.v, slots=torch.arange(2, device="cuda"), keep=True, **z)
    held = o["v"].float()
    assert torch.all(torch.isnan(held[0, 0, :16])) and torch.all(torch.isfinite(held[0, 0, 16:]))
    assert held[0, 1, 20] == -6 * 448 and torch.all(held[0, 1, 16:32].abs() <= 448 * 6)
    assert torch.all(torch.isfinite(held[1]))


def test_infinite_columns_that_pass_stay():
    c = Case(1, 1, 1, 128, 64, norm=False, seed=2)
    c.q = c.q.clone()
    c.q[0, 0, 100] = float("inf")
    c.q[0, 0, 101] = float("nan")
    for c.interleaved in (False, True):
        q = c.run()["q"][0, 0].float()
        assert q[100] == float("inf") and torch.isnan(q[101])
        assert torch.isfinite(q).sum() == 126


def test_nan_stays_in_its_head():
    c = Case(3, 4, 2, 128, seed=2)
    c.q, good = c.q.clone(), c.run()["q"]
    c.q[1, 2, 5] = float("nan")
    q = c.run()["q"]
    assert torch.all(torch.isnan(q[1, 2]))
    q[1, 2] = good[1, 2]
    assert torch.equal(q, good)


def test_in_place():
    c = Case(40, 8, 2, 128, layout="apart", seed=4)
    want = c.run()
    a = mk.mk_qk_norm_rope_t(
        q=c.q.data_ptr(), k=c.k.data_ptr(), q_stride=8 * 128, q_head_stride=128, k_stride=2 * 128, k_head_stride=128,
        q_weight=c.qw.data_ptr(), k_weight=c.kw.data_ptr(), positions=c.pos.data_ptr(), inv_freq=c.inv.data_ptr(),
        q_out=c.q.data_ptr(), k_out=c.k.data_ptr(), T=40, Hq=8, Hkv=2, D=128, rot=128, axes=1, eps=EPS)
    assert mk.mk_qk_norm_rope(a) == mk.MK_OK and mk.mk_get_status() == mk.MK_OK
    assert torch.equal(c.q, want["q"]) and torch.equal(c.k, want["k"])


def test_slots_outside_the_pool_are_reported():
    c = Case(4, 2, 2, 64, seed=6)
    kv = torch.zeros((4, 2, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    pool = kv[1:3]  # what lies beside it must stay
    slots = torch.tensor([3, 16, 2 ** 40, 15], device="cuda")
    o = c.run(v=c.v, slots=slots, k_cache=pool[:, 0], v_cache=pool[:, 1], check=False)
    assert mk.mk_get_status() == mk.MK_ERR_DEVICE_FAULT
    assert mk.mk_last_error_detail()["info"] in (1, 2)
    assert mk.mk_get_status() == mk.MK_OK
    c.check(o["q"], c.q, c.qw)
    assert torch.equal(pool[0, 1, 3], c.v[0]) and torch.equal(pool[1, 1, 7], c.v[3])
    assert int((kv != 0).any(-1).any(-1).sum()) == 4


def test_offsets_past_32_bits():
    # a pool of more than 2^31 slots, and so of more than 2^32 bytes, written at its end
    D, page = 16, 2 ** 20
    pages = 2 ** 31 // page + 1
    z = {}
    for n in ("k", "v"):
        z[n + "_cache"] = torch.empty((pages, page, 1, D // 2), dtype=torch.uint8, device="cuda")
        z[n + "_scales"] = torch.empty((pages, page, 1, 1), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    c = Case(3, 1, 1, D, seed=7)
    slots = torch.tensor([pages * page - 1, 2 ** 31, 2 ** 31 - 1], device="cuda")
    o = c.run(v=c.v, slots=slots, keep=True, **z)
    at = slots // page, slots % page
    for n in ("k", "v"):
        scale = z[n + "_scales"].view(torch.uint8)[at].view(torch.float8_e4m3fn).double()
        assert torch.equal(unpack(z[n + "_cache"][at]) * scale, o[n].double())
