"""mk_paged_attention where cached keys and values are not finite: what the
formula gives, in the columns and heads that it concerns and no others."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()


# one head a group, more than 16 and, with many sequences, groups of 32
@pytest.mark.parametrize("B,Hq,Hkv", [(3, 4, 4), (3, 24, 1), (90, 64, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinite_values(B, Hq, Hkv, D):
    lens = [700, 5, 1] + [40 + i for i in range(B - 3)]
    c = Case(lens, Hq, Hkv, D, 16, seed=D + Hq)
    want = c.run()["out"]
    spots = {0: 300, 1: 4, 2: 0}  # in sequence b, a key whose values are not finite
    values = (INF, -INF, NAN)
    for b, key in spots.items():
        page = int(c.table[b, key // 16])
        for i, v in enumerate(values):
            c.v[page, key % 16, :, 8 + i] = v
        c.v[page, key % 16, :, 12] = INF
    page = int(c.table[0, 200 // 16])
    c.v[page, 200 % 16, :, 12] = -INF  # both signs in one column
    got = c.run()["out"]
    for b in range(B):
        special = list(range(8, 11)) + [12] if b in spots else []
        rest = [i for i in range(D) if i not in special]
        assert torch.equal(got[b][:, rest], want[b][:, rest])
        if special:
            assert torch.all(got[b][:, 8] == INF) and torch.all(got[b][:, 9] == -INF)
            assert torch.all(torch.isnan(got[b][:, 10]))
            assert torch.all(torch.isnan(got[b][:, 12])) if b == 0 else torch.all(got[b][:, 12] == INF)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinite_scores(D):
    c = Case([700, 90, 90], 8, 2, D, 16, seed=D)
    want = c.run()
    c.q[0, :, 0] = c.q[0, :, 0].abs() + 1  # so that the sign of the score is known
    plain = c.run()
    for b, key, v in ((0, 300, -INF), (1, 20, NAN)):
        c.k[int(c.table[b, key // 16]), key % 16, 0, 0] = v
    got = c.run()
    # -inf: the key has no weight
    q, k, val = c.q[0].double(), c.k[c.table[0, :44].long()].flatten(0, 1)[:700].double(), c.v[
        c.table[0, :44].long()].flatten(0, 1)[:700].double()
    s = torch.einsum("hd,nd->hn", q[:4], torch.nan_to_num(k[:, 0], neginf=0.0)) * c.scale
    s[:, 300] = -INF
    ref = torch.softmax(s, 1) @ val[:, 0]
    assert torch.all((got["out"][0, :4].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -10)
    assert torch.all((got["lse"][0, :4].double() - torch.logsumexp(s, 1)).abs() <= 2.0 ** -10)
    # NaN: the heads that read it, all of them
    assert torch.all(torch.isnan(got["out"][1, :4].float())) and torch.all(torch.isnan(got["lse"][1, :4]))
    assert torch.equal(got["out"][0, 4:], plain["out"][0, 4:]) and torch.equal(got["out"][1, 4:], want["out"][1, 4:])
    assert torch.equal(got["out"][2], want["out"][2])
