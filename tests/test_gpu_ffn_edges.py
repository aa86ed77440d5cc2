"""mk_moe_ffn_decode at the edges of its own plan: blocks of h that several warps
complete.  Layers, reference and tolerances are those of
test_gpu_ffn_decode.py."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk
from test_gpu_ffn_decode import Layer

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from moe_token_dispatch_persistent_gb300 import build

    build.build()
    yield
    mk.mk_release_workspace()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,H,F,E,k", [(50, 256, 512, 3, 2), (60, 2048, 1024, 2, 2), (128, 1024, 2048, 8, 4)])
def test_rows_completed_by_several_warps_are_seen(T, H, F, E, k, fp8):
    # one to many pieces of h; the blocks' rows are published by the last of three warps
    layer = Layer(T, H, F, E, k, fp8, seed=T + F)
    outs = [layer.run(check=False) for _ in range(100)]
    assert mk.mk_get_status() == mk.MK_OK
    layer.check(outs[0])
    assert all(torch.equal(o, outs[0]) for o in outs)
