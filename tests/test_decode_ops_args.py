"""The decode-step operators refuse bad arguments before any CUDA call (so
these run without a GPU), and the bindings refuse wrong tensors."""
import pytest

import moe_token_dispatch_persistent_gb300 as mk
from moe_token_dispatch_persistent_gb300 import build as mkbuild

BAD, UNSUPPORTED = mk.MK_ERR_INVALID_ARG, mk.MK_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mkbuild.build()
    return mk.lib()


# pointers are never read: 64 stands for one that is aligned
NORM = dict(x=64, x_stride=512, residual=64, residual_stride=512, weight=64, T=4, H=512, eps=1e-6, out=64, out8=64,
            scale=64, residual_out=64, stream=1)


@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(H=0), BAD), (dict(H=32769, x_stride=40000, residual_stride=40000), UNSUPPORTED),
    (dict(eps=-1e-6), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD),
    (dict(x=None), BAD), (dict(weight=None), BAD), (dict(out=None, out8=None, scale=None), BAD),
    (dict(out8=None), BAD), (dict(scale=None), BAD), (dict(residual=None), BAD),
    (dict(x=65), BAD), (dict(out=65), BAD), (dict(scale=66), BAD), (dict(residual_out=63), BAD),
    (dict(x_stride=511), BAD), (dict(residual_stride=0), BAD),
])
def test_add_rmsnorm_refusals(change, want):
    assert mk.mk_add_rmsnorm(**{**NORM, **change}) == want


def test_add_rmsnorm_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mk.add_rmsnorm(x, w)  # not on a GPU


ATTN = dict(q=64, q_stride=1024, k_cache=64, v_cache=64, page_stride=8192, token_stride=512, head_stride=128,
            block_table=64, seq_lens=64, B=2, Hq=8, Hkv=4, D=128, page_size=16, max_pages=10, num_pages=20, scale=0.1,
            out=64, lse=64, stream=1)


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hkv=3), BAD), (dict(page_size=0), BAD),
    (dict(max_pages=-1), BAD), (dict(num_pages=-1), BAD), (dict(num_pages=0), BAD),
    (dict(D=96), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(max_pages=2 ** 27), UNSUPPORTED),                # a length would pass 31 bits
    (dict(B=4096, max_pages=2 ** 17), UNSUPPORTED),         # the tiles of all sequences would
    (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
    (dict(q=None), BAD), (dict(k_cache=None), BAD), (dict(v_cache=None), BAD), (dict(block_table=None), BAD),
    (dict(seq_lens=None), BAD), (dict(out=None), BAD),
    (dict(q=66), BAD), (dict(k_cache=72), BAD), (dict(v_cache=72), BAD), (dict(out=68), BAD), (dict(lse=66), BAD),
    (dict(q_stride=1023), BAD), (dict(q_stride=1025), BAD),
    (dict(page_stride=8196), BAD), (dict(token_stride=508), BAD), (dict(head_stride=-128), BAD),
])
def test_paged_attention_refusals(change, want):
    assert mk.mk_paged_attention(**{**ATTN, **change}) == want


def test_paged_attention_workspace_size():
    one = mk.mk_paged_attention_workspace_size(1, 32, 8)
    assert 0 < one <= mk.mk_paged_attention_workspace_size(4096, 32, 8)
    assert mk.mk_paged_attention_workspace_size(1, 32, 5) == 0
    assert mk.mk_paged_attention_workspace_size(4097, 32, 8) == 0
    assert mk.mk_paged_attention_workspace_size(-1, 32, 8) == 0


def test_paged_attention_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    q, kv = torch.zeros((1, 8, 64), dtype=torch.bfloat16), torch.zeros((2, 16, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mk.paged_attention(q, kv, kv, torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32))


FFN = dict(x=64, x_scale=None, logits=64, T=4, H=512, E=8, k=2, W1=64, W3=64, W2=64, W1_scale=None, W3_scale=None,
           W2_scale=None, F=1024, weights=mk.MK_WEIGHT_BF16, out=64, stream=1)
FFN8 = dict(FFN, x_scale=64, W1_scale=64, W3_scale=64, W2_scale=64, weights=mk.MK_WEIGHT_E4M3)


@pytest.mark.parametrize("base", [FFN, FFN8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(T=129), UNSUPPORTED), (dict(k=0), BAD), (dict(k=9, E=16), BAD), (dict(E=1), BAD),
    (dict(E=257), UNSUPPORTED), (dict(H=0), BAD), (dict(H=500), BAD), (dict(F=1000), BAD),
    (dict(H=32768 + 128), UNSUPPORTED), (dict(F=32768 + 128), UNSUPPORTED), (dict(weights=2), BAD),
    (dict(x=None), BAD), (dict(logits=None), BAD), (dict(W1=None), BAD), (dict(W3=None), BAD), (dict(W2=None), BAD),
    (dict(out=None), BAD), (dict(x=72), BAD), (dict(W2=72), BAD), (dict(out=72), BAD), (dict(logits=66), BAD),
])
def test_moe_ffn_decode_refusals(base, change, want):
    assert mk.mk_moe_ffn_decode(**{**base, **change}) == want


@pytest.mark.parametrize("name", ["x_scale", "W1_scale", "W3_scale", "W2_scale"])
def test_moe_ffn_decode_scales_belong_to_8_bits(name):
    assert mk.mk_moe_ffn_decode(**{**FFN, name: 64}) == BAD
    assert mk.mk_moe_ffn_decode(**{**FFN8, name: None}) == BAD
    assert mk.mk_moe_ffn_decode(**{**FFN8, name: 66}) == BAD
    assert mk.mk_moe_ffn_decode(**{**FFN8, "H": 576}) == BAD  # a multiple of 64 only


def test_moe_ffn_decode_workspace_size():
    a = mk.mk_moe_ffn_decode_workspace_size(1, 512, 1024, 8, 2)
    assert 0 < a < mk.mk_moe_ffn_decode_workspace_size(128, 512, 1024, 8, 2)
    assert mk.mk_moe_ffn_decode_workspace_size(129, 512, 1024, 8, 2) == 0
    assert mk.mk_moe_ffn_decode_workspace_size(1, 576, 1024, 8, 2, mk.MK_WEIGHT_E4M3) == 0


def test_moe_ffn_decode_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((4, 64, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mk.moe_ffn_decode(x, torch.zeros((2, 4)), w, w, w, 2)
