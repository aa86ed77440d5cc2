"""The cache's operators refuse bad arguments before any CUDA call (so these run
without a GPU), and the bindings refuse wrong tensors."""
import ctypes

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
ROPE = dict(q=64, k=64, q_stride=1024, q_head_stride=128, k_stride=512, k_head_stride=128, q_weight=64, k_weight=64,
            positions=64, inv_freq=64, q_out=64, k_out=64, T=4, Hq=8, Hkv=4, D=128, rot=128, axes=1, eps=1e-6)
BF16 = dict(ROPE, v=64, v_stride=512, v_head_stride=128, slots=64, k_cache=64, v_cache=64, page_stride=8192,
            token_stride=512, head_stride=128, cache=mk.MK_CACHE_BF16, page_size=16, num_pages=20)
FP4 = dict(BF16, k_scales=64, v_scales=64, page_stride=4096, token_stride=256, head_stride=64, scale_page_stride=512,
           scale_token_stride=32, scale_head_stride=8, k_factor=64, v_factor=64, v_out=64, cache=mk.MK_CACHE_FP4)


def rope(fields):
    return mk.mk_qk_norm_rope(mk.mk_qk_norm_rope_t(**fields), 1)


def test_argument_block_has_one_layout():
    assert ctypes.sizeof(mk.mk_qk_norm_rope_t) == mk._rope_args.size == 296
    assert mk.mk_qk_norm_rope(None, 1) == BAD


@pytest.mark.parametrize("base", [ROPE, BF16, FP4], ids=["none", "bf16", "fp4"])
@pytest.mark.parametrize("change,want", [
    (dict(T=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(D=120), BAD), (dict(D=0), BAD), (dict(D=272, rot=128), UNSUPPORTED),
    (dict(rot=136), BAD), (dict(rot=144), BAD), (dict(rot=-16), BAD), (dict(rot=24), BAD),
    (dict(axes=0), BAD), (dict(axes=5), UNSUPPORTED), (dict(axes=2), BAD), (dict(pairs=2), BAD), (dict(cache=3), BAD),
    (dict(cache=-1), BAD), (dict(reserved=1), BAD), (dict(Hq=65537), UNSUPPORTED),
    (dict(eps=-1e-6), BAD), (dict(eps=NAN), BAD), (dict(eps=INF), BAD),
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(q_out=None), BAD), (dict(positions=None), BAD), (dict(inv_freq=None), BAD),
    (dict(q=72), BAD), (dict(k=72), BAD), (dict(q_out=72), BAD), (dict(k_out=72), BAD), (dict(q_weight=66), BAD),
    (dict(k_weight=72), BAD), (dict(positions=66), BAD), (dict(inv_freq=66), BAD),
    (dict(q_stride=1028), BAD), (dict(k_head_stride=132), BAD), (dict(q_head_stride=-128), BAD),
])
def test_qk_norm_rope_refusals(base, change, want):
    assert rope({**base, **change}) == want


@pytest.mark.parametrize("base", [BF16, FP4], ids=["bf16", "fp4"])
@pytest.mark.parametrize("change", [
    dict(v=None), dict(v=72), dict(v_stride=516), dict(slots=None), dict(slots=68), dict(k_cache=None), dict(v_cache=None),
    dict(k_cache=66), dict(v_cache=66), dict(page_size=0), dict(num_pages=-1), dict(page_stride=-16), dict(token_stride=-8),
    dict(head_stride=2), dict(page_stride=8194)])
def test_qk_norm_rope_cache_refusals(base, change):
    assert rope({**base, **change}) == BAD


@pytest.mark.parametrize("change", [dict(k_scales=None), dict(v_scales=None), dict(scale_page_stride=-1), dict(scale_head_stride=-8),
                                    dict(k_factor=66), dict(v_factor=66), dict(v_out=72)])
def test_qk_norm_rope_scales_refusals(change):
    assert rope({**FP4, **change}) == BAD


def test_qk_norm_rope_outputs_belong_to_their_form():
    assert rope({**ROPE, "k_out": None}) == BAD   # without a cache the keys go nowhere
    assert rope({**BF16, "v_out": 64}) == BAD     # a bf16 cache holds the values as they are


def test_qk_norm_rope_pair_axis_is_checked():
    each = (ctypes.c_uint8 * 64)(*([0, 1] * 31 + [0, 2]))
    assert rope({**ROPE, "axes": 2, "pair_axis": ctypes.addressof(each)}) == BAD
    each[0] = 1
    assert rope({**ROPE, "axes": 1, "pair_axis": ctypes.addressof(each)}) == BAD


def test_qk_norm_rope_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mk.qk_norm_rope(q, q, torch.zeros(2, dtype=torch.int32), torch.zeros(32))  # not on a GPU


ATTN = dict(q=64, q_stride=1024, k_cache=64, v_cache=64, page_stride=4096, token_stride=256, head_stride=64, k_scales=64,
            v_scales=64, scale_page_stride=512, scale_token_stride=32, scale_head_stride=8, k_factor=64, v_factor=64,
            block_table=64, seq_lens=64, B=2, Hq=8, Hkv=4, D=128, page_size=16, max_pages=10, num_pages=20, scale=0.1, out=64,
            lse=64, stream=1)


@pytest.mark.parametrize("change,want", [
    (dict(B=-1), BAD), (dict(Hq=0), BAD), (dict(Hkv=0), BAD), (dict(Hkv=3), BAD), (dict(page_size=0), BAD),
    (dict(max_pages=-1), BAD), (dict(num_pages=-1), BAD), (dict(num_pages=0), BAD),
    (dict(D=96), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(max_pages=2 ** 27), UNSUPPORTED),                # a length would pass 31 bits
    (dict(B=4096, max_pages=2 ** 17), UNSUPPORTED),         # the tiles of all sequences would
    (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
    (dict(q=None), BAD), (dict(k_cache=None), BAD), (dict(v_cache=None), BAD), (dict(k_scales=None), BAD),
    (dict(v_scales=None), BAD), (dict(block_table=None), BAD), (dict(seq_lens=None), BAD), (dict(out=None), BAD),
    (dict(q=72), BAD), (dict(k_cache=72), BAD), (dict(v_cache=72), BAD), (dict(k_scales=68), BAD), (dict(v_scales=68), BAD),
    (dict(out=68), BAD), (dict(lse=66), BAD), (dict(k_factor=66), BAD), (dict(v_factor=66), BAD),
    (dict(q_stride=1020), BAD), (dict(q_stride=1028), BAD),
    (dict(page_stride=4104), BAD), (dict(token_stride=248), BAD), (dict(head_stride=-64), BAD),
    (dict(scale_page_stride=508), BAD), (dict(scale_token_stride=36), BAD), (dict(scale_head_stride=-8), BAD),
])
def test_paged_attention_fp4_refusals(change, want):
    assert mk.mk_paged_attention_fp4(**{**ATTN, **change}) == want


def test_paged_attention_fp4_workspace_size():
    one = mk.mk_paged_attention_fp4_workspace_size(1, 32, 8)
    assert 0 < one <= mk.mk_paged_attention_fp4_workspace_size(4096, 32, 8)
    for args in ((1, 32, 5), (4097, 32, 8), (-1, 32, 8)):
        assert mk.mk_paged_attention_fp4_workspace_size(*args) == 0


def test_paged_attention_fp4_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros((1, 8, 64), dtype=torch.bfloat16)
    z = mk.fp4_cache(2, 16, 4, 64, device="cpu")
    assert z["k_cache"].shape == (2, 16, 4, 32) and z["k_scales"].shape == (2, 16, 4, 4)
    with pytest.raises(ValueError):
        mk.paged_attention_fp4(q, block_table=torch.zeros((1, 2), dtype=torch.int32), seq_lens=torch.ones(1, dtype=torch.int32), **z)


POOL = dict(block_table=64, seq_lens=64, refs=64, rows=4, max_pages=10, num_pages=20, page_size=16, n=2, stream=1)
BUF = dict(caches=[(64, 1024, 512)])
FORK = (mk.mk_fork_sequences, dict(POOL, parent=64, child=64))
FREE = (mk.mk_free_sequences, dict(POOL, seqs=64))
EXTEND = (mk.mk_extend_sequences, dict(POOL, seqs=64, count=64, most=3, slots=64, **BUF))
COMPACT = (mk.mk_compact_pages, {k: v for k, v in dict(POOL, table_out=64, refs_out=64, **BUF).items() if k != "n"})
COPY = (mk.mk_copy_pages, dict(num_pages=20, src=64, dst=64, n=2, stream=1, **BUF))
ENTRIES = [FORK, FREE, EXTEND, COMPACT]
NAMES = ["fork", "free", "extend", "compact"]


@pytest.mark.parametrize("entry", ENTRIES, ids=NAMES)
@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), BAD), (dict(max_pages=-1), BAD), (dict(num_pages=-1), BAD), (dict(page_size=0), BAD),
    (dict(rows=65537), UNSUPPORTED), (dict(max_pages=2 ** 27), UNSUPPORTED), (dict(num_pages=2 ** 30 + 1), UNSUPPORTED),
    (dict(block_table=None), BAD), (dict(seq_lens=None), BAD), (dict(refs=None), BAD),
    (dict(block_table=66), BAD), (dict(seq_lens=66), BAD), (dict(refs=66), BAD),
])
def test_pool_refusals(entry, change, want):
    call, fields = entry
    assert call(**{**fields, **change}) == want


@pytest.mark.parametrize("entry", [FORK, FREE, EXTEND, COPY], ids=["fork", "free", "extend", "copy"])
def test_list_refusals(entry):
    call, fields = entry
    for name in ("parent", "child", "seqs", "count", "src", "dst"):
        if name in fields:
            assert call(**{**fields, name: None}) == BAD
            assert call(**{**fields, name: 66}) == BAD
    assert call(**{**fields, "n": -1}) == BAD
    if call is not mk.mk_copy_pages:
        assert call(**{**fields, "n": 4097}) == UNSUPPORTED


@pytest.mark.parametrize("entry", [EXTEND, COMPACT, COPY], ids=["extend", "compact", "copy"])
@pytest.mark.parametrize("caches", [[(None, 1024, 512)], [(64, 511, 512)], [(64, 1024, 0)], [(64, 2 ** 33, 2 ** 31 + 1)],
                                    [(64, 1024, 512), (64, -1, 512)]])
def test_buffer_refusals(entry, caches):
    call, fields = entry
    assert call(**{**fields, "caches": caches}) == BAD


def test_extend_and_compact_refusals():
    assert mk.mk_extend_sequences(**{**EXTEND[1], "most": -1}) == BAD
    assert mk.mk_extend_sequences(**{**EXTEND[1], "slots": 68}) == BAD
    for name in ("table_out", "refs_out"):
        assert mk.mk_compact_pages(**{**COMPACT[1], name: None}) == BAD
        assert mk.mk_compact_pages(**{**COMPACT[1], name: 66}) == BAD


def test_pages_workspace_size():
    assert 0 < mk.mk_pages_workspace_size(10, 20, 2) < mk.mk_pages_workspace_size(1000, 20, 4096)
    for args in ((-1, 20, 2), (10, -1, 2), (10, 20, 4097), (10, 20, -1)):
        assert mk.mk_pages_workspace_size(*args) == 0


def test_page_operators_bindings_refuse_wrong_tensors():
    torch = pytest.importorskip("torch")
    z = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros((4, 4), dtype=torch.int32)
    for call in (lambda: mk.copy_pages([], z, z), lambda: mk.fork_sequences(table, z, z, z, z, 4),
                 lambda: mk.free_sequences(table, z, z, z, 4), lambda: mk.extend_sequences(table, z, z, z, z, 1, [], 4),
                 lambda: mk.compact_pages(table, z, z, [], 4)):
        with pytest.raises(ValueError):
            call()
