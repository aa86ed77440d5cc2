"""GB300-native MoE token dispatch + expert GEMM in one persistent kernel.

Thin ctypes binding over the C ABI in ``include/mk.h``: the functions below
carry the C names and only marshal arguments (tensor -> device pointer,
current torch stream -> cudaStream_t).  Every step of the path runs in the
CUDA library ``_build/libmk.so``; there is no CPU fallback.  When the library
is missing every call raises ``MkLibraryMissing`` (build it with
``moe_token_dispatch_persistent_gb300.build.build()``).
"""
from __future__ import annotations

import ctypes
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmk.so")

MK_OK = 0
MK_ERR_INVALID_ARG = 1
MK_ERR_UNSUPPORTED = 2
MK_ERR_CUDA = 3
MK_ERR_TIMEOUT = 4
MK_ERR_DEVICE_FAULT = 5
MK_ERR_NOT_IMPLEMENTED = 6
MK_ERR_WORKSPACE = 7

MK_MODE_FUSED = 0
MK_MODE_UNFUSED = 1
MK_MODE_DISPATCH_ONLY = 2
MK_OUT_BF16 = 0
MK_OUT_F32 = 1
MK_FAULT_NONE = 0
MK_FAULT_DROP_TILE_FLAG = 1
MK_MMA_AUTO = 0
MK_MMA_SINGLE = 1
MK_MMA_PAIR = 2
MK_MMA_WIDE = 3
MK_GATHER_AUTO = 0
MK_GATHER_STAGED = 1
MK_GATHER_DIRECT = 2
MK_GATHER_GATHER4 = 3
MK_WEIGHT_BF16 = 0
MK_WEIGHT_E4M3 = 1
MK_CACHE_NONE = 0
MK_CACHE_BF16 = 1
MK_CACHE_FP4 = 2
MK_PAIR_HALVES = 0
MK_PAIR_NEIGHBOURS = 1

# Entry points declared in include/mk.h (checked by the tests).
ABI_FUNCTIONS = (
    "mk_config_default",
    "mk_moe_dispatch_gemm",
    "mk_moe_dispatch_gemm_ex",
    "mk_moe_dispatch_gemm_combine",
    "mk_moe_dispatch_gated",
    "mk_moe_dispatch_gemm_host",
    "mk_moe_dispatch_gemm_noalloc",
    "mk_moe_ep_sim",
    "mk_moe_ep_sim_gated",
    "mk_ep_workspace_size",
    "mk_add_rmsnorm",
    "mk_paged_attention",
    "mk_paged_attention_workspace_size",
    "mk_moe_ffn_decode",
    "mk_moe_ffn_decode_workspace_size",
    "mk_qk_norm_rope",
    "mk_paged_attention_fp4",
    "mk_paged_attention_fp4_workspace_size",
    "mk_copy_pages",
    "mk_fork_sequences",
    "mk_free_sequences",
    "mk_extend_sequences",
    "mk_compact_pages",
    "mk_pages_workspace_size",
    "mk_workspace_size",
    "mk_get_status",
    "mk_last_error_detail",
    "mk_last_launch_info",
    "mk_read_trace",
    "mk_release_workspace",
    "mk_status_string",
    "mk_version",
)


class MkLibraryMissing(RuntimeError):
    pass


class MkError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_name(status)} ({status})")


class mk_config_t(ctypes.Structure):
    _fields_ = [
        ("mode", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("dispatch_ctas", ctypes.c_int32),
        ("grid_ctas", ctypes.c_int32),
        ("n_group", ctypes.c_int32),
        ("debug_fault", ctypes.c_int32),
        ("spin_limit_ns", ctypes.c_int64),
        ("trace", ctypes.c_int32),
        ("l2_prefetch", ctypes.c_int32),
        ("mma_pair", ctypes.c_int32),
        ("gather", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 4),
    ]


class mk_launch_info_t(ctypes.Structure):
    _fields_ = [
        ("grid_ctas", ctypes.c_int32),
        ("dispatch_ctas", ctypes.c_int32),
        ("launches", ctypes.c_int32),
        ("n_group", ctypes.c_int32),
        ("workspace_bytes", ctypes.c_int64),
        ("mma_pair", ctypes.c_int32),
        ("gather", ctypes.c_int32),
        ("route_lanes", ctypes.c_int32),
        ("route_chunks", ctypes.c_int32),
    ]


_lib_handle = None
_p = ctypes.c_void_p
_i = ctypes.c_int
_i64 = ctypes.c_int64


class mk_qk_norm_rope_t(ctypes.Structure):
    _fields_ = (
        [(n, _p) for n in ("q", "k", "v")]
        + [(n, _i64) for n in ("q_stride", "q_head_stride", "k_stride", "k_head_stride", "v_stride", "v_head_stride")]
        + [("q_weight", _p), ("k_weight", _p), ("positions", _p), ("position_stride", _i64), ("inv_freq", _p)]
        + [(n, _p) for n in ("pair_axis", "q_out", "k_out", "v_out", "slots", "k_cache", "v_cache")]
        + [(n, _i64) for n in ("page_stride", "token_stride", "head_stride")]
        + [("k_scales", _p), ("v_scales", _p)]
        + [(n, _i64) for n in ("scale_page_stride", "scale_token_stride", "scale_head_stride")]
        + [("k_factor", _p), ("v_factor", _p)]
        + [(n, ctypes.c_int32) for n in ("T", "Hq", "Hkv", "D", "rot", "axes", "pairs", "cache", "page_size", "num_pages")]
        + [("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]
    )


# The same in order, for a call's arguments packed at once (a field at a time costs 6 us).
_rope_args = struct.Struct("=3Q6q3QqQ7Q3q2Q3q2Q10ifi")


def lib(path: str | None = None) -> ctypes.CDLL:
    """The loaded CUDA library (raises MkLibraryMissing if it was not built)."""
    global _lib_handle
    if _lib_handle is not None and path is None:
        return _lib_handle
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise MkLibraryMissing(f"CUDA library not found at {p}; build it first")
    h = ctypes.CDLL(p)
    h.mk_config_default.argtypes = [ctypes.POINTER(mk_config_t)]
    h.mk_config_default.restype = None
    sig = [_p, _p, _i, _i, _i, _i, _p, _i, _p, _p, _p, _p, _p]
    h.mk_moe_dispatch_gemm.argtypes = sig
    h.mk_moe_dispatch_gemm.restype = _i
    h.mk_moe_dispatch_gemm_ex.argtypes = sig + [ctypes.POINTER(mk_config_t), _p, ctypes.c_size_t]
    h.mk_moe_dispatch_gemm_ex.restype = _i
    h.mk_moe_dispatch_gemm_combine.argtypes = sig[:-1] + [_p, _p, ctypes.POINTER(mk_config_t), _p,
                                                           ctypes.c_size_t]
    h.mk_moe_dispatch_gemm_combine.restype = _i
    h.mk_moe_dispatch_gated.argtypes = [_p, _p, _i, _i, _i, _i, _p, _p, _i, _p, _p, _p, _p, _p,
                                        ctypes.POINTER(mk_config_t), _p, ctypes.c_size_t]
    h.mk_moe_dispatch_gated.restype = _i
    h.mk_moe_dispatch_gemm_host.argtypes = sig + [ctypes.POINTER(mk_config_t)]
    h.mk_moe_dispatch_gemm_host.restype = _i
    h.mk_moe_dispatch_gemm_noalloc.argtypes = sig + [ctypes.POINTER(mk_config_t)]
    h.mk_moe_dispatch_gemm_noalloc.restype = _i
    h.mk_moe_ep_sim.argtypes = [_p, _p, _i, _i, _i, _i, _p, _i, _i, _p, _p, _p, _p, _p, _p,
                                ctypes.POINTER(mk_config_t), _p, ctypes.c_size_t]
    h.mk_moe_ep_sim.restype = _i
    h.mk_moe_ep_sim_gated.argtypes = [_p, _p, _i, _i, _i, _i, _p, _p, _i, _i, _p, _p, _p, _p, _p, _p,
                                      ctypes.POINTER(mk_config_t), _p, ctypes.c_size_t]
    h.mk_moe_ep_sim_gated.restype = _i
    h.mk_ep_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
    h.mk_ep_workspace_size.restype = ctypes.c_size_t
    h.mk_workspace_size.argtypes = [_i, _i, _i, _i, _i, ctypes.POINTER(mk_config_t)]
    h.mk_workspace_size.restype = ctypes.c_size_t
    h.mk_add_rmsnorm.argtypes = [_p, _i64, _p, _i64, _p, _i, _i, ctypes.c_float, _p, _p, _p, _p, _p]
    h.mk_add_rmsnorm.restype = _i
    h.mk_paged_attention.argtypes = [_p, _i64, _p, _p, _i64, _i64, _i64, _p, _p, _i, _i, _i, _i, _i, _i, _i,
                                     ctypes.c_float, _p, _p, _p, _p, ctypes.c_size_t]
    h.mk_paged_attention.restype = _i
    h.mk_paged_attention_workspace_size.argtypes = [_i, _i, _i]
    h.mk_paged_attention_workspace_size.restype = ctypes.c_size_t
    h.mk_moe_ffn_decode.argtypes = [_p, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p, _p, _p, _i, _i, _p, _p, _p,
                                    ctypes.c_size_t]
    h.mk_moe_ffn_decode.restype = _i
    h.mk_moe_ffn_decode_workspace_size.argtypes = [_i, _i, _i, _i, _i, _i]
    h.mk_moe_ffn_decode_workspace_size.restype = ctypes.c_size_t
    h.mk_qk_norm_rope.argtypes = [_p, _p]
    h.mk_qk_norm_rope.restype = _i
    h.mk_paged_attention_fp4.argtypes = [_p, _i64, _p, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p,
                                         _i, _i, _i, _i, _i, _i, _i, ctypes.c_float, _p, _p, _p, _p, ctypes.c_size_t]
    h.mk_paged_attention_fp4.restype = _i
    h.mk_paged_attention_fp4_workspace_size.argtypes = [_i, _i, _i]
    h.mk_paged_attention_fp4_workspace_size.restype = ctypes.c_size_t
    pool = [_p, _p, _p, _i, _i, _i, _i]
    buffers = [_p, _p, _p, _i]
    end = [_p, _p, ctypes.c_size_t]
    h.mk_copy_pages.argtypes = buffers + [_i, _p, _p, _i, _p]
    h.mk_copy_pages.restype = _i
    h.mk_fork_sequences.argtypes = pool + [_p, _p, _i] + end
    h.mk_fork_sequences.restype = _i
    h.mk_free_sequences.argtypes = pool + [_p, _i, _p]
    h.mk_free_sequences.restype = _i
    h.mk_extend_sequences.argtypes = pool + [_p, _p, _i, _i, _p] + buffers + end
    h.mk_extend_sequences.restype = _i
    h.mk_compact_pages.argtypes = pool + [_p, _p] + buffers + end
    h.mk_compact_pages.restype = _i
    h.mk_pages_workspace_size.argtypes = [_i, _i, _i]
    h.mk_pages_workspace_size.restype = ctypes.c_size_t
    h.mk_get_status.argtypes = [_p]
    h.mk_get_status.restype = _i
    h.mk_last_error_detail.argtypes = [ctypes.POINTER(ctypes.c_int32)] * 3
    h.mk_last_error_detail.restype = None
    h.mk_last_launch_info.argtypes = [ctypes.POINTER(mk_launch_info_t)]
    h.mk_last_launch_info.restype = None
    h.mk_read_trace.argtypes = [_p, _p, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_uint64), ctypes.c_size_t]
    h.mk_read_trace.restype = _i
    h.mk_release_workspace.argtypes = []
    h.mk_release_workspace.restype = None
    h.mk_status_string.argtypes = [_i]
    h.mk_status_string.restype = ctypes.c_char_p
    h.mk_version.argtypes = []
    h.mk_version.restype = _i
    if path is None:
        _lib_handle = h
    return h


def status_name(s: int) -> str:
    try:
        return lib().mk_status_string(int(s)).decode()
    except MkLibraryMissing:
        return str(s)


# ------------------------------------------------------------ marshalling --

def _ptr(v):
    if v is None:
        return None
    if hasattr(v, "data_ptr"):
        return v.data_ptr() or None
    return int(v) or None


def _stream(s):
    if s is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


def _check(status: int, what: str):
    if status != MK_OK:
        raise MkError(status, what)


# ----------------------------------------------------------- C-named calls --

def mk_config_default() -> mk_config_t:
    c = mk_config_t()
    lib().mk_config_default(ctypes.byref(c))
    return c


def mk_version() -> int:
    return int(lib().mk_version())


def mk_status_string(s: int) -> str:
    return lib().mk_status_string(int(s)).decode()


def mk_workspace_size(T, H, F, E, k, cfg: mk_config_t | None = None) -> int:
    return int(lib().mk_workspace_size(T, H, F, E, k, ctypes.byref(cfg) if cfg is not None else None))


def mk_moe_dispatch_gemm(x, logits, T, H, E, k, W, F, y_sorted, src_index, expert_offsets, gate_w, stream=None) -> int:
    return int(lib().mk_moe_dispatch_gemm(_ptr(x), _ptr(logits), T, H, E, k, _ptr(W), F, _ptr(y_sorted),
                                          _ptr(src_index), _ptr(expert_offsets), _ptr(gate_w), _stream(stream)))


def mk_moe_dispatch_gemm_ex(x, logits, T, H, E, k, W, F, y_sorted, src_index, expert_offsets, gate_w, stream=None,
                            cfg: mk_config_t | None = None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_moe_dispatch_gemm_ex(_ptr(x), _ptr(logits), T, H, E, k, _ptr(W), F, _ptr(y_sorted),
                                             _ptr(src_index), _ptr(expert_offsets), _ptr(gate_w), _stream(stream),
                                             ctypes.byref(cfg) if cfg is not None else None, _ptr(workspace),
                                             int(ws_bytes)))


def mk_moe_dispatch_gemm_combine(x, logits, T, H, E, k, W, F, y_sorted, src_index, expert_offsets, gate_w, out,
                                 stream=None, cfg: mk_config_t | None = None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_moe_dispatch_gemm_combine(_ptr(x), _ptr(logits), T, H, E, k, _ptr(W), F, _ptr(y_sorted),
                                                  _ptr(src_index), _ptr(expert_offsets), _ptr(gate_w), _ptr(out),
                                                  _stream(stream), ctypes.byref(cfg) if cfg is not None else None,
                                                  _ptr(workspace), int(ws_bytes)))


def mk_moe_dispatch_gated(x, logits, T, H, E, k, W1, W3, F, h_sorted, src_index, expert_offsets, gate_w,
                          stream=None, cfg: mk_config_t | None = None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_moe_dispatch_gated(_ptr(x), _ptr(logits), T, H, E, k, _ptr(W1), _ptr(W3), F, _ptr(h_sorted),
                                           _ptr(src_index), _ptr(expert_offsets), _ptr(gate_w), _stream(stream),
                                           ctypes.byref(cfg) if cfg is not None else None, _ptr(workspace),
                                           int(ws_bytes)))


def moe_gated(x, logits, W1, W3, k, cfg: mk_config_t | None = None, stream=None, check=True):
    """Dispatch + gated expert FFN on torch tensors; ``y_sorted`` holds h."""
    T, H = x.shape
    E, _, F = W1.shape
    o = alloc_outputs(T, F, E, k, cfg.out_dtype if cfg is not None else MK_OUT_BF16, x.device)
    st = mk_moe_dispatch_gated(x, logits, T, H, E, k, W1, W3, F, o["y_sorted"], o["src_index"],
                               o["expert_offsets"], o["gate_w"], stream, cfg)
    _check(st, "mk_moe_dispatch_gated")
    if check:
        _check(mk_get_status(stream), "device status")
    return o


def moe_layer(x, logits, W, k, cfg: mk_config_t | None = None, stream=None, check=True):
    """Dispatch + expert GEMM + combine on torch tensors; returns the outputs
    of moe_dispatch_gemm plus ``out[T,F]``."""
    import torch

    T, H = x.shape
    E, _, F = W.shape
    o = alloc_outputs(T, F, E, k, cfg.out_dtype if cfg is not None else MK_OUT_BF16, x.device)
    o["out"] = torch.empty((T, F), dtype=o["y_sorted"].dtype, device=x.device)
    st = mk_moe_dispatch_gemm_combine(x, logits, T, H, E, k, W, F, o["y_sorted"], o["src_index"],
                                      o["expert_offsets"], o["gate_w"], o["out"], stream, cfg)
    _check(st, "mk_moe_dispatch_gemm_combine")
    if check:
        _check(mk_get_status(stream), "device status")
    return o


def mk_moe_ep_sim(x, logits, T, H, E, k, W, F, ranks, y_tok, src_index, expert_offsets, gate_w, out=None,
                  stream=None, cfg: mk_config_t | None = None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_moe_ep_sim(_ptr(x), _ptr(logits), T, H, E, k, _ptr(W), F, ranks, _ptr(y_tok),
                                   _ptr(src_index), _ptr(expert_offsets), _ptr(gate_w), _ptr(out), _stream(stream),
                                   ctypes.byref(cfg) if cfg is not None else None, _ptr(workspace), int(ws_bytes)))


def mk_moe_ep_sim_gated(x, logits, T, H, E, k, W1, W3, F, ranks, h_tok, src_index, expert_offsets, gate_w,
                        out=None, stream=None, cfg: mk_config_t | None = None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_moe_ep_sim_gated(_ptr(x), _ptr(logits), T, H, E, k, _ptr(W1), _ptr(W3), F, ranks,
                                         _ptr(h_tok), _ptr(src_index), _ptr(expert_offsets), _ptr(gate_w), _ptr(out),
                                         _stream(stream), ctypes.byref(cfg) if cfg is not None else None,
                                         _ptr(workspace), int(ws_bytes)))


def mk_ep_workspace_size(T, H, F, E, k, ranks) -> int:
    return int(lib().mk_ep_workspace_size(T, H, F, E, k, ranks))


def moe_ep_sim(x, logits, W, k, ranks, cfg: mk_config_t | None = None, stream=None, combine=True, check=True,
               W3=None):
    """Expert parallelism over ``ranks`` logical ranks simulated on one GPU;
    returns ``y_tok[T*k,F]`` (token-major), the receive metadata
    (``src_index``, ``gate_w``, ``expert_offsets``) and, with ``combine``,
    ``out[T,F]``.  With ``W3`` the experts are the gated (SwiGLU) FFN with
    ``W`` as W1, and ``y_tok`` holds h."""
    import torch

    T, H = x.shape
    E, _, F = W.shape
    o = alloc_outputs(T, F, E, k, cfg.out_dtype if cfg is not None else MK_OUT_BF16, x.device)
    o["y_tok"] = o.pop("y_sorted")
    o["out"] = torch.empty((T, F), dtype=o["y_tok"].dtype, device=x.device) if combine else None
    if W3 is None:
        st = mk_moe_ep_sim(x, logits, T, H, E, k, W, F, ranks, o["y_tok"], o["src_index"], o["expert_offsets"],
                           o["gate_w"], o["out"], stream, cfg)
    else:
        st = mk_moe_ep_sim_gated(x, logits, T, H, E, k, W, W3, F, ranks, o["y_tok"], o["src_index"],
                                 o["expert_offsets"], o["gate_w"], o["out"], stream, cfg)
    _check(st, "mk_moe_ep_sim")
    if check:
        _check(mk_get_status(stream), "device status")
    return o


def mk_moe_dispatch_gemm_host(x_host, logits_host, T, H, E, k, W, F, y_host, src_host, offsets_host, gate_host,
                              stream=None, cfg: mk_config_t | None = None) -> int:
    return int(lib().mk_moe_dispatch_gemm_host(_ptr(x_host), _ptr(logits_host), T, H, E, k, _ptr(W), F,
                                               _ptr(y_host), _ptr(src_host), _ptr(offsets_host), _ptr(gate_host),
                                               _stream(stream), ctypes.byref(cfg) if cfg is not None else None))


MK_NOALLOC_SCRATCH_BYTES = 64 << 20


def mk_moe_dispatch_gemm_noalloc(x, logits, T, H, E, k, W, F, y_sorted, src_index, expert_offsets, gate_w,
                                 stream=None, cfg: mk_config_t | None = None) -> int:
    """Allocation-free call: the library's fixed 64 MiB device array is the
    workspace (for callers that may not allocate device memory while they
    run this, e.g. inside a framework that owns the device-memory budget).
    Calls that overlap on the GPU share that array and race."""
    return int(lib().mk_moe_dispatch_gemm_noalloc(_ptr(x), _ptr(logits), T, H, E, k, _ptr(W), F, _ptr(y_sorted),
                                                  _ptr(src_index), _ptr(expert_offsets), _ptr(gate_w),
                                                  _stream(stream), ctypes.byref(cfg) if cfg is not None else None))


def mk_get_status(stream=None) -> int:
    return int(lib().mk_get_status(_stream(stream)))


def mk_last_error_detail():
    a, b, c = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    lib().mk_last_error_detail(ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
    return dict(site=a.value, cta=b.value, info=c.value)


def mk_last_launch_info() -> dict:
    i = mk_launch_info_t()
    lib().mk_last_launch_info(ctypes.byref(i))
    return {f: getattr(i, f) for f, _ in mk_launch_info_t._fields_}


def mk_read_trace(T, H, E, k, n_ctas, stream=None, workspace=None):
    import numpy as np

    buf = (ctypes.c_uint64 * (n_ctas * 16))()
    _check(int(lib().mk_read_trace(_stream(stream), _ptr(workspace), T, H, E, k, buf, n_ctas * 16)), "mk_read_trace")
    return np.frombuffer(buf, dtype=np.uint64).reshape(n_ctas, 16).copy()


def mk_release_workspace() -> None:
    lib().mk_release_workspace()


# ------------------------------------------------------------- convenience --

def make_config(mode=MK_MODE_FUSED, out_dtype=MK_OUT_BF16, dispatch_ctas=0, grid_ctas=0, n_group=0,
                debug_fault=MK_FAULT_NONE, spin_limit_ns=0, trace=0, l2_prefetch=0,
                mma_pair=0, gather=0) -> mk_config_t:
    c = mk_config_default()
    c.mode, c.out_dtype, c.dispatch_ctas, c.grid_ctas = mode, out_dtype, dispatch_ctas, grid_ctas
    c.n_group, c.debug_fault, c.spin_limit_ns, c.trace = n_group, debug_fault, spin_limit_ns, trace
    c.l2_prefetch, c.mma_pair, c.gather = l2_prefetch, mma_pair, gather
    return c


def alloc_outputs(T, F, E, k, out_dtype=MK_OUT_BF16, device="cuda"):
    """Output tensors of the right shapes (torch, on ``device``)."""
    import torch

    ydt = torch.float32 if out_dtype == MK_OUT_F32 else torch.bfloat16
    return dict(
        y_sorted=torch.empty((T * k, F), dtype=ydt, device=device),
        src_index=torch.empty(T * k, dtype=torch.int32, device=device),
        expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=device),
        gate_w=torch.empty(T * k, dtype=torch.float32, device=device),
    )


def moe_dispatch_gemm(x, logits, W, k, cfg: mk_config_t | None = None, out=None, stream=None, workspace=None,
                      ws_bytes=0, check=True):
    """Run the path on torch tensors x[T,H] bf16, logits[T,E] f32, W[E,H,F] bf16 (device).

    Returns the dict of outputs (allocated when ``out`` is None).  With
    ``check`` the stream is synchronised and device errors are raised.
    """
    T, H = x.shape
    E, H2, F = W.shape
    if H2 != H or tuple(logits.shape) != (T, E):
        raise ValueError("shape mismatch between x, logits and W")
    if out is None:
        out = alloc_outputs(T, F, E, k, cfg.out_dtype if cfg is not None else MK_OUT_BF16, x.device)
    st = mk_moe_dispatch_gemm_ex(x, logits, T, H, E, k, W, F, out["y_sorted"], out["src_index"],
                                 out["expert_offsets"], out["gate_w"], stream, cfg, workspace, ws_bytes)
    _check(st, "mk_moe_dispatch_gemm_ex")
    if check:
        _check(mk_get_status(stream), "device status")
    return out


# ------------------------------------------- operators of a decode step --

def mk_add_rmsnorm(x, x_stride, residual, residual_stride, weight, T, H, eps, out, out8, scale, residual_out,
                   stream=None) -> int:
    return int(lib().mk_add_rmsnorm(_ptr(x), x_stride, _ptr(residual), residual_stride, _ptr(weight), T, H, eps,
                                    _ptr(out), _ptr(out8), _ptr(scale), _ptr(residual_out), _stream(stream)))


# The tensor forms below are called once per layer and token, so they do
# little: checks without temporaries, the raw stream handle, one allocation
# per output, and the C entry.  ``check`` waits for the stream and looks at the
# device's error word, as in the forms above: leave it out in a decode loop and
# under stream capture.  On the host of a GB300 (us): torch.cuda.
# current_stream 2.9, the raw handle 0.1; torch.empty 1.5, the allocator's own
# entry 0.8.

_torch = None
_raw_stream = None  # device index -> cudaStream_t of its current stream
_device = None      # () -> index of the current device, the one the C entries launch on
_empty = None       # (shape, strides, dtype, current device's index) -> uninitialised CUDA tensor


def _allocates(entry):
    """Whether the allocator's own entry, which torch does not document, does what it is used for."""
    import torch

    try:
        t = entry((3, 5), (5, 1), torch.bfloat16)
        return (type(t) is torch.Tensor and t.shape == (3, 5) and t.stride() == (5, 1) and t.dtype is torch.bfloat16
                and t.get_device() == torch.cuda.current_device())
    except Exception:  # missing, or another signature
        return False


def _load_torch():
    global _torch, _raw_stream, _device, _empty
    import torch

    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    guards = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
    direct = getattr(guards, "_empty_strided_cuda", None)  # on the current device
    if not _allocates(direct):
        direct = None

    def empty(shape, strides, dtype, device):
        if direct is not None:
            return direct(shape, strides, dtype)
        return torch.empty_strided(shape, strides, dtype=dtype, device=torch.device("cuda", device))

    _empty = empty
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch
    return torch


def _on_device(dev):
    if dev != _device():
        raise ValueError(f"the tensors are on device {dev}, the current one is {_device()}")


def _other_stream(stream, device):
    """A stream that the caller names, as a torch stream; None when it is the
    current one."""
    handle = _stream(stream)
    if handle == _raw_stream(device):
        return None
    if isinstance(stream, _torch.cuda.Stream):
        return stream
    return _torch.cuda.ExternalStream(handle, device) if handle else _torch.cuda.default_stream(device)


def _empty_on(stream):
    """_empty from a stream's own memory: what the current stream's pool gives
    out may have earlier work of that stream pending on it."""
    def empty(*args):
        with _torch.cuda.stream(stream):
            return _empty(*args)

    return empty


def _finish(status, what, stream, other, check, taken, made):
    """Errors of a call.  When it ran on another stream than the current one,
    the allocator is told who uses what: the other stream the caller's tensors
    (`taken`), the current one those that the call has made."""
    if other is not None:
        for t in taken:
            if hasattr(t, "record_stream"):
                t.record_stream(other)
        here = _torch.cuda.current_stream(other.device)
        for t in made:
            if t is not None:
                t.record_stream(here)
    if status != MK_OK:
        raise MkError(status, what)
    if check:
        _check(mk_get_status(stream), "device status")


def add_rmsnorm(x, weight, residual=None, eps=1e-6, bf16=True, e4m3=False, residual_out=None, stream=None, check=True):
    """Residual addition + RMS norm on torch tensors x[T,H] bf16 (rows may be
    strided), weight[H] bf16, residual[T,H] bf16.

    Returns a dict: ``out`` (bf16) unless ``bf16`` is false, ``out8``
    (float8_e4m3fn) and ``scale`` (one f32 per 128 columns) with ``e4m3``,
    and with a residual the new stream ``residual`` (in ``residual_out`` when
    given, which may be the residual itself).
    """
    torch = _torch or _load_torch()
    b16 = torch.bfloat16
    T, H = x.shape
    dev = x.get_device()
    if dev < 0 or x.dtype is not b16 or (x.stride(1) != 1 and H != 1):
        raise ValueError("x must be a CUDA bf16 [T,H] tensor with contiguous rows")
    _on_device(dev)
    if weight.dtype is not b16 or weight.get_device() != dev or weight.shape != (H,) or not weight.is_contiguous():
        raise ValueError("weight must be bf16 [H] on x's device")
    other = None if stream is None else _other_stream(stream, dev)
    empty, shape, strides = _empty if other is None else _empty_on(other), (T, H), (H, 1)
    o = {}
    out = out8 = scale = new = p_out = p_out8 = p_scale = p_res = p_new = None
    if bf16:
        o["out"] = out = empty(shape, strides, b16, dev)
        p_out = out.data_ptr()
    if e4m3:
        groups = -(-H // 128)
        o["out8"] = out8 = empty(shape, strides, torch.float8_e4m3fn, dev)
        o["scale"] = scale = empty((T, groups), (groups, 1), torch.float32, dev)
        p_out8, p_scale = out8.data_ptr(), scale.data_ptr()
    elif not bf16:
        raise ValueError("no output asked for")
    r_stride = 0
    if residual is not None:
        if (residual.dtype is not b16 or residual.get_device() != dev or residual.shape != shape
                or (residual.stride(1) != 1 and H != 1)):
            raise ValueError("residual must be bf16 [T,H] with contiguous rows on x's device")
        if residual_out is None:
            residual_out = new = empty(shape, strides, b16, dev)
        elif (residual_out.dtype is not b16 or residual_out.get_device() != dev or residual_out.shape != shape
              or not residual_out.is_contiguous()):
            raise ValueError("residual_out must be contiguous bf16 [T,H] on x's device")
        o["residual"] = residual_out
        r_stride, p_res, p_new = residual.stride(0), residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    status = lib().mk_add_rmsnorm(x.data_ptr(), x.stride(0), p_res, r_stride, weight.data_ptr(), T, H, eps, p_out, p_out8,
                                  p_scale, p_new, _raw_stream(dev) if stream is None else _stream(stream))
    if status or check or other is not None:
        _finish(status, "mk_add_rmsnorm", stream, other, check,
                (x, weight, residual, None if new is residual_out else residual_out), (out, out8, scale, new))
    return o


def mk_paged_attention(q, q_stride, k_cache, v_cache, page_stride, token_stride, head_stride, block_table, seq_lens, B,
                       Hq, Hkv, D, page_size, max_pages, num_pages, scale, out, lse=None, stream=None, workspace=None,
                       ws_bytes: int = 0) -> int:
    return int(lib().mk_paged_attention(_ptr(q), q_stride, _ptr(k_cache), _ptr(v_cache), page_stride, token_stride,
                                        head_stride, _ptr(block_table), _ptr(seq_lens), B, Hq, Hkv, D, page_size,
                                        max_pages, num_pages, scale, _ptr(out), _ptr(lse), _stream(stream),
                                        _ptr(workspace), int(ws_bytes)))


def mk_paged_attention_workspace_size(B, Hq, Hkv) -> int:
    return int(lib().mk_paged_attention_workspace_size(B, Hq, Hkv))


def paged_attention(q, k_cache, v_cache, block_table, seq_lens, scale=None, stream=None, workspace=None, ws_bytes=0,
                    check=True):
    """Attention of one new token per sequence, on torch tensors: q[B,Hq,D]
    bf16, k_cache and v_cache [pages, page_size, Hkv, D] bf16 (views with equal
    strides, the last dimension contiguous), block_table[B,max_pages] i32,
    seq_lens[B] i32 (cached keys, the new token's among them).

    ``scale`` defaults to D ** -0.5.  Returns ``out`` [B,Hq,D] bf16 and
    ``lse`` [B,Hq] f32.
    """
    torch = _torch or _load_torch()
    b16, i32 = torch.bfloat16, torch.int32
    B, Hq, D = q.shape
    dev = q.get_device()
    if dev < 0 or q.dtype is not b16:
        raise ValueError("q must be a CUDA bf16 [B,Hq,D] tensor")
    _on_device(dev)
    q_stride, q_head, q_last = q.stride()
    if q_last != 1 or (q_head != D and Hq != 1):
        raise ValueError("the heads of a sequence's q must be contiguous")
    pages, page_size, Hkv, kd = shape = k_cache.shape
    page, token, head, last = strides = k_cache.stride()
    if (kd != D or last != 1 or k_cache.dtype is not b16 or v_cache.dtype is not b16 or k_cache.get_device() != dev
            or v_cache.get_device() != dev):
        raise ValueError("caches must be bf16 [pages, page_size, Hkv, D] on q's device, D contiguous")
    if v_cache.shape != shape or (v_cache.stride() != strides and any(
            n > 1 and a != b for n, a, b in zip(shape, strides, v_cache.stride()))):
        raise ValueError("k_cache and v_cache must agree in shape and strides")
    rows, max_pages = block_table.shape
    if rows != B or block_table.dtype is not i32 or block_table.get_device() != dev or not block_table.is_contiguous():
        raise ValueError("block_table must be i32 [B,max_pages]")
    if (seq_lens.shape != (B,) or seq_lens.dtype is not i32 or seq_lens.get_device() != dev
            or not seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be i32 [B]")
    other = None if stream is None else _other_stream(stream, dev)
    empty = _empty if other is None else _empty_on(other)
    out = empty((B, Hq, D), (Hq * D, D, 1), b16, dev)
    lse = empty((B, Hq), (Hq, 1), torch.float32, dev)
    status = lib().mk_paged_attention(
        q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), page, token, head, block_table.data_ptr(),
        seq_lens.data_ptr(), B, Hq, Hkv, D, page_size, max_pages, pages, D ** -0.5 if scale is None else scale,
        out.data_ptr(), lse.data_ptr(), _raw_stream(dev) if stream is None else _stream(stream), _ptr(workspace),
        ws_bytes)
    if status or check or other is not None:
        _finish(status, "mk_paged_attention", stream, other, check,
                (q, k_cache, v_cache, block_table, seq_lens, workspace), (out, lse))
    return {"out": out, "lse": lse}


def mk_moe_ffn_decode(x, x_scale, logits, T, H, E, k, W1, W3, W2, W1_scale, W3_scale, W2_scale, F, weights, out,
                      stream=None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_moe_ffn_decode(_ptr(x), _ptr(x_scale), _ptr(logits), T, H, E, k, _ptr(W1), _ptr(W3), _ptr(W2),
                                       _ptr(W1_scale), _ptr(W3_scale), _ptr(W2_scale), F, weights, _ptr(out),
                                       _stream(stream), _ptr(workspace), int(ws_bytes)))


def mk_moe_ffn_decode_workspace_size(T, H, F, E, k, weights=MK_WEIGHT_BF16) -> int:
    return int(lib().mk_moe_ffn_decode_workspace_size(T, H, F, E, k, weights))


def moe_ffn_decode(x, logits, W1, W3, W2, k, x_scale=None, W1_scale=None, W3_scale=None, W2_scale=None, stream=None,
                   workspace=None, ws_bytes=0, check=True):
    """The whole gated expert layer for a few tokens on torch tensors: x[T,H],
    logits[T,E] f32, W1 and W3 [E,H,F], W2 [E,F,H], all bf16, or all
    float8_e4m3fn with ``x_scale`` [T,H/128] (as add_rmsnorm gives it) and a
    weight scale per 128 x 128 block.  An expert whose logit is -inf is left
    out.  Returns ``out`` [T,H] bf16."""
    torch = _torch or _load_torch()
    T, H = x.shape
    E, _, F = W1.shape
    dev, dtype = x.get_device(), x.dtype
    fp8 = dtype is torch.float8_e4m3fn
    if dev < 0 or not (fp8 or dtype is torch.bfloat16):
        raise ValueError("x must be a CUDA bf16 or float8_e4m3fn [T,H] tensor")
    _on_device(dev)
    up = (E, H, F)
    if W1.shape != up or W3.shape != up or W2.shape != (E, F, H):
        raise ValueError("W1 and W3 must be [E,H,F] and W2 [E,F,H]")
    for t in (x, W1, W3, W2):
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            raise ValueError("x and the weights must be contiguous, of one type and on one device")
    scales = (x_scale, W1_scale, W3_scale, W2_scale)
    need = ((logits, (T, E)),)
    if fp8:
        h, f = H // 128, F // 128
        need = (need[0], (x_scale, (T, h)), (W1_scale, (E, h, f)), (W3_scale, (E, h, f)), (W2_scale, (E, f, h)))
    elif scales != (None, None, None, None):
        raise ValueError("scales belong to float8_e4m3fn weights")
    f32 = torch.float32
    for t, shape in need:
        if t is None or t.shape != shape or t.dtype is not f32 or t.get_device() != dev or not t.is_contiguous():
            raise ValueError("logits [T,E], x_scale [T,H/128] and the weights' scales (a value per 128 x 128 block) "
                             "must be contiguous f32 on x's device")
    other = None if stream is None else _other_stream(stream, dev)
    out = (_empty if other is None else _empty_on(other))((T, H), (H, 1), torch.bfloat16, dev)
    status = lib().mk_moe_ffn_decode(
        x.data_ptr(), x_scale.data_ptr() if fp8 else None, logits.data_ptr(), T, H, E, k, W1.data_ptr(), W3.data_ptr(),
        W2.data_ptr(), *([t.data_ptr() for t in scales[1:]] if fp8 else (None, None, None)), F,
        MK_WEIGHT_E4M3 if fp8 else MK_WEIGHT_BF16, out.data_ptr(),
        _raw_stream(dev) if stream is None else _stream(stream), _ptr(workspace), ws_bytes)
    if status or check or other is not None:
        _finish(status, "mk_moe_ffn_decode", stream, other, check, (x, logits, W1, W3, W2, *scales, workspace), (out,))
    return {"out": out}


# ------------------------------------- operators of a key-value cache --

def mk_qk_norm_rope(args: mk_qk_norm_rope_t, stream=None) -> int:
    return int(lib().mk_qk_norm_rope(ctypes.addressof(args) if args is not None else None, _stream(stream)))


def fp4_cache(pages, page_size, heads, D, device="cuda"):
    """Memory for a layer's keys and values in 4 bits: ``k_cache`` and
    ``v_cache`` [pages, page_size, heads, D/2] uint8, ``k_scales`` and
    ``v_scales`` [pages, page_size, heads, D/16] float8_e4m3fn, zeros.  A head's
    rows of a page lie side by side, so that one head's scales fill whole
    32-byte sectors of memory."""
    import torch

    def rows(cols, dtype):
        t = torch.zeros((2, pages, heads, page_size, cols), dtype=torch.uint8, device=device).view(dtype)
        return t.transpose(2, 3)

    values, scales = rows(D // 2, torch.uint8), rows(D // 16, torch.float8_e4m3fn)
    return dict(k_cache=values[0], v_cache=values[1], k_scales=scales[0], v_scales=scales[1])


def _cache_pair(k, v, dtype, cols, what):
    """Shape and strides that the two tensors of a cache share."""
    shape, strides = k.shape, k.stride()
    if k.dtype is not dtype or v.dtype is not dtype or k.get_device() != v.get_device() or len(shape) != 4:
        raise ValueError(f"{what} must be {dtype} [pages, page_size, Hkv, {cols}] on q's device")
    if v.shape != shape or (v.stride() != strides and any(
            n > 1 and a != b for n, a, b in zip(shape, strides, v.stride()))):
        raise ValueError(f"{what} must agree in shape and strides")
    if shape[3] != cols or (strides[3] != 1 and cols != 1):
        raise ValueError(f"{what} must have {cols} contiguous values a row")
    return shape, strides


def _fp4_cache_checks(dev, D, shape, k_scales, v_scales, Hkv, k_factor, v_factor):
    """Strides of the scales of a 4-bit cache."""
    torch = _torch
    s_shape, s_strides = _cache_pair(k_scales, v_scales, torch.float8_e4m3fn, D // 16, "k_scales and v_scales")
    if s_shape[:3] != shape[:3] or k_scales.get_device() != dev:
        raise ValueError("the scales must be [pages, page_size, Hkv, D/16] of the caches' pages")
    for f in (k_factor, v_factor):
        if f is not None and (f.dtype is not torch.float32 or f.get_device() != dev or f.shape != (Hkv,)
                              or not f.is_contiguous()):
            raise ValueError("k_factor and v_factor must be f32 [Hkv] on q's device")
    return s_strides


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, pair_axis=None,
                 v=None, slots=None, k_cache=None, v_cache=None, k_scales=None, v_scales=None, k_factor=None,
                 v_factor=None, keep=None, stream=None, check=True):
    """Norms of the heads of queries and keys, their rotation by position and
    the way of keys and values into a paged cache, on torch tensors: q[T,Hq,D],
    k[T,Hkv,D] bf16 (tokens and heads may be strided), positions [T] or
    [axes,T] i32, inv_freq [rot/2] f32 (the first ``rot`` columns of a head are
    rotated; ``interleaved``: neighbours as pairs, else i and i + rot/2).

    ``pair_axis``: a whole number per pair, the row of ``positions`` that turns
    it.  ``q_weight`` and ``k_weight`` [D] bf16; without one, no norm.

    With a cache: v[T,Hkv,D] bf16, slots[T] i64 (page * page_size + token in the
    page; negative: none), and ``k_cache``, ``v_cache`` [pages, page_size, Hkv,
    D] bf16, or [.., D/2] uint8 with ``k_scales``, ``v_scales`` [.., D/16]
    float8_e4m3fn (see ``fp4_cache``) and, if wanted, ``k_factor``, ``v_factor``
    [Hkv] f32.

    Returns ``q`` [T,Hq,D] bf16; without a cache, or with ``keep``, ``k`` too,
    and with ``keep`` and a 4-bit cache ``k`` and ``v`` as the cache holds them.
    """
    torch = _torch or _load_torch()
    b16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    T, Hq, D = q.shape
    dev = q.get_device()
    if dev < 0 or q.dtype is not b16:
        raise ValueError("q must be a CUDA bf16 [T,Hq,D] tensor")
    _on_device(dev)
    Hkv = k.shape[1] if k.dim() == 3 else 0
    heads = (T, Hkv, D)
    q_stride, q_head, q_last = q.stride()
    if k.dtype is not b16 or k.get_device() != dev or k.shape != heads:
        raise ValueError("q and k must be bf16 [T,heads,D] on one device")
    k_stride, k_head, k_last = k.stride()
    if q_last != 1 or k_last != 1:
        raise ValueError("the columns of a head must be contiguous")
    if inv_freq.dtype is not f32 or inv_freq.dim() != 1 or inv_freq.get_device() != dev or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be f32 [rot/2] on q's device")
    half = inv_freq.shape[0]
    axes, pos_stride = 1, 0
    if positions.dim() == 2:
        axes = positions.shape[0]
        pos_stride, last = positions.stride()
        good = positions.shape[1] == T and (last == 1 or T <= 1)
    else:
        good = positions.shape == (T,) and positions.is_contiguous()
    if not good or positions.dtype is not i32 or positions.get_device() != dev:
        raise ValueError("positions must be i32 [T] or [axes,T] on q's device, an axis contiguous")
    p_qw = p_kw = p_axis = p_v = p_slots = p_kc = p_vc = p_ks = p_vs = p_kf = p_vf = p_k = p_held = 0
    if q_weight is not None:
        if q_weight.dtype is not b16 or q_weight.get_device() != dev or q_weight.shape != (D,) or not q_weight.is_contiguous():
            raise ValueError("q_weight must be bf16 [D] on q's device")
        p_qw = q_weight.data_ptr()
    if k_weight is not None:
        if k_weight.dtype is not b16 or k_weight.get_device() != dev or k_weight.shape != (D,) or not k_weight.is_contiguous():
            raise ValueError("k_weight must be bf16 [D] on q's device")
        p_kw = k_weight.data_ptr()
    if pair_axis is not None:
        each = bytes(pair_axis) if not isinstance(pair_axis, int) else b""  # (ValueError for a number outside a byte)
        if len(each) != half or (half and max(each) >= axes):
            raise ValueError("pair_axis must name a row of positions for each of inv_freq")
        if half:
            each = (ctypes.c_uint8 * half).from_buffer_copy(each)
            p_axis = ctypes.addressof(each)
    elif axes > 1:
        raise ValueError("positions of several axes need pair_axis")
    cache, page_size, pages, v_stride, v_head = MK_CACHE_NONE, 0, 0, 0, 0
    page, token, head = s_page, s_token, s_head = 0, 0, 0
    if k_cache is None:
        if not (v is None and slots is None and v_cache is None and k_scales is None and v_scales is None
                and k_factor is None and v_factor is None):
            raise ValueError("v, slots, scales and factors belong to a cache")
        if keep is False:
            raise ValueError("without a cache the keys are an output")
        keep = True
    else:
        if v is None or slots is None or v_cache is None:
            raise ValueError("a cache needs v, slots, k_cache and v_cache")
        if v.dtype is not b16 or v.get_device() != dev or v.shape != heads:
            raise ValueError("v must be bf16 [T,Hkv,D] on q's device")
        v_stride, v_head, v_last = v.stride()
        if v_last != 1:
            raise ValueError("the columns of a head must be contiguous")
        if slots.dtype is not torch.int64 or slots.get_device() != dev or slots.shape != (T,) or not slots.is_contiguous():
            raise ValueError("slots must be i64 [T] on q's device")
        fp4 = k_cache.dtype is torch.uint8
        shape, (page, token, head, _) = _cache_pair(k_cache, v_cache, torch.uint8 if fp4 else b16, D // 2 if fp4 else D,
                                                    "k_cache and v_cache")
        pages, page_size, n, _ = shape
        if k_cache.get_device() != dev or n != Hkv:
            raise ValueError("k_cache and v_cache must be [pages, page_size, Hkv, columns] on q's device")
        if fp4:
            cache = MK_CACHE_FP4
            if k_scales is None or v_scales is None:
                raise ValueError("a 4-bit cache needs k_scales and v_scales")
            s_page, s_token, s_head, _ = _fp4_cache_checks(dev, D, shape, k_scales, v_scales, Hkv, k_factor, v_factor)
            p_ks, p_vs = k_scales.data_ptr(), v_scales.data_ptr()
            p_kf = 0 if k_factor is None else k_factor.data_ptr()
            p_vf = 0 if v_factor is None else v_factor.data_ptr()
        else:
            cache = MK_CACHE_BF16
            if not (k_scales is None and v_scales is None and k_factor is None and v_factor is None):
                raise ValueError("scales and factors belong to a 4-bit cache")
        p_v, p_slots, p_kc, p_vc = v.data_ptr(), slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr()
    other = None if stream is None else _other_stream(stream, dev)
    empty = _empty if other is None else _empty_on(other)
    out = empty((T, Hq, D), (Hq * D, D, 1), b16, dev)
    o = {"q": out}
    if keep:
        o["k"] = t = empty(heads, (Hkv * D, D, 1), b16, dev)
        p_k = t.data_ptr()
        if cache == MK_CACHE_FP4:
            o["v"] = t = empty(heads, (Hkv * D, D, 1), b16, dev)
            p_held = t.data_ptr()
    args = _rope_args.pack(
        q.data_ptr(), k.data_ptr(), p_v, q_stride, q_head, k_stride, k_head, v_stride, v_head, p_qw, p_kw,
        positions.data_ptr(), pos_stride, inv_freq.data_ptr(), p_axis, out.data_ptr(), p_k, p_held, p_slots, p_kc, p_vc, page,
        token, head, p_ks, p_vs, s_page, s_token, s_head, p_kf, p_vf, T, Hq, Hkv, D, 2 * half, axes,
        MK_PAIR_NEIGHBOURS if interleaved else MK_PAIR_HALVES, cache, page_size, pages, eps, 0)
    status = lib().mk_qk_norm_rope(args, _raw_stream(dev) if stream is None else _stream(stream))
    if status or check or other is not None:
        _finish(status, "mk_qk_norm_rope", stream, other, check,
                (q, k, v, positions, inv_freq, q_weight, k_weight, slots, k_cache, v_cache, k_scales, v_scales, k_factor,
                 v_factor), o.values())
    return o


def mk_paged_attention_fp4(q, q_stride, k_cache, v_cache, page_stride, token_stride, head_stride, k_scales, v_scales,
                           scale_page_stride, scale_token_stride, scale_head_stride, k_factor, v_factor, block_table,
                           seq_lens, B, Hq, Hkv, D, page_size, max_pages, num_pages, scale, out, lse=None, stream=None,
                           workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_paged_attention_fp4(
        _ptr(q), q_stride, _ptr(k_cache), _ptr(v_cache), page_stride, token_stride, head_stride, _ptr(k_scales),
        _ptr(v_scales), scale_page_stride, scale_token_stride, scale_head_stride, _ptr(k_factor), _ptr(v_factor),
        _ptr(block_table), _ptr(seq_lens), B, Hq, Hkv, D, page_size, max_pages, num_pages, scale, _ptr(out), _ptr(lse),
        _stream(stream), _ptr(workspace), int(ws_bytes)))


def mk_paged_attention_fp4_workspace_size(B, Hq, Hkv) -> int:
    return int(lib().mk_paged_attention_fp4_workspace_size(B, Hq, Hkv))


def paged_attention_fp4(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, scale=None, k_factor=None,
                        v_factor=None, stream=None, workspace=None, ws_bytes=0, check=True):
    """Attention of one new token per sequence over a 4-bit cache, on torch
    tensors: q[B,Hq,D] bf16, k_cache and v_cache [pages, page_size, Hkv, D/2]
    uint8, k_scales and v_scales [pages, page_size, Hkv, D/16] float8_e4m3fn (as
    ``fp4_cache`` makes them and ``qk_norm_rope`` fills them), k_factor and
    v_factor [Hkv] f32 or None, block_table[B,max_pages] i32, seq_lens[B] i32.

    ``scale`` defaults to D ** -0.5.  Returns ``out`` [B,Hq,D] bf16 and
    ``lse`` [B,Hq] f32.
    """
    torch = _torch or _load_torch()
    b16, i32 = torch.bfloat16, torch.int32
    B, Hq, D = q.shape
    dev = q.get_device()
    if dev < 0 or q.dtype is not b16:
        raise ValueError("q must be a CUDA bf16 [B,Hq,D] tensor")
    _on_device(dev)
    q_stride, q_head, q_last = q.stride()
    if q_last != 1 or (q_head != D and Hq != 1):
        raise ValueError("the heads of a sequence's q must be contiguous")
    shape, strides = _cache_pair(k_cache, v_cache, torch.uint8, D // 2, "k_cache and v_cache")
    pages, page_size, Hkv, _ = shape
    if k_cache.get_device() != dev:
        raise ValueError("k_cache and v_cache must be on q's device")
    s_strides = _fp4_cache_checks(dev, D, shape, k_scales, v_scales, Hkv, k_factor, v_factor)
    rows, max_pages = block_table.shape
    if rows != B or block_table.dtype is not i32 or block_table.get_device() != dev or not block_table.is_contiguous():
        raise ValueError("block_table must be i32 [B,max_pages]")
    if (seq_lens.shape != (B,) or seq_lens.dtype is not i32 or seq_lens.get_device() != dev
            or not seq_lens.is_contiguous()):
        raise ValueError("seq_lens must be i32 [B]")
    other = None if stream is None else _other_stream(stream, dev)
    empty = _empty if other is None else _empty_on(other)
    out = empty((B, Hq, D), (Hq * D, D, 1), b16, dev)
    lse = empty((B, Hq), (Hq, 1), torch.float32, dev)
    status = lib().mk_paged_attention_fp4(
        q.data_ptr(), q_stride, k_cache.data_ptr(), v_cache.data_ptr(), strides[0], strides[1], strides[2],
        k_scales.data_ptr(), v_scales.data_ptr(), s_strides[0], s_strides[1], s_strides[2],
        None if k_factor is None else k_factor.data_ptr(), None if v_factor is None else v_factor.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, D, page_size, max_pages, pages,
        D ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(),
        _raw_stream(dev) if stream is None else _stream(stream), _ptr(workspace), ws_bytes)
    if status or check or other is not None:
        _finish(status, "mk_paged_attention_fp4", stream, other, check,
                (q, k_cache, v_cache, k_scales, v_scales, k_factor, v_factor, block_table, seq_lens, workspace), (out, lse))
    return {"out": out, "lse": lse}


# Buffers in the C forms below: a list of (device pointer or tensor, bytes between pages, bytes of a page).

def _buffers(caches):
    n = len(caches)
    return ((ctypes.c_void_p * n)(*[_ptr(b[0]) for b in caches]), (ctypes.c_int64 * n)(*[b[1] for b in caches]),
            (ctypes.c_int64 * n)(*[b[2] for b in caches]), n)


def mk_copy_pages(caches, num_pages, src, dst, n, stream=None) -> int:
    return int(lib().mk_copy_pages(*_buffers(caches), num_pages, _ptr(src), _ptr(dst), n, _stream(stream)))


def mk_fork_sequences(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, parent, child, n, stream=None,
                      workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_fork_sequences(_ptr(block_table), _ptr(seq_lens), _ptr(refs), rows, max_pages, num_pages, page_size,
                                       _ptr(parent), _ptr(child), n, _stream(stream), _ptr(workspace), int(ws_bytes)))


def mk_free_sequences(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, seqs, n, stream=None) -> int:
    return int(lib().mk_free_sequences(_ptr(block_table), _ptr(seq_lens), _ptr(refs), rows, max_pages, num_pages, page_size,
                                       _ptr(seqs), n, _stream(stream)))


def mk_extend_sequences(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, seqs, count, n, most, slots,
                        caches, stream=None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_extend_sequences(_ptr(block_table), _ptr(seq_lens), _ptr(refs), rows, max_pages, num_pages,
                                         page_size, _ptr(seqs), _ptr(count), n, most, _ptr(slots), *_buffers(caches),
                                         _stream(stream), _ptr(workspace), int(ws_bytes)))


def mk_compact_pages(block_table, seq_lens, refs, rows, max_pages, num_pages, page_size, table_out, refs_out, caches,
                     stream=None, workspace=None, ws_bytes: int = 0) -> int:
    return int(lib().mk_compact_pages(_ptr(block_table), _ptr(seq_lens), _ptr(refs), rows, max_pages, num_pages, page_size,
                                      _ptr(table_out), _ptr(refs_out), *_buffers(caches), _stream(stream), _ptr(workspace),
                                      int(ws_bytes)))


def mk_pages_workspace_size(max_pages, num_pages, n) -> int:
    return int(lib().mk_pages_workspace_size(max_pages, num_pages, n))


_i64_arrays = {}  # C array types by length


def _page_buffers(caches, dev, pages=None):
    """The three C arrays of tensors whose first dimension is the page and whose
    pages are dense, in whatever order of the other dimensions: their addresses,
    their length, what holds them and the tensors, and the number of pages."""
    if isinstance(caches, _torch.Tensor):
        raise ValueError("caches are a list of tensors: one tensor's pages would be taken for caches")
    caches = tuple(caches)  # (once: it may be a generator)
    base, strides, sizes = [], [], []
    shape = stride = dtype = None
    for t in caches:
        if t.get_device() != dev:
            raise ValueError("the caches must be on one device")
        if t.shape != shape or t.stride() != stride or t.dtype is not dtype:  # a layer's is the one before's
            shape, stride, dtype = t.shape, t.stride(), t.dtype
            if len(shape) < 2:
                raise ValueError("a cache's first dimension is its pages")
            if pages is None:
                pages = shape[0]
            if shape[0] != pages:
                raise ValueError("the caches must have the same number of pages")
            if pages and t.is_contiguous():
                dense = t.numel() // pages
            else:
                dense = 1
                for s, n in sorted(zip(stride[1:], shape[1:])):
                    if n > 1 and s != dense:
                        raise ValueError("the values of a page must lie one after the other")
                    dense *= n
            size = t.element_size()
            block, step = dense * size, stride[0] * size
        base.append(t.data_ptr())
        strides.append(step)
        sizes.append(block)
    n = len(base)
    kind = _i64_arrays.get(n)
    if kind is None:
        kind = _i64_arrays[n] = ctypes.c_int64 * (3 * n)
    arrays = kind(*base, *strides, *sizes)
    at = ctypes.addressof(arrays)
    return at, at + 8 * n, at + 16 * n, n, (arrays, *caches), pages


def _i32_list(t, dev, n, what):
    if t.dtype is not _torch.int32 or t.get_device() != dev or not t.is_contiguous() or t.dim() != 1 or (
            n is not None and t.shape[0] != n):
        raise ValueError(f"{what} must be i32 on the table's device, one entry for each sequence of the list")
    return t.shape[0]


def _pool(block_table, seq_lens, refs, page_size):
    """Arguments of a pool that every entry takes."""
    torch = _torch or _load_torch()
    dev = block_table.get_device()
    if dev < 0 or block_table.dtype is not torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a CUDA i32 [rows,max_pages] tensor")
    _on_device(dev)
    rows, max_pages = block_table.shape
    for t, shape, what in ((seq_lens, (rows,), "seq_lens must be i32 [rows]"), (refs, None, "refs must be i32 [pages]")):
        if t.dtype is not torch.int32 or t.get_device() != dev or t.dim() != 1 or not t.is_contiguous() or (
                shape is not None and t.shape != shape):
            raise ValueError(what + " on the table's device")
    return dev, (block_table.data_ptr(), seq_lens.data_ptr(), refs.data_ptr(), rows, max_pages, refs.shape[0], page_size)


def copy_pages(caches, src, dst, stream=None, check=True):
    """Copies page ``src[i]`` to page ``dst[i]`` in each of ``caches``, tensors
    [pages, ...] whose pages are dense (a layer's keys or values, in bf16 or 4
    bits, or their scales); src and dst i32 on the caches' device.  The pages of
    dst differ, and none of them is in src."""
    torch = _torch or _load_torch()
    dev = src.get_device()
    if dev < 0 or src.dtype is not torch.int32:
        raise ValueError("src must be a CUDA i32 tensor")
    _on_device(dev)
    n = _i32_list(src, dev, None, "src")
    _i32_list(dst, dev, n, "dst")
    base, strides, sizes, number, held, pages = _page_buffers(caches, dev)
    other = None if stream is None else _other_stream(stream, dev)
    status = lib().mk_copy_pages(base, strides, sizes, number, pages or 0, src.data_ptr(), dst.data_ptr(), n,
                                 _raw_stream(dev) if stream is None else _stream(stream))
    if status or check or other is not None:
        _finish(status, "mk_copy_pages", stream, other, check, (src, dst, *held), ())


def fork_sequences(block_table, seq_lens, refs, parent, child, page_size, stream=None, workspace=None, ws_bytes=0, check=True):
    """Sequence ``child[i]`` gives its pages back and shares those of
    ``parent[i]`` (as before the call): block_table[rows,max_pages],
    seq_lens[rows], refs[pages], parent and child, all i32, change in place."""
    dev, pool = _pool(block_table, seq_lens, refs, page_size)
    n = _i32_list(child, dev, None, "child")
    _i32_list(parent, dev, n, "parent")
    other = None if stream is None else _other_stream(stream, dev)
    status = lib().mk_fork_sequences(*pool, parent.data_ptr(), child.data_ptr(), n,
                                     _raw_stream(dev) if stream is None else _stream(stream), _ptr(workspace), ws_bytes)
    if status or check or other is not None:
        _finish(status, "mk_fork_sequences", stream, other, check, (block_table, seq_lens, refs, parent, child, workspace), ())


def free_sequences(block_table, seq_lens, refs, seqs, page_size, stream=None, check=True):
    """The sequences ``seqs`` (i32) give their pages back; their lengths become 0."""
    dev, pool = _pool(block_table, seq_lens, refs, page_size)
    n = _i32_list(seqs, dev, None, "seqs")
    other = None if stream is None else _other_stream(stream, dev)
    status = lib().mk_free_sequences(*pool, seqs.data_ptr(), n, _raw_stream(dev) if stream is None else _stream(stream))
    if status or check or other is not None:
        _finish(status, "mk_free_sequences", stream, other, check, (block_table, seq_lens, refs, seqs), ())


def extend_sequences(block_table, seq_lens, refs, seqs, count, most, caches, page_size, stream=None, workspace=None,
                     ws_bytes=0, check=True):
    """Makes room for ``count[i]`` (at most ``most``) new tokens of sequence
    ``seqs[i]``: a last page that is not full and shared is copied in each of
    ``caches`` first, new pages are the lowest free ones.  Returns their places,
    i64 [len(seqs), most] (-1 behind the last), as ``qk_norm_rope`` takes them."""
    dev, pool = _pool(block_table, seq_lens, refs, page_size)
    n = _i32_list(seqs, dev, None, "seqs")
    _i32_list(count, dev, n, "count")
    base, strides, sizes, number, held, _ = _page_buffers(caches, dev, refs.shape[0])
    other = None if stream is None else _other_stream(stream, dev)
    slots = (_empty if other is None else _empty_on(other))((n, most), (most, 1), _torch.int64, dev)
    status = lib().mk_extend_sequences(*pool, seqs.data_ptr(), count.data_ptr(), n, most, slots.data_ptr(), base, strides,
                                       sizes, number, _raw_stream(dev) if stream is None else _stream(stream), _ptr(workspace),
                                       ws_bytes)
    if status or check or other is not None:
        _finish(status, "mk_extend_sequences", stream, other, check,
                (block_table, seq_lens, refs, seqs, count, workspace, *held), (slots,))
    return slots


def compact_pages(block_table, seq_lens, refs, caches, page_size, table_out=None, refs_out=None, stream=None, workspace=None,
                  ws_bytes=0, check=True):
    """Moves the pages in use to the front of each of ``caches``.  Returns
    ``block_table`` and ``refs`` as they are then, in ``table_out`` and
    ``refs_out`` when given (which may be block_table and refs themselves)."""
    dev, pool = _pool(block_table, seq_lens, refs, page_size)
    base, strides, sizes, number, held, _ = _page_buffers(caches, dev, refs.shape[0])
    other = None if stream is None else _other_stream(stream, dev)
    empty = _empty if other is None else _empty_on(other)
    made = []
    i32 = _torch.int32
    if table_out is None:
        made.append(table_out := empty((pool[3], pool[4]), (pool[4], 1), i32, dev))
    elif table_out.dtype is not i32 or table_out.get_device() != dev or table_out.shape != block_table.shape or not table_out.is_contiguous():
        raise ValueError("table_out must be like block_table")
    if refs_out is None:
        made.append(refs_out := empty((pool[5],), (1,), i32, dev))
    elif refs_out.dtype is not i32 or refs_out.get_device() != dev or refs_out.shape != refs.shape or not refs_out.is_contiguous():
        raise ValueError("refs_out must be like refs")
    status = lib().mk_compact_pages(*pool, table_out.data_ptr(), refs_out.data_ptr(), base, strides, sizes, number,
                                    _raw_stream(dev) if stream is None else _stream(stream), _ptr(workspace), ws_bytes)
    if status or check or other is not None:
        _finish(status, "mk_compact_pages", stream, other, check,
                (block_table, seq_lens, refs, table_out, refs_out, workspace, *held), made)
    return {"block_table": table_out, "refs": refs_out}
