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
