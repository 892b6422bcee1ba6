"""Python binding of the W4 C ABI (``include/w4.h``) for MI355X (gfx950).

Each function has the name of the C entry point it calls and only marshals
arguments: torch tensors supply device memory and the current HIP stream,
every step of the computation runs in the HIP library ``libw4.so``.  There is
no CPU or PyTorch fallback: if the library is not built, or a call returns a
non-zero status, the function raises.

With ``stream=`` a call runs on that stream, and results and workspaces that it
allocates come from that stream's memory; its inputs have to be ready there.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

import torch

__all__ = [
    "W4Error", "SYM", "ASYM", "MAX_FRACS", "lib", "library_path",
    "w4_quantize_blockwise", "w4_mse_clip_search", "w4_prepack", "w4_quantize_rows_e4m3",
    "w4a16_gemm", "w4a16_gemm_noalloc", "w4a8_gemm", "w4_gemm_workspace_bytes", "w4a8_gemm_workspace_bytes", "w4_status_string",
    "w4_last_error",
    "w4_abi_version", "w4_portable_save", "w4_portable_info_read", "w4_portable_load",
    "w4a16_gate_up", "w4a16_gate_up_workspace_bytes", "w4a8_gate_up", "w4a8_gate_up_workspace_bytes", "w4a8_gemm_e4m3", "ACT_SILU", "ACT_GELU_TANH",
    "w4_nf4_levels", "w4_nf4_quantize", "w4_nf4_gemv",
    "FRACS_PLAIN", "FRACS_11",
    "w4_kv_cache", "w4_kv_append", "w4_tree_attention", "w4_tree_attention_workspace_bytes", "w4_sample",
    "w4_kv_move", "w4_adjust_logits",
    "w4a16_linear", "w4a8_linear", "w4a8_linear_e4m3", "w4_route", "w4_route_workspace_bytes", "w4a16_moe", "w4a16_moe_workspace_bytes",
]

HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(HERE, "libw4.so")

SYM = 0
ASYM = 1
MAX_FRACS = 32
FRACS_PLAIN = (1.0,)
# 1.00 down to 0.50 in steps of 0.05 (gowda.ai "LLM fast inference", "MSE clipping")
FRACS_11 = (1.00, 0.95, 0.90, 0.85, 0.80, 0.75, 0.70, 0.65, 0.60, 0.55, 0.50)

_MODES = {"sym": SYM, "asym": ASYM, SYM: SYM, ASYM: ASYM}
ACT_SILU = 1
ACT_GELU_TANH = 2
_ACTS = {"silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH, ACT_SILU: ACT_SILU, ACT_GELU_TANH: ACT_GELU_TANH}


class W4Error(RuntimeError):
    """A W4 call returned a non-zero status."""

    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} failed with status {status}: {message}")
        self.status = status


class _PortableInfo(ctypes.Structure):
    """``w4_portable_info`` of ``include/w4.h``."""
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("G", ctypes.c_int32), ("mode", ctypes.c_int32),
                ("n_fracs", ctypes.c_int32), ("has_clip", ctypes.c_int32), ("payload_bytes", ctypes.c_uint64),
                ("fracs", ctypes.c_float * MAX_FRACS)]


class _KvCache(ctypes.Structure):
    """``w4_kv_cache`` of ``include/w4.h``."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("layers", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded ``libw4.so`` (raises if it was never built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"W4 HIP library not built: {library_path} is missing "
                           "(run __graft_entry__.build() or python w4_dequant_gemm_amd/build.py)")
    L = ctypes.CDLL(library_path)
    P, i64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.w4_quantize_blockwise.argtypes = [P, i64, i64, I, I, P, I, P, P, P, P, P]
    L.w4_mse_clip_search.argtypes = [P, i64, i64, I, I, P, I, P, P, P]
    L.w4_prepack.argtypes = [P, P, P, i64, i64, I, I, P, P, P]
    L.w4_quantize_rows_e4m3.argtypes = [P, i64, i64, P, P, P]
    sz_t = ctypes.c_size_t
    L.w4a16_gemm.argtypes = [P, i64, i64, P, P, i64, I, P, P, sz_t, P]
    L.w4a16_gemm_noalloc.argtypes = [P, i64, i64, P, P, i64, I, P, P]
    L.w4a16_gemm_noalloc.restype = I
    L.w4a8_gemm.argtypes = [P, i64, i64, P, P, i64, I, P, P, P, P, sz_t, P]
    L.w4_gemm_workspace_bytes.argtypes = [i64, i64, i64]
    L.w4_gemm_workspace_bytes.restype = sz_t
    L.w4a8_gemm_workspace_bytes.argtypes = [i64, i64, i64]
    L.w4a8_gemm_workspace_bytes.restype = sz_t
    L.w4a16_gate_up.argtypes = [P, i64, i64, P, P, P, P, i64, I, I, P, P, sz_t, P]
    L.w4a16_gate_up_workspace_bytes.argtypes = [i64, i64, i64]
    L.w4a16_gate_up_workspace_bytes.restype = sz_t
    L.w4a8_gate_up.argtypes = [P, i64, i64, P, P, P, P, i64, I, I, P, P, P, P, P, P, sz_t, P]
    L.w4a8_gate_up_workspace_bytes.argtypes = [i64, i64, i64]
    L.w4a8_gate_up_workspace_bytes.restype = sz_t
    L.w4a8_gemm_e4m3.argtypes = [P, P, i64, i64, P, P, i64, I, P, P, sz_t, P]
    L.w4a8_gemm_e4m3.restype = I
    L.w4a16_gate_up.restype = I
    L.w4_nf4_levels.argtypes = [P]
    L.w4_nf4_quantize.argtypes = [P, i64, i64, P, P, P, P]
    L.w4_nf4_gemv.argtypes = [P, i64, P, P, P, i64, P, P]
    for name in ("w4_nf4_levels", "w4_nf4_quantize", "w4_nf4_gemv"):
        getattr(L, name).restype = I
    L.w4a8_gate_up.restype = I
    cp = ctypes.c_char_p
    L.w4_portable_save.argtypes = [cp, i64, i64, I, I, P, I, P, P, P, P]
    L.w4_portable_info_read.argtypes = [cp, ctypes.POINTER(_PortableInfo)]
    L.w4_portable_load.argtypes = [cp, P, P, P, P]
    for name in ("w4_portable_save", "w4_portable_info_read", "w4_portable_load"):
        getattr(L, name).restype = I
    for name in ("w4_quantize_blockwise", "w4_mse_clip_search", "w4_prepack", "w4_quantize_rows_e4m3",
                 "w4a16_gemm", "w4a8_gemm"):
        getattr(L, name).restype = I
    f32, C = ctypes.c_float, ctypes.POINTER(_KvCache)
    L.w4_kv_append.argtypes = [P, i64, P, i64, P, i64, i64, I, C, P, P, i64, I, I, P, P, P, f32, P, P]
    L.w4_tree_attention.argtypes = [P, i64, i64, I, C, P, i64, P, P, i64, i64, i64, P, I, P, i64, f32, P, P, sz_t, P]
    L.w4_tree_attention_workspace_bytes.argtypes = [i64, i64, I, I, I, I, i64, i64, i64]
    L.w4_tree_attention_workspace_bytes.restype = sz_t
    L.w4_sample.argtypes = [P, I, i64, i64, i64, P, P, P, P, P, P, P, P]
    L.w4_kv_move.argtypes = [C, P, i64, P, P, i64, P, i64, P]
    L.w4_adjust_logits.argtypes = [P, I, i64, i64, i64, P, i64, P, P, P, P, P, P, P, P, i64, P, i64, P, i64, P]
    for name in ("w4_kv_append", "w4_tree_attention", "w4_sample", "w4_kv_move", "w4_adjust_logits"):
        getattr(L, name).restype = I
    L.w4a16_linear.argtypes = [P, i64, i64, P, P, i64, I, P, I, P, P, P, sz_t, P]
    L.w4a8_linear.argtypes = [P, i64, i64, P, P, i64, I, P, I, P, P, P, P, P, sz_t, P]
    L.w4a8_linear_e4m3.argtypes = [P, P, i64, i64, P, P, i64, I, P, I, P, P, P, sz_t, P]
    for name in ("w4a16_linear", "w4a8_linear", "w4a8_linear_e4m3"):
        getattr(L, name).restype = I
    L.w4_route.argtypes = [P, i64, i64, P, i64, I, I, P, I, f32, P, P, P, sz_t, P]
    L.w4_route_workspace_bytes.argtypes = [i64, i64, i64]
    L.w4_route_workspace_bytes.restype = sz_t
    L.w4a16_moe.argtypes = [P, i64, i64, P, P, I, P, P, P, P, P, P, i64, i64, I, I, P, P, P, sz_t, P]
    L.w4a16_moe_workspace_bytes.argtypes = [i64, I, i64, i64, i64, I]
    L.w4a16_moe_workspace_bytes.restype = sz_t
    for name in ("w4_route", "w4a16_moe"):
        getattr(L, name).restype = I
    L.w4_status_string.argtypes = [I]
    L.w4_status_string.restype = ctypes.c_char_p
    L.w4_last_error.argtypes = []
    L.w4_last_error.restype = ctypes.c_char_p
    L.w4_abi_version.argtypes = []
    L.w4_abi_version.restype = I
    _lib = L
    return L


_call_path = os.path.join(HERE, "_w4call.so")
_call = None


def _short():
    """The compiled way of the usual small calls (``csrc/pycall.cpp``), bound to the loaded library."""
    global _call
    if _call is None:
        import importlib.util
        if not os.path.exists(_call_path):
            raise RuntimeError(f"W4 binding not built: {_call_path} is missing "
                               "(run __graft_entry__.build() or python w4_dequant_gemm_amd/build.py)")
        spec = importlib.util.spec_from_file_location("_w4call", _call_path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        names = ("w4a16_linear", "w4a8_linear", "w4_gemm_workspace_bytes", "w4a8_gemm_workspace_bytes", "w4_route",
                 "w4_route_workspace_bytes", "w4a16_moe", "w4a16_moe_workspace_bytes", "w4_adjust_logits")
        module.bind(*(ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in names))
        _call = module
    return _call


def w4_status_string(status: int) -> str:
    return lib().w4_status_string(status).decode()


def w4_last_error() -> str:
    return lib().w4_last_error().decode()


def w4_abi_version() -> int:
    return int(lib().w4_abi_version())


# ------------------------------------------------------------------ helpers

def _check(fn: str, status: int):
    if status != 0:
        raise W4Error(fn, status, w4_last_error())


def _dev(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _ptr(fn: str, t: torch.Tensor, name: str, dtype, device: int):
    """Address of a contiguous tensor of ``dtype`` on GPU ``device`` (the checks of ``_dev`` in half their time: a
    mixture-of-experts call makes a dozen of them, as long as a launch takes)."""
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{fn}: {name} must be a device tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on cuda:{device} as the others are")
    raise ValueError(f"{fn}: {name} must be contiguous")


def _any_ptr(fn: str, t: Optional[torch.Tensor], name: str, device: int):
    """As ``_ptr`` for a workspace or codes of any one-byte type; None stays None."""
    return None if t is None else _ptr(fn, t, name, t.dtype, device)


def _vec_ptr(fn: str, t, name: str, n: int, dtype, device: int):
    if t is None:
        return None
    if t.numel() != n:
        raise ValueError(f"{fn}: {name} has {t.numel()} elements, expected {n}")
    return _ptr(fn, t, name, dtype, device)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _gpu(fn: str, t: torch.Tensor, name: str) -> int:
    """The index of the GPU that holds ``t``, which has to be the current one: the kernels run there."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{fn}: {name} must be a device tensor")
    if device != _current_device():
        raise ValueError(f"{fn}: {name} is on cuda:{device}, and the current device is cuda:{_current_device()}")
    return device


# the current stream's handle as an integer, without building a Stream object
# (about 2 us of host time per call otherwise, as much as a launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _stream(device, stream=None):
    if stream is None:
        if device.index is not None:
            return _raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    else:
        its = getattr(stream, "device", device).index      # (anything with a handle may be a stream)
        if device.index is not None and its is not None and its != device.index:
            raise ValueError(f"the stream is one of cuda:{its}, and the tensors are on {device}")
    return stream.cuda_stream


def _fracs(fracs: Sequence[float]):
    arr = (ctypes.c_float * len(fracs))(*[float(f) for f in fracs])
    return arr, len(fracs)


def _scratch(nbytes: int, device, stream):
    """Memory that only a call on ``stream`` uses.  It comes from that stream's own pool: what was freed on the
    current stream may still be in use there."""
    if stream is None:
        return torch.empty((nbytes,), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty((nbytes,), dtype=torch.uint8, device=device)


def _empty(shape, dtype, device, stream=None):
    """Memory for a result of a call on ``stream``: from that stream's own pool (as ``_scratch``), and not handed
    out again before what the current stream does with it is through."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _check_product_shapes(fn: str, X, wq, sz, G: int, Y=None, xq=None, xscale=None, up=None):
    """Shape checks the C ABI cannot make (it sees only pointers): the GPU
    layout of an [N, K] weight is N*K/2 bytes of codes and 4*N*K/G bytes of
    scale/zero words; outputs and W4A8 buffers must match [M, N] and [M, K].
    Raises ValueError before anything is launched."""
    if X.dim() != 2:
        raise ValueError(f"{fn}: X must be 2-D [M, K], got shape {tuple(X.shape)}")
    M, K = X.shape
    if wq.dim() != 2:
        raise ValueError(f"{fn}: wq must be 2-D [N, K/8], got shape {tuple(wq.shape)}")
    N = wq.shape[0]
    if G <= 0 or K % G != 0 or K % 8 != 0:
        raise ValueError(f"{fn}: K = {K} must be a multiple of 8 and of the group size G = {G}")
    if _nbytes(wq) != N * K // 2:
        raise ValueError(f"{fn}: wq holds {_nbytes(wq)} bytes; an [{N}, {K}] weight needs N*K/2 = {N * K // 2} "
                         f"(K of X does not match the weight?)")
    if _nbytes(sz) != 4 * N * (K // G):
        raise ValueError(f"{fn}: sz holds {_nbytes(sz)} bytes; an [{N}, {K}] weight with G = {G} needs "
                         f"{4 * N * (K // G)}")
    if Y is not None and tuple(Y.shape) != (M, N):
        raise ValueError(f"{fn}: output has shape {tuple(Y.shape)}, expected ({M}, {N})")
    if xq is not None and (tuple(xq.shape) != (M, K) or xq.element_size() != 1):
        raise ValueError(f"{fn}: xq must be one byte per element with shape ({M}, {K}), got "
                         f"{tuple(xq.shape)} of {xq.dtype}")
    if xscale is not None and xscale.numel() != M:
        raise ValueError(f"{fn}: xscale has {xscale.numel()} elements, expected {M}")
    if up is not None:
        if tuple(up["wq"].shape) != tuple(wq.shape) or _nbytes(up["wq"]) != _nbytes(wq):
            raise ValueError(f"{fn}: the up weight's wq {tuple(up['wq'].shape)} differs from the gate's "
                             f"{tuple(wq.shape)}")
        if _nbytes(up["sz"]) != _nbytes(sz):
            raise ValueError(f"{fn}: the up weight's sz differs in size from the gate's")
    return M, K, N


@functools.lru_cache(maxsize=4096)
def _need_bytes(M: int, K: int, N: int, w4a8: bool) -> int:
    # a function of the shape only
    return w4a8_gemm_workspace_bytes(M, K, N) if w4a8 else w4_gemm_workspace_bytes(M, K, N)


def _workspace(M: int, K: int, N: int, device, workspace, stream, w4a8=False):
    """(pointer, bytes) of the product's workspace: the caller's tensor, or a
    new byte tensor of the fastest schedule's size when the shape uses one
    (of ``stream``'s own memory)."""
    need = _need_bytes(M, K, N, w4a8)
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = _scratch(need, device, stream)
    return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- quantizer

def w4_quantize_blockwise(W: torch.Tensor, G: int, mode, fracs: Sequence[float] = FRACS_PLAIN, *,
                          packed=None, scale=None, zero=None, clip_idx=None, want_clip: bool = True,
                          stream=None) -> dict:
    """Quantize fp32 ``W[N, K]`` in groups of ``G`` (see ``w4.h``).

    Returns ``packed`` (uint8 [N, K/2], canonical nibbles), ``scale`` and
    ``zero`` (float16 [N, K/G]; zero is None for symmetric) and
    ``clip_idx`` (uint8 [N, K/G] or None).
    """
    m = _MODES[mode]
    N, K = W.shape
    dev = W.device
    ng = K // G if G else 0
    packed = _empty((N, K // 2), torch.uint8, dev, stream) if packed is None else packed
    scale = _empty((N, ng), torch.float16, dev, stream) if scale is None else scale
    if m == ASYM and zero is None:
        zero = _empty((N, ng), torch.float16, dev, stream)
    if m == SYM:
        zero = None
    if want_clip and clip_idx is None:
        clip_idx = _empty((N, ng), torch.uint8, dev, stream)
    fr, nf = _fracs(fracs)
    rc = lib().w4_quantize_blockwise(_dev(W, "W", torch.float32), N, K, G, m, fr, nf,
                                     _dev(packed, "packed"), _dev(scale, "scale"), _dev(zero, "zero"),
                                     _dev(clip_idx, "clip_idx"), _stream(dev, stream))
    _check("w4_quantize_blockwise", rc)
    return {"packed": packed, "scale": scale, "zero": zero, "clip_idx": clip_idx}


def w4_mse_clip_search(W: torch.Tensor, G: int, mode, fracs: Sequence[float], *, clip_idx=None,
                       sse=None, want_sse: bool = False, stream=None) -> dict:
    """Per-group index of the chosen clip fraction (and every candidate's error)."""
    m = _MODES[mode]
    N, K = W.shape
    dev = W.device
    ng = K // G if G else 0
    clip_idx = _empty((N, ng), torch.uint8, dev, stream) if clip_idx is None else clip_idx
    if want_sse and sse is None:
        sse = _empty((N, ng, len(fracs)), torch.float32, dev, stream)
    fr, nf = _fracs(fracs)
    rc = lib().w4_mse_clip_search(_dev(W, "W", torch.float32), N, K, G, m, fr, nf,
                                  _dev(clip_idx, "clip_idx"), _dev(sse, "sse"), _stream(dev, stream))
    _check("w4_mse_clip_search", rc)
    return {"clip_idx": clip_idx, "sse": sse}


def w4_prepack(packed: torch.Tensor, scale: torch.Tensor, zero: Optional[torch.Tensor], G: int, mode, *,
               wq=None, sz=None, stream=None) -> dict:
    """Portable packing -> GPU layout: ``wq`` (int32 [N, K/8]) and ``sz`` (int32 [N, K/G])."""
    m = _MODES[mode]
    N, K2 = packed.shape
    K = 2 * K2
    dev = packed.device
    wq = _empty((N, K // 8), torch.int32, dev, stream) if wq is None else wq
    sz = _empty((N, K // G if G else 0), torch.int32, dev, stream) if sz is None else sz
    rc = lib().w4_prepack(_dev(packed, "packed"), _dev(scale, "scale"), _dev(zero if m == ASYM else None, "zero"),
                          N, K, G, m, _dev(wq, "wq"), _dev(sz, "sz"), _stream(dev, stream))
    _check("w4_prepack", rc)
    return {"wq": wq, "sz": sz}


# ------------------------------------------------------ portable file form

def _host_bytes(t, name, dtype):
    """A C-contiguous host numpy view of tensor/array ``t`` with element type ``dtype``."""
    import numpy as np
    if t is None:
        return None
    if isinstance(t, torch.Tensor):
        t = t.detach()
        if t.dtype == torch.float16:
            t = t.view(torch.int16)
        t = t.cpu().numpy()
    a = np.ascontiguousarray(t)
    if a.dtype.itemsize != np.dtype(dtype).itemsize:
        raise ValueError(f"{name} must have {np.dtype(dtype).itemsize}-byte elements, got {a.dtype}")
    return a.view(dtype)


def _ptr_np(a):
    return None if a is None else ctypes.c_void_p(a.ctypes.data)


def w4_portable_save(path: str, packed, scale, zero, G: int, mode, fracs: Sequence[float] = FRACS_PLAIN,
                     clip_idx=None) -> None:
    """Writes the canonical arrays (device or host tensors, or numpy arrays) to ``path``."""
    import numpy as np
    m = _MODES[mode]
    pk = _host_bytes(packed, "packed", np.uint8)
    sc = _host_bytes(scale, "scale", np.uint16)
    ze = _host_bytes(zero, "zero", np.uint16) if m == ASYM else None
    ci = _host_bytes(clip_idx, "clip_idx", np.uint8)
    N, K2 = pk.shape
    arr, n = _fracs(fracs)
    rc = lib().w4_portable_save(os.fsencode(path), N, 2 * K2, G, m, arr, n, _ptr_np(pk), _ptr_np(sc), _ptr_np(ze),
                                _ptr_np(ci))
    _check("w4_portable_save", rc)


def w4_portable_info_read(path: str) -> dict:
    """Header of a portable file: N, K, G, mode, fracs, has_clip, payload_bytes."""
    info = _PortableInfo()
    _check("w4_portable_info_read", lib().w4_portable_info_read(os.fsencode(path), ctypes.byref(info)))
    return {"N": info.N, "K": info.K, "G": info.G, "mode": info.mode, "has_clip": bool(info.has_clip),
            "fracs": tuple(info.fracs[i] for i in range(info.n_fracs)), "payload_bytes": info.payload_bytes}


def w4_portable_load(path: str, device=None, *, prepack: bool = True, stream=None) -> dict:
    """Reads a portable file.  With ``device`` (a GPU) the canonical arrays are
    uploaded there and, with ``prepack``, rearranged into the GPU layout
    (``wq``, ``sz``) at once: the load-time prepack.  Without ``device`` the
    arrays stay in host memory (numpy)."""
    import numpy as np
    info = w4_portable_info_read(path)
    N, K, G = info["N"], info["K"], info["G"]
    asym = info["mode"] == ASYM
    packed = np.empty((N, K // 2), np.uint8)
    scale = np.empty((N, K // G), np.uint16)
    zero = np.empty((N, K // G), np.uint16) if asym else None
    clip = np.empty((N, K // G), np.uint8) if info["has_clip"] else None
    rc = lib().w4_portable_load(os.fsencode(path), _ptr_np(packed), _ptr_np(scale), _ptr_np(zero), _ptr_np(clip))
    _check("w4_portable_load", rc)
    out = dict(info)
    if device is None:
        out.update(packed=packed, scale=scale, zero=zero, clip_idx=clip)
        return out
    dev = torch.device(device)
    out["packed"] = torch.from_numpy(packed).to(dev)
    out["scale"] = torch.from_numpy(scale.view(np.float16)).to(dev)
    out["zero"] = torch.from_numpy(zero.view(np.float16)).to(dev) if asym else None
    out["clip_idx"] = torch.from_numpy(clip).to(dev) if clip is not None else None
    if prepack:
        out.update(w4_prepack(out["packed"], out["scale"], out["zero"], G, info["mode"], stream=stream))
    return out


# --------------------------------------------------------------- multiplies

def w4_quantize_rows_e4m3(X: torch.Tensor, *, xq=None, xscale=None, stream=None):
    """Per-row dynamic E4M3 of bf16 ``X[M, K]``: returns (xq uint8 [M, K], xscale fp32 [M])."""
    M, K = X.shape
    dev = X.device
    xq = _empty((M, K), torch.uint8, dev, stream) if xq is None else xq
    xscale = _empty((M,), torch.float32, dev, stream) if xscale is None else xscale
    rc = lib().w4_quantize_rows_e4m3(_dev(X, "X", torch.bfloat16), M, K, _dev(xq, "xq"),
                                     _dev(xscale, "xscale", torch.float32), _stream(dev, stream))
    _check("w4_quantize_rows_e4m3", rc)
    return xq, xscale


def w4_gemm_workspace_bytes(M: int, K: int, N: int) -> int:
    """Device workspace bytes a product of this shape needs (0 for most)."""
    return int(lib().w4_gemm_workspace_bytes(M, K, N))


def w4a8_gemm_workspace_bytes(M: int, K: int, N: int) -> int:
    """Workspace bytes for the fastest ``w4a8_gemm`` schedule (above 128 rows
    also the widened activations); at least ``w4_gemm_workspace_bytes``."""
    return int(lib().w4a8_gemm_workspace_bytes(M, K, N))


def w4a16_gemm(X: torch.Tensor, wq: torch.Tensor, sz: torch.Tensor, G: int, *, Y=None, workspace=None,
               stream=None):
    """``Y[M, N] = bf16(X . W'^T)`` from bf16 ``X[M, K]`` and the GPU-layout weights.

    ``workspace``: a device tensor of at least ``w4_gemm_workspace_bytes(M, K, N)``
    bytes; allocated here when omitted and the shape needs one."""
    M, K, N = _check_product_shapes("w4a16_gemm", X, wq, sz, G, Y=Y)
    dev = X.device
    Y = _empty((M, N), torch.bfloat16, dev, stream) if Y is None else Y
    ws, ws_bytes = _workspace(M, K, N, dev, workspace, stream)
    rc = lib().w4a16_gemm(_dev(X, "X", torch.bfloat16), M, K, _dev(wq, "wq"), _dev(sz, "sz"), N, G,
                          _dev(Y, "Y", torch.bfloat16), ws, ws_bytes, _stream(dev, stream))
    _check("w4a16_gemm", rc)
    return Y


def w4a16_gemm_noalloc(X: torch.Tensor, wq: torch.Tensor, sz: torch.Tensor, G: int, Y: torch.Tensor, *,
                       stream=None):
    """``w4a16_gemm`` into the caller's ``Y`` with the library's own scratch
    memory (no allocation by the library or here); calls that overlap on one
    GPU must not be issued together."""
    M, K, N = _check_product_shapes("w4a16_gemm_noalloc", X, wq, sz, G, Y=Y)
    dev = X.device
    rc = lib().w4a16_gemm_noalloc(_dev(X, "X", torch.bfloat16), M, K, _dev(wq, "wq"), _dev(sz, "sz"), N, G,
                                  _dev(Y, "Y", torch.bfloat16), _stream(dev, stream))
    _check("w4a16_gemm_noalloc", rc)
    return Y


def w4a8_gemm(X: torch.Tensor, wq: torch.Tensor, sz: torch.Tensor, G: int, *, Y=None, xq=None, xscale=None,
              workspace=None, stream=None):
    """W4A8: per-row E4M3 of ``X`` then ``Y = bf16(xscale * Xq . W'^T)``; returns (Y, xq, xscale)."""
    M, K, N = _check_product_shapes("w4a8_gemm", X, wq, sz, G, Y=Y, xq=xq, xscale=xscale)
    dev = X.device
    Y = _empty((M, N), torch.bfloat16, dev, stream) if Y is None else Y
    xq = _empty((M, K), torch.uint8, dev, stream) if xq is None else xq
    xscale = _empty((M,), torch.float32, dev, stream) if xscale is None else xscale
    ws, ws_bytes = _workspace(M, K, N, dev, workspace, stream, w4a8=True)
    rc = lib().w4a8_gemm(_dev(X, "X", torch.bfloat16), M, K, _dev(wq, "wq"), _dev(sz, "sz"), N, G,
                         _dev(Y, "Y", torch.bfloat16), _dev(xq, "xq"), _dev(xscale, "xscale", torch.float32),
                         ws, ws_bytes, _stream(dev, stream))
    _check("w4a8_gemm", rc)
    return Y, xq, xscale


# activations of the products with an epilogue (gate and up take the gated two)
_LINEAR_ACTS = {None: 0, "none": 0, "silu": ACT_SILU, "gelu_tanh": ACT_GELU_TANH, "relu": 3, "gelu": 4}


def _linear_shapes(fn: str, X, wq, sz, G: int, Y, xq=None, xscale=None):
    """(M, K, N), as ``_check_product_shapes``."""
    xs, ws = X.shape, wq.shape
    if len(xs) == 2 and len(ws) == 2 and G > 0 and Y is None and xq is None:
        (M, K), N = xs, ws[0]
        if K % G == 0 and K % 8 == 0 and wq.nbytes == N * K // 2 and sz.nbytes == 4 * N * (K // G) and (
                xscale is None or xscale.numel() == M):
            return M, K, N
    return _check_product_shapes(fn, X, wq, sz, G, Y=Y, xq=xq, xscale=xscale)


def _epilogue_args(fn: str, M: int, N: int, bias, act, residual, gpu: int):
    if act not in _LINEAR_ACTS:
        raise ValueError(f"{fn}: act must be None, 'none', 'silu', 'gelu_tanh', 'relu' or 'gelu', got {act!r}")
    if residual is None:
        r = None
    elif tuple(residual.shape) != (M, N):
        raise ValueError(f"{fn}: residual has shape {tuple(residual.shape)}, expected ({M}, {N})")
    else:
        r = _ptr(fn, residual, "residual", torch.bfloat16, gpu)
    return _vec_ptr(fn, bias, "bias", N, torch.float32, gpu), _LINEAR_ACTS[act], r


def w4a16_linear(X: torch.Tensor, wq: torch.Tensor, sz: torch.Tensor, G: int, *, bias=None, act=None, residual=None,
                 Y=None, workspace=None, stream=None):
    """``w4a16_gemm`` with its epilogue: ``Y[M, N] = bf16(act(X . W'^T + bias) + residual)``.  ``bias`` is fp32 [N],
    ``act`` None, ``"silu"``, ``"gelu_tanh"``, ``"gelu"`` (erf) or ``"relu"``, ``residual`` bf16 [M, N] (may be ``Y``)."""
    fn = "w4a16_linear"
    if Y is None and workspace is None and stream is None and act in _LINEAR_ACTS:
        gpu = X.get_device()
        if gpu >= 0 and gpu == _current_device():
            r = (_call or _short()).linear(gpu, _raw_stream(gpu), X, wq, sz, G, bias, _LINEAR_ACTS[act], residual, 0)
            if r is not None:
                return r
    M, K, N = _linear_shapes(fn, X, wq, sz, G, Y)
    dev = X.device
    b, a, r = _epilogue_args(fn, M, N, bias, act, residual, X.get_device())
    gpu = _gpu(fn, X, "X")
    _any_ptr(fn, workspace, "workspace", gpu)
    Y = _empty((M, N), torch.bfloat16, dev, stream) if Y is None else Y
    ws, ws_bytes = _workspace(M, K, N, dev, workspace, stream)
    rc = lib().w4a16_linear(_ptr(fn, X, "X", torch.bfloat16, gpu), M, K, _ptr(fn, wq, "wq", torch.int32, gpu),
                            _ptr(fn, sz, "sz", torch.int32, gpu), N, G, b, a, r, _ptr(fn, Y, "Y", torch.bfloat16, gpu),
                            ws, ws_bytes, _stream(dev, stream))
    if rc:
        _check(fn, rc)
    return Y


def w4a8_linear(X: torch.Tensor, wq: torch.Tensor, sz: torch.Tensor, G: int, *, bias=None, act=None, residual=None,
                Y=None, xq=None, xscale=None, workspace=None, stream=None):
    """``w4a8_gemm`` with the epilogue of ``w4a16_linear``; returns (Y, xq, xscale)."""
    fn = "w4a8_linear"
    if Y is None and xq is None and xscale is None and workspace is None and stream is None and act in _LINEAR_ACTS:
        gpu = X.get_device()
        if gpu >= 0 and gpu == _current_device():
            r = (_call or _short()).linear(gpu, _raw_stream(gpu), X, wq, sz, G, bias, _LINEAR_ACTS[act], residual, 1)
            if r is not None:
                return r
    M, K, N = _linear_shapes(fn, X, wq, sz, G, Y, xq, xscale)
    dev = X.device
    b, a, r = _epilogue_args(fn, M, N, bias, act, residual, X.get_device())
    gpu = _gpu(fn, X, "X")
    _any_ptr(fn, workspace, "workspace", gpu)
    Y = _empty((M, N), torch.bfloat16, dev, stream) if Y is None else Y
    xq = _empty((M, K), torch.uint8, dev, stream) if xq is None else xq
    xscale = _empty((M,), torch.float32, dev, stream) if xscale is None else xscale
    ws, ws_bytes = _workspace(M, K, N, dev, workspace, stream, w4a8=True)
    rc = lib().w4a8_linear(_ptr(fn, X, "X", torch.bfloat16, gpu), M, K, _ptr(fn, wq, "wq", torch.int32, gpu),
                           _ptr(fn, sz, "sz", torch.int32, gpu), N, G, b, a, r, _ptr(fn, Y, "Y", torch.bfloat16, gpu),
                           _any_ptr(fn, xq, "xq", gpu), _ptr(fn, xscale, "xscale", torch.float32, gpu), ws, ws_bytes,
                           _stream(dev, stream))
    if rc:
        _check(fn, rc)
    return Y, xq, xscale


def w4a8_linear_e4m3(xq: torch.Tensor, xscale: torch.Tensor, wq: torch.Tensor, sz: torch.Tensor, G: int, *, bias=None,
                     act=None, residual=None, Y=None, workspace=None, stream=None):
    """``w4a8_gemm_e4m3`` with the epilogue of ``w4a16_linear``: a down projection on ``w4a8_gate_up``'s E4M3 rows added
    to the residual stream, say."""
    fn = "w4a8_linear_e4m3"
    if xq.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise ValueError(f"{fn}: xq must hold E4M3 codes (torch.uint8 or torch.float8_e4m3fn), got {xq.dtype}")
    M, K, N = _linear_shapes(fn, xq, wq, sz, G, Y, None, xscale)
    dev = xq.device
    b, a, r = _epilogue_args(fn, M, N, bias, act, residual, xq.get_device())
    gpu = _gpu(fn, xq, "xq")
    _any_ptr(fn, workspace, "workspace", gpu)
    Y = _empty((M, N), torch.bfloat16, dev, stream) if Y is None else Y
    ws, ws_bytes = _workspace(M, K, N, dev, workspace, stream, w4a8=True)
    rc = lib().w4a8_linear_e4m3(_ptr(fn, xq, "xq", xq.dtype, gpu), _ptr(fn, xscale, "xscale", torch.float32, gpu), M, K,
                                _ptr(fn, wq, "wq", torch.int32, gpu), _ptr(fn, sz, "sz", torch.int32, gpu), N, G, b, a, r,
                                _ptr(fn, Y, "Y", torch.bfloat16, gpu), ws, ws_bytes, _stream(dev, stream))
    if rc:
        _check(fn, rc)
    return Y


def w4a16_gate_up_workspace_bytes(M: int, K: int, N: int) -> int:
    """Workspace bytes that let ``w4a16_gate_up`` split K in its last round (0: no split)."""
    return int(lib().w4a16_gate_up_workspace_bytes(M, K, N))


def w4a16_gate_up(X: torch.Tensor, gate: dict, up: dict, G: int, act="silu", *, H=None, workspace=None,
                  stream=None):
    """Gate and up projections in one pass: ``H = bf16(act(X . Wg'^T) * (X . Wu'^T))``
    for bf16 ``X[M, K]`` (above 32 rows K must be a multiple of 64); ``gate`` and ``up`` are GPU layouts from
    ``w4_prepack`` (``wq``, ``sz``); ``act`` is ``"silu"`` or ``"gelu_tanh"``.  ``workspace``: a device
    tensor (an empty one for none); by default one of ``w4a16_gate_up_workspace_bytes`` is allocated."""
    M, K, N = _check_product_shapes("w4a16_gate_up", X, gate["wq"], gate["sz"], G, Y=H, up=up)
    dev = X.device
    H = _empty((M, N), torch.bfloat16, dev, stream) if H is None else H
    if workspace is None:
        need = w4a16_gate_up_workspace_bytes(M, K, N)
        workspace = _scratch(need, dev, stream) if need else None
    ws = _dev(workspace, "workspace") if workspace is not None and workspace.numel() else None
    ws_bytes = _nbytes(workspace) if ws is not None else 0
    rc = lib().w4a16_gate_up(_dev(X, "X", torch.bfloat16), M, K, _dev(gate["wq"], "gate wq"), _dev(gate["sz"], "gate sz"),
                             _dev(up["wq"], "up wq"), _dev(up["sz"], "up sz"), N, G, _ACTS[act],
                             _dev(H, "H", torch.bfloat16), ws, ws_bytes, _stream(dev, stream))
    _check("w4a16_gate_up", rc)
    return H


def w4a8_gate_up_workspace_bytes(M: int, K: int, N: int) -> int:
    """Workspace bytes ``w4a8_gate_up`` needs to emit the E4M3 form of H."""
    return int(lib().w4a8_gate_up_workspace_bytes(M, K, N))


def w4a8_gate_up(X: torch.Tensor, gate: dict, up: dict, G: int, act="silu", *, H=None, xq=None, xscale=None,
                 emit_e4m3: bool = False, hq=None, hscale=None, workspace=None, stream=None):
    """W4A8 form of ``w4a16_gate_up``: per-row E4M3 of ``X`` first; returns (H, xq, xscale).

    With ``emit_e4m3`` (or ``hq`` given) the same pass also produces H's rows
    quantized to E4M3 for the down projection (``w4a8_gemm_e4m3``) and
    returns (H, xq, xscale, hq, hscale)."""
    M, K, N = _check_product_shapes("w4a8_gate_up", X, gate["wq"], gate["sz"], G, Y=H, xq=xq, xscale=xscale,
                                    up=up)
    dev = X.device
    emit = emit_e4m3 or hq is not None
    if emit:
        if hq is not None and (tuple(hq.shape) != (M, N) or hq.element_size() != 1):
            raise ValueError(f"w4a8_gate_up: hq must be one byte per element with shape ({M}, {N})")
        if hscale is not None and hscale.numel() != M:
            raise ValueError(f"w4a8_gate_up: hscale has {hscale.numel()} elements, expected {M}")
    H = _empty((M, N), torch.bfloat16, dev, stream) if H is None else H
    xq = _empty((M, K), torch.uint8, dev, stream) if xq is None else xq
    xscale = _empty((M,), torch.float32, dev, stream) if xscale is None else xscale
    ws, ws_bytes = None, 0
    if emit:
        hq = _empty((M, N), torch.uint8, dev, stream) if hq is None else hq
        hscale = _empty((M,), torch.float32, dev, stream) if hscale is None else hscale
        if workspace is None:
            workspace = _scratch(max(w4a8_gate_up_workspace_bytes(M, K, N), 16), dev, stream)
        ws, ws_bytes = _dev(workspace, "workspace"), _nbytes(workspace)
    rc = lib().w4a8_gate_up(_dev(X, "X", torch.bfloat16), M, K, _dev(gate["wq"], "gate wq"), _dev(gate["sz"], "gate sz"),
                            _dev(up["wq"], "up wq"), _dev(up["sz"], "up sz"), N, G, _ACTS[act],
                            _dev(H, "H", torch.bfloat16), _dev(xq, "xq"), _dev(xscale, "xscale", torch.float32),
                            _dev(hq, "hq") if emit else None, _dev(hscale, "hscale", torch.float32) if emit else None,
                            ws, ws_bytes, _stream(dev, stream))
    _check("w4a8_gate_up", rc)
    return (H, xq, xscale, hq, hscale) if emit else (H, xq, xscale)


def w4a8_gemm_e4m3(xq: torch.Tensor, xscale: torch.Tensor, wq: torch.Tensor, sz: torch.Tensor, G: int, *, Y=None,
                   workspace=None, stream=None):
    """W4A8 product on activations already quantized per row: ``Y = bf16(xscale * Xq . W'^T)``."""
    if xq.element_size() != 1:
        raise ValueError("w4a8_gemm_e4m3: xq must hold one byte per element")
    M, K, N = _check_product_shapes("w4a8_gemm_e4m3", xq, wq, sz, G, Y=Y, xscale=xscale)
    dev = xq.device
    Y = _empty((M, N), torch.bfloat16, dev, stream) if Y is None else Y
    ws, ws_bytes = _workspace(M, K, N, dev, workspace, stream, w4a8=True)
    rc = lib().w4a8_gemm_e4m3(_dev(xq, "xq"), _dev(xscale, "xscale", torch.float32), M, K, _dev(wq, "wq"),
                              _dev(sz, "sz"), N, G, _dev(Y, "Y", torch.bfloat16), ws, ws_bytes, _stream(dev, stream))
    _check("w4a8_gemm_e4m3", rc)
    return Y


# -------------------------------------------------- mixture of experts

_SCORES = {"softmax": 0, "sigmoid": 1}


@functools.lru_cache(maxsize=4096)
def w4_route_workspace_bytes(T: int, H: int, E: int) -> int:
    """Workspace bytes ``w4_route`` needs."""
    return int(lib().w4_route_workspace_bytes(T, H, E))


def w4_route(X: torch.Tensor, router: torch.Tensor, top_k: int, *, score="softmax", bias=None, renormalize: bool = True,
             scale: float = 1.0, ids=None, weights=None, workspace=None, stream=None):
    """Each token's ``top_k`` experts by the bf16 ``router`` [E, H] for bf16 ``X`` [T, H]: (ids int32 [T, top_k],
    weights fp32 [T, top_k]).  ``score`` is ``"softmax"`` or ``"sigmoid"``; ``bias`` (fp32 [E]) is added to the
    scores to choose but not to weigh."""
    fn = "w4_route"
    if ids is None and weights is None and workspace is None and stream is None and score in _SCORES:
        gpu = X.get_device()
        if gpu >= 0 and gpu == _current_device():
            r = (_call or _short()).route(gpu, _raw_stream(gpu), X, router, top_k, _SCORES[score], bias, renormalize, scale)
            if r is not None:
                return r
    xs, rs = X.shape, router.shape
    if len(xs) != 2 or len(rs) != 2 or xs[1] != rs[1]:
        raise ValueError(f"{fn}: X must be [T, H] and router [E, H], got {tuple(xs)} and {tuple(rs)}")
    if score not in _SCORES:
        raise ValueError(f"{fn}: score must be one of {sorted(_SCORES)}, got {score!r}")
    (T, H), E, dev = xs, rs[0], X.device
    b = _vec_ptr(fn, bias, "bias", E, torch.float32, X.get_device())
    gpu = _gpu(fn, X, "X")
    ids = _empty((T, top_k), torch.int32, dev, stream) if ids is None else ids
    weights = _empty((T, top_k), torch.float32, dev, stream) if weights is None else weights
    ws, ws_bytes = None, 0
    need = w4_route_workspace_bytes(T, H, E)
    if need:
        workspace = _scratch(need, dev, stream) if workspace is None else workspace
        ws, ws_bytes = _any_ptr(fn, workspace, "workspace", gpu), workspace.nbytes
    rc = lib().w4_route(_ptr(fn, X, "X", torch.bfloat16, gpu), T, H, _ptr(fn, router, "router", torch.bfloat16, gpu), E, top_k,
                        _SCORES[score], b, renormalize, scale, _vec_ptr(fn, ids, "ids", T * top_k, torch.int32, gpu),
                        _vec_ptr(fn, weights, "weights", T * top_k, torch.float32, gpu), ws, ws_bytes, _stream(dev, stream))
    if rc:
        _check(fn, rc)
    return ids, weights


@functools.lru_cache(maxsize=4096)
def w4a16_moe_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int, G: int) -> int:
    """Workspace bytes ``w4a16_moe`` needs."""
    return int(lib().w4a16_moe_workspace_bytes(T, top_k, E, H, I, G))


def _experts(fn: str, w: dict, name: str, E: int, N: int, K: int, G: int, gpu: int):
    """Addresses of E stacked GPU layouts of [N, K] weights."""
    wq, sz = w["wq"], w["sz"]
    if wq.nbytes != E * N * K // 2 or sz.nbytes != 4 * E * N * (K // G):
        raise ValueError(f"{fn}: {name} holds {wq.nbytes} bytes of codes and {sz.nbytes} of scales; {E} experts "
                         f"of [{N}, {K}] with G = {G} need {E * N * K // 2} and {4 * E * N * (K // G)}")
    return _ptr(fn, wq, name, torch.int32, gpu), _ptr(fn, sz, name, torch.int32, gpu)


def w4a16_moe(X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate: dict, up: dict, down: dict, G: int,
              act="silu", *, residual=None, Y=None, workspace=None, stream=None):
    """The experts' gated MLPs for bf16 ``X`` [T, H]: token t's choices are ``ids`` (int32 [T, top_k]; outside the
    experts: none) with ``weights`` (fp32).  ``gate``, ``up`` and ``down`` are GPU layouts of ``w4_prepack`` stacked
    over the experts (``wq`` [E, N, K/8], ``sz`` [E, N, K/G]).  Returns bf16 [T, H], ``residual`` (bf16 [T, H]) added."""
    fn = "w4a16_moe"
    if Y is None and workspace is None and stream is None and act in _ACTS:
        gpu = X.get_device()
        if gpu >= 0 and gpu == _current_device():
            r = (_call or _short()).moe(gpu, _raw_stream(gpu), X, ids, weights, gate["wq"], gate["sz"], up["wq"], up["sz"],
                                        down["wq"], down["sz"], G, _ACTS[act], residual)
            if r is not None:
                return r
    if act not in _ACTS:
        raise ValueError(f"{fn}: act must be 'silu' or 'gelu_tanh', got {act!r}")
    xs, js, gs = X.shape, ids.shape, gate["wq"].shape
    if len(xs) != 2 or len(js) != 2 or js[0] != xs[0] or weights.shape != js:
        raise ValueError(f"{fn}: X must be [T, H], ids and weights [T, top_k], got {tuple(xs)}, {tuple(js)} and "
                         f"{tuple(weights.shape)}")
    if len(gs) != 3:
        raise ValueError(f"{fn}: gate wq must be [E, I, H/8], got {tuple(gs)}")
    (T, H), top_k, (E, I, _), dev = xs, js[1], gs, X.device
    if G <= 0 or H % G or I % G:
        raise ValueError(f"{fn}: H = {H} and I = {I} must be multiples of the group size G = {G}")
    if (residual is not None and residual.shape != xs) or (Y is not None and Y.shape != xs):
        t, name = (residual, "residual") if residual is not None and residual.shape != xs else (Y, "Y")
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {(T, H)}")
    gpu = X.get_device()
    g, u, d = (_experts(fn, gate, "gate", E, I, H, G, gpu), _experts(fn, up, "up", E, I, H, G, gpu),
               _experts(fn, down, "down", E, H, I, G, gpu))
    _gpu(fn, X, "X")
    Y = _empty((T, H), torch.bfloat16, dev, stream) if Y is None else Y
    if workspace is None:
        workspace = _scratch(w4a16_moe_workspace_bytes(T, top_k, E, H, I, G), dev, stream)
    rc = lib().w4a16_moe(_ptr(fn, X, "X", torch.bfloat16, gpu), T, H, _ptr(fn, ids, "ids", torch.int32, gpu),
                         _ptr(fn, weights, "weights", torch.float32, gpu), top_k, g[0], g[1], u[0], u[1], d[0], d[1], E, I, G,
                         _ACTS[act], None if residual is None else _ptr(fn, residual, "residual", torch.bfloat16, gpu),
                         _ptr(fn, Y, "Y", torch.bfloat16, gpu), _any_ptr(fn, workspace, "workspace", gpu), workspace.nbytes,
                         _stream(dev, stream))
    if rc:
        _check(fn, rc)
    return Y


# -------------------------------------------------------- NF4 comparator

def w4_nf4_levels():
    """The 16 NF4 levels (float32, ascending) the library's kernels use."""
    import numpy as np
    out = np.empty(16, np.float32)
    _check("w4_nf4_levels", lib().w4_nf4_levels(_ptr_np(out)))
    return out


def w4_nf4_quantize(W: torch.Tensor, *, stream=None) -> dict:
    """NF4 of fp32 ``W[N, K]`` (K a multiple of 64): ``packed`` (uint8 [N, K/2]),
    ``absmax_q`` (uint8 [N*K/64]) and ``absmax_c2`` (float32 [ceil(N*K/64/256)])."""
    N, K = W.shape
    dev = W.device
    nb = N * (K // 64)
    packed = _empty((N, K // 2), torch.uint8, dev, stream)
    aq = _empty((nb,), torch.uint8, dev, stream)
    c2 = _empty(((nb + 255) // 256,), torch.float32, dev, stream)
    rc = lib().w4_nf4_quantize(_dev(W, "W", torch.float32), N, K, _dev(packed, "packed"), _dev(aq, "absmax_q"),
                               _dev(c2, "absmax_c2", torch.float32), _stream(dev, stream))
    _check("w4_nf4_quantize", rc)
    return {"packed": packed, "absmax_q": aq, "absmax_c2": c2}


def w4_nf4_gemv(x: torch.Tensor, nf4: dict, *, y=None, stream=None):
    """``y[N] = bf16(W' . x)`` for one bf16 row ``x[K]`` and NF4 weights from ``w4_nf4_quantize``."""
    K = x.numel()
    N = nf4["packed"].shape[0]
    dev = x.device
    y = _empty((N,), torch.bfloat16, dev, stream) if y is None else y
    rc = lib().w4_nf4_gemv(_dev(x, "x", torch.bfloat16), K, _dev(nf4["packed"], "packed"), _dev(nf4["absmax_q"], "absmax_q"),
                           _dev(nf4["absmax_c2"], "absmax_c2", torch.float32), N, _dev(y, "y", torch.bfloat16),
                           _stream(dev, stream))
    _check("w4_nf4_gemv", rc)
    return y


# ------------------------------------------- decoding around the products

def w4_kv_cache(pages: int, kv_heads: int, head_dim: int, page_size: int, *, e4m3: bool = False, layers=None,
                device="cuda"):
    """A zeroed paged cache ``(k, v)`` in the library's layout (``w4_kv_cache`` in ``w4.h``): bf16, or E4M3
    codes (uint8).  With ``layers`` the arrays hold that many layers; ``k[i]``, ``v[i]`` is one of them."""
    c = 16 if e4m3 else 8
    if page_size <= 0 or page_size % 16 or head_dim <= 0 or head_dim % c:
        raise ValueError(f"w4_kv_cache: page_size must be a multiple of 16 and head_dim of {c}, got {page_size} and {head_dim}")
    lead = (pages, kv_heads, page_size // 16)
    lead = lead if layers is None else (layers, *lead)
    dtype = torch.uint8 if e4m3 else torch.bfloat16
    return (torch.zeros((*lead, head_dim // c, 16, c), dtype=dtype, device=device),
            torch.zeros((*lead, 16 // c, head_dim, c), dtype=dtype, device=device))


@functools.lru_cache(maxsize=4096)
def _cache_geometry(fn: str, shape, sv, dtype, dtype_v, layers: bool):
    # a function of the arrays' shapes and types only: the tail of _KvCache
    n = len(shape)
    if n != 6 and not (layers and n == 7):
        raise ValueError(f"{fn}: k_cache must be [pages, kv_heads, page_size/16, head_dim/c, 16, c]"
                         f"{' or have the layers first' if layers else ''}, got {tuple(shape)}")
    pages, heads, blocks, chunks, rows, c = shape[-6:]
    one_byte = dtype.itemsize == 1
    if rows != 16 or c != (16 if one_byte else 8):
        raise ValueError(f"{fn}: k_cache of {dtype} must end in [head_dim/{16 if one_byte else 8}, 16, "
                         f"{16 if one_byte else 8}], got {tuple(shape)}")
    if dtype not in (torch.bfloat16, torch.uint8, torch.float8_e4m3fn):
        raise ValueError(f"{fn}: the cache must be torch.bfloat16 or hold E4M3 codes (torch.uint8 or torch.float8_e4m3fn), "
                         f"got {dtype}")
    if dtype_v != dtype or tuple(sv) != (*shape[:-3], 16 // c, chunks * c, c):
        raise ValueError(f"{fn}: v_cache {tuple(sv)} of {dtype_v} does not belong to k_cache {tuple(shape)} of {dtype}")
    return pages, shape[0] if n == 7 else 1, heads, chunks * c, 16 * blocks, 1 if one_byte else 0


def _cache_arg(fn: str, k, v, k_scale, v_scale, layers: bool = False):
    """The C description of a cache (k, v) of ``w4_kv_cache``'s shapes, and its (kv_heads, head_dim)."""
    geometry = _cache_geometry(fn, k.shape, v.shape, k.dtype, v.dtype, layers)
    heads = geometry[2]
    a = _KvCache(_dev(k, "k_cache"), _dev(v, "v_cache"), _vec(fn, k_scale, "k_scale", heads, torch.float32),
                 _vec(fn, v_scale, "v_scale", heads, torch.float32), *geometry)
    return a, heads, geometry[3]


def _rows_arg(fn: str, x, name: str, heads: int, dim: int, T=None):
    """Pointer and row stride of bf16 rows [T, heads, dim] whose heads are contiguous."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or (T is not None and shape[0] != T):
        raise ValueError(f"{fn}: {name} must be [{'T' if T is None else T}, {heads}, {dim}], got {tuple(shape)}")
    if x.dtype != torch.bfloat16:
        raise ValueError(f"{fn}: {name} must be torch.bfloat16, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{fn}: {name} must be a device tensor")
    st, sh, sd = x.stride()
    if (sd != 1 and dim > 1) or (sh != dim and heads > 1):
        raise ValueError(f"{fn}: the heads of a row of {name} must be contiguous (strides {x.stride()})")
    return x.data_ptr(), (st if shape[0] > 1 else heads * dim)   # (a single row's stride means nothing)


def _vec(fn: str, x, name: str, n: int, dtype):
    if x is None:
        return None
    if x.numel() != n:
        raise ValueError(f"{fn}: {name} has {x.numel()} elements, expected {n}")
    return _dev(x, name, dtype)


def w4_kv_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                 k_cache: torch.Tensor, v_cache: torch.Tensor, *, rope=None, positions=None, interleaved: bool = False,
                 q_norm=None, k_norm=None, eps: float = 1e-6, k_scale=None, v_scale=None, Q=None, stream=None):
    """Norm (optional) and rotate (optional) the query and key heads of ``q``, ``k`` [T, heads, D]; keys and the
    values ``v`` go to the cache slots ``slots`` (int32 [T], negative: not stored), the queries are returned
    (bf16 [T, Hq, D]; None without ``q``).  ``rope`` is fp32 [positions, rot]: rot/2 cosines, then the sines."""
    fn = "w4_kv_append"
    cache, hk, dim = _cache_arg(fn, k_cache, v_cache, k_scale, v_scale)
    T = k.shape[0]
    kp, ks = _rows_arg(fn, k, "k", hk, dim, T)
    vp, vs = _rows_arg(fn, v, "v", hk, dim, T)
    qp, qs, hq, Qp = None, 0, 0, None
    if q is not None:
        hq = q.shape[1] if q.dim() == 3 else 0
        qp, qs = _rows_arg(fn, q, "q", hq, dim, T)
        if Q is None:
            Q = _empty((T, hq, dim), torch.bfloat16, q.device, stream)
        elif tuple(Q.shape) != (T, hq, dim):
            raise ValueError(f"{fn}: Q has shape {tuple(Q.shape)}, expected {(T, hq, dim)}")
        Qp = _dev(Q, "Q", torch.bfloat16)
    rot = rows = 0
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError(f"{fn}: rope must be [positions, rot], got {tuple(rope.shape)}")
        rows, rot = rope.shape
    rc = lib().w4_kv_append(qp, qs, kp, ks, vp, vs, T, hq, cache, _vec(fn, slots, "slots", T, torch.int32),
                            _dev(rope, "rope", torch.float32), rows, rot, interleaved,
                            _vec(fn, positions, "positions", T, torch.int32), _vec(fn, q_norm, "q_norm", dim, torch.float32),
                            _vec(fn, k_norm, "k_norm", dim, torch.float32), eps, Qp, _stream(k.device, stream))
    _check(fn, rc)
    return Q


@functools.lru_cache(maxsize=4096)
def w4_tree_attention_workspace_bytes(T: int, B: int, Hq: int, kv_heads: int, head_dim: int, e4m3: bool, max_q: int,
                                      max_kv: int, window: int = 0) -> int:
    """Workspace bytes ``w4_tree_attention`` needs for these sizes (0: none)."""
    return int(lib().w4_tree_attention_workspace_bytes(T, B, Hq, kv_heads, head_dim, 1 if e4m3 else 0, max_q, max_kv, window))


def w4_tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                      kv_len: torch.Tensor, q_start: torch.Tensor, max_q: int, max_kv: int, *, tree=None,
                      positions=None, window: int = 0, scale: Optional[float] = None, k_scale=None, v_scale=None,
                      O=None, workspace=None, stream=None):
    """Attention of each sequence's last tokens, ``q`` [T, Hq, D], over its cached keys and values (the tokens'
    own among them).  Sequence b has rows q_start[b] .. q_start[b + 1] - 1 and kv_len[b] cached tokens on the
    pages page_table[b] (all int32); ``max_q`` and ``max_kv`` bound them from above.  ``tree``: int64
    [T, ceil(max_q / 64)] masks of the nodes each node sees; None: a chain.  ``window`` > 0 needs ``positions``
    (int32 [T]) with a tree.  Returns bf16 [T, Hq, D]."""
    fn = "w4_tree_attention"
    cache, hk, dim = _cache_arg(fn, k_cache, v_cache, k_scale, v_scale)
    T, Hq = (q.shape[0], q.shape[1]) if q.dim() == 3 else (0, 0)
    qp, qs = _rows_arg(fn, q, "q", Hq, dim)
    if page_table.dim() != 2:
        raise ValueError(f"{fn}: page_table must be [B, pages], got {tuple(page_table.shape)}")
    B, table_pages = page_table.shape
    words = 0
    if tree is not None:
        if tree.dim() != 2 or tree.shape[0] != T:
            raise ValueError(f"{fn}: tree must be [{T}, words], got {tuple(tree.shape)}")
        words = tree.shape[1]
    if O is None:
        O = _empty((T, Hq, dim), torch.bfloat16, q.device, stream)
    elif tuple(O.shape) != (T, Hq, dim):
        raise ValueError(f"{fn}: O has shape {tuple(O.shape)}, expected {(T, Hq, dim)}")
    if workspace is None:
        need = w4_tree_attention_workspace_bytes(T, B, Hq, hk, dim, cache.dtype == 1, max_q, max_kv, window)
        workspace = _scratch(need, q.device, stream) if need else None
    ws_bytes = _nbytes(workspace) if workspace is not None else 0
    rc = lib().w4_tree_attention(qp, qs, T, Hq, cache, _dev(page_table, "page_table", torch.int32), table_pages,
                                 _vec(fn, kv_len, "kv_len", B, torch.int32),
                                 _vec(fn, q_start, "q_start", B + 1, torch.int32), B, max_q, max_kv,
                                 _dev(tree, "tree", torch.int64), words,
                                 _vec(fn, positions, "positions", T, torch.int32), window,
                                 dim ** -0.5 if scale is None else scale, _dev(O, "O", torch.bfloat16),
                                 _dev(workspace, "workspace"), ws_bytes, _stream(q.device, stream))
    _check(fn, rc)
    return O


def w4_sample(logits: torch.Tensor, u: torch.Tensor, *, temperature=None, top_k=None, top_p=None, min_p=None,
              tokens=None, probs=None, stream=None):
    """One token per row of ``logits`` [B, V] (bf16 or fp32; rows may be strided) from the uniform numbers ``u``
    [B].  ``temperature``, ``top_p``, ``min_p`` (fp32 [B]) and ``top_k`` (int32 [B]) are per row or None.
    Returns (tokens int32 [B], probs fp32 [B])."""
    fn = "w4_sample"
    if logits.dim() != 2 or not logits.is_cuda or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"{fn}: logits must be a device tensor [B, V] with contiguous rows")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{fn}: logits must be torch.bfloat16 or torch.float32, got {logits.dtype}")
    B, V = logits.shape
    dev = logits.device
    tokens = _empty((B,), torch.int32, dev, stream) if tokens is None else tokens
    probs = _empty((B,), torch.float32, dev, stream) if probs is None else probs
    rc = lib().w4_sample(logits.data_ptr(), 1 if logits.dtype == torch.float32 else 0, B, V,
                         logits.stride(0) if B > 1 else V,
                         _vec(fn, u, "u", B, torch.float32), _vec(fn, temperature, "temperature", B, torch.float32),
                         _vec(fn, top_k, "top_k", B, torch.int32), _vec(fn, top_p, "top_p", B, torch.float32),
                         _vec(fn, min_p, "min_p", B, torch.float32), _vec(fn, tokens, "tokens", B, torch.int32),
                         _vec(fn, probs, "probs", B, torch.float32), _stream(dev, stream))
    _check(fn, rc)
    return tokens, probs


def _logits_arg(fn: str, x, name: str):
    """Pointer, type and row stride of logits [B, V] whose rows are contiguous."""
    if x.dim() != 2 or not x.is_cuda or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError(f"{fn}: {name} must be a device tensor [B, V] with contiguous rows")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{fn}: {name} must be torch.bfloat16 or torch.float32, got {x.dtype}")
    return x.data_ptr(), (1 if x.dtype == torch.float32 else 0), (x.stride(0) if x.shape[0] > 1 else x.shape[1])


def w4_adjust_logits(logits: torch.Tensor, *, history=None, history_start=None, prompt_len=None, repetition=None,
                     presence=None, frequency=None, bias_start=None, bias_ids=None, bias_values=None, mask=None,
                     out=None, stream=None):
    """Penalties for repeated tokens, biases and masks on ``logits`` [B, V] (bf16 or fp32; rows may be strided).
    Row b's earlier tokens are ``history`` (int32) [history_start[b] : history_start[b + 1]], the first
    ``prompt_len[b]`` of them its prompt, which only ``repetition`` counts; ``repetition``, ``presence`` and
    ``frequency`` are fp32 [B].  ``bias_ids`` (int32) and ``bias_values`` (fp32) are split by ``bias_start`` alike.
    ``mask``: int32 [B, ceil(V / 32)] or [1, ...] for all rows, a bit a token, 0 forbids it.  Returns ``out`` (new
    by default; ``out=logits`` works in place)."""
    fn = "w4_adjust_logits"
    if out is None and stream is None:
        gpu = logits.get_device()
        if gpu >= 0 and gpu == _current_device():
            r = (_call or _short()).adjust(gpu, _raw_stream(gpu), logits, history, history_start, prompt_len, repetition,
                                           presence, frequency, bias_start, bias_ids, bias_values, mask)
            if r is not None:
                return r
    xp, f32, xs = _logits_arg(fn, logits, "logits")
    (B, V), dev, gpu = logits.shape, logits.device, _gpu(fn, logits, "logits")
    if out is None:
        out = _empty((B, V), logits.dtype, dev, stream)
        op, os_ = out.data_ptr(), V
    else:
        if out.shape != logits.shape or out.dtype != logits.dtype:
            raise ValueError(f"{fn}: out must be {logits.dtype} of shape {(B, V)}, got {out.dtype} of {tuple(out.shape)}")
        op, _, os_ = _logits_arg(fn, out, "out")
        if out.get_device() != gpu:
            raise ValueError(f"{fn}: out is on {out.device}, not on cuda:{gpu} as the logits are")
    hp, nh, hs, bi, bv, bs, nb, mp, ms = None, 0, None, None, None, None, 0, None, 0
    if history is not None or history_start is not None:
        if history is None or history_start is None:
            raise ValueError(f"{fn}: history and history_start must both be given or both be None")
        nh, hp = history.numel(), _ptr(fn, history, "history", torch.int32, gpu)
        hs = _vec_ptr(fn, history_start, "history_start", B + 1, torch.int32, gpu)
    if bias_ids is not None or bias_start is not None or bias_values is not None:
        if bias_ids is None or bias_start is None or bias_values is None:
            raise ValueError(f"{fn}: bias_start, bias_ids and bias_values must all be given or all be None")
        nb, bi = bias_ids.numel(), _ptr(fn, bias_ids, "bias_ids", torch.int32, gpu)
        bv = _vec_ptr(fn, bias_values, "bias_values", nb, torch.float32, gpu)
        bs = _vec_ptr(fn, bias_start, "bias_start", B + 1, torch.int32, gpu)
    if mask is not None:
        words = -(-V // 32)
        if mask.dim() != 2 or mask.shape[1] != words or mask.shape[0] not in (1, B):
            raise ValueError(f"{fn}: mask must be [{B} or 1, {words}], got {tuple(mask.shape)}")
        mp, ms = _ptr(fn, mask, "mask", torch.int32, gpu), (words if mask.shape[0] > 1 else 0)
    f = torch.float32
    rc = lib().w4_adjust_logits(xp, f32, B, V, xs, hp, nh, hs, _vec_ptr(fn, prompt_len, "prompt_len", B, torch.int32, gpu),
                                _vec_ptr(fn, repetition, "repetition", B, f, gpu), _vec_ptr(fn, presence, "presence", B, f, gpu),
                                _vec_ptr(fn, frequency, "frequency", B, f, gpu), bs, bi, bv, nb, mp, ms, op, os_,
                                _stream(dev, stream))
    if rc:
        _check(fn, rc)
    return out


def w4_kv_move(k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor, base: torch.Tensor,
               path: torch.Tensor, count: torch.Tensor, *, stream=None) -> None:
    """Token base[b] + path[b, j] of sequence b moves to base[b] + j for j < count[b] (int32, path rows strictly
    ascending), in every layer of the cache ([layers, ...] or one layer)."""
    fn = "w4_kv_move"
    cache, _, _ = _cache_arg(fn, k_cache, v_cache, None, None, layers=True)
    if page_table.dim() != 2 or path.dim() != 2 or path.shape[0] != page_table.shape[0]:
        raise ValueError(f"{fn}: page_table must be [B, pages] and path [B, length], got {tuple(page_table.shape)} and "
                         f"{tuple(path.shape)}")
    B, table_pages = page_table.shape
    rc = lib().w4_kv_move(cache, _dev(page_table, "page_table", torch.int32), table_pages,
                          _vec(fn, base, "base", B, torch.int32), _dev(path, "path", torch.int32), path.shape[1],
                          _vec(fn, count, "count", B, torch.int32), B, _stream(k_cache.device, stream))
    _check(fn, rc)
