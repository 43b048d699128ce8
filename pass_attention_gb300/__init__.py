"""liboss: online-softmax row softmax, fused attention forward, split-KV
decode, the (m, l, O) merge, and a paged key-value cache with the attention
that fills and reads it, on one GB300 (sm_103a).

This module is the thin Python binding over the C ABI in ``include/oss.h``:
it checks tensor dtypes and devices, allocates outputs with PyTorch, passes
raw device pointers and the current CUDA stream to ``liboss.so`` and turns a
non-OK status into an exception. Every step of the computation runs in the
library's CUDA kernels; there is no CPU fallback, and a missing library is an
error.
"""

from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import Optional

import torch

__all__ = [
    "OssError",
    "library_path",
    "load",
    "softmax_rows",
    "softmax_rows_from_host",
    "softmax_rows_multipass",
    "softmax_rows_16bit",
    "softmax_rows_workspace_bytes",
    "attention_fwd",
    "attention_fwd_from_host",
    "attention_fwd_partial",
    "attention_fwd_workspace_bytes",
    "attention_decode_splitkv",
    "merge_partials",
    "decode_from_host",
    "attention_fwd_packed",
    "kv_cache_append",
    "attention_decode_paged",
    "kv_cache_evict",
    "attention_decode_shared",
    "kv_cache_append_fp8",
    "kv_cache_read_fp8",
    "attention_decode_paged_fp8",
    "check_device_error",
    "debug_inject_fault",
    "set_rescale_policy",
    "rescale_policy",
    "RESCALE_POLICIES",
    "abi_version",
    "EXPORTED_SYMBOLS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "liboss.so")

OS_OK = 0
STATUS_NAMES = {
    0: "OS_OK",
    1: "OS_ERR_INVALID_ARGUMENT",
    2: "OS_ERR_MISALIGNED",
    3: "OS_ERR_UNSUPPORTED",
    4: "OS_ERR_CUDA",
    5: "OS_ERR_TIMEOUT",
    6: "OS_ERR_BAD_INDEX",
}

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f32 = ctypes.c_float


# os_paged_cache of include/oss.h, packed: k_pages, v_pages, ld_page, ld_head,
# ld_slot, page_table, ld_table, kv_len, num_pages, heads, page_size, head_dim,
# dtype, batch, max_pages (its bytes take the place of a pointer to it; a
# ctypes.Structure costs a microsecond more per call)
_PAGED_CACHE = struct.Struct("@PPqqqPqPiiiiiii")
# os_paged_cache_fp8: the same, then k_scales, v_scales, ld_scale_page, ld_scale_head
_PAGED_CACHE_FP8 = struct.Struct("@PPqqqPqPiiiiiiiPPqq")

# name -> (restype, argtypes), the signatures of include/oss.h
_SIGNATURES = {
    "os_softmax_rows": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32, _vp]),
    "os_softmax_rows_16bit": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32, _i32, _vp]),
    "os_softmax_rows_ws": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32, _vp, _i64, _vp]),
    "os_softmax_rows_16bit_ws": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32, _i32, _vp,
                                        _i64, _vp]),
    "os_softmax_rows_workspace_bytes": (_i64, [_i64, _i64, _i32]),
    "os_softmax_rows_from_host": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _f32, _i64,
                                         _vp]),
    "os_softmax_rows_multipass": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _f32, _i32,
                                         _vp]),
    "os_attention_fwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32,
                                ctypes.c_int, _vp]),
    "os_attention_fwd_ws": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32,
                                   ctypes.c_int, _vp, _i64, _vp]),
    "os_attention_fwd_workspace_bytes": (_i64, [_i32, _i32, _i32, _i32, _i32, ctypes.c_int]),
    "os_attention_fwd_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                        _f32, ctypes.c_int, _vp]),
    "os_attention_fwd_partial": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32,
                                        ctypes.c_int, _vp, _vp, _vp, _i32, _i32, _vp]),
    "os_attention_decode_splitkv": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                           _f32, _vp, _vp, _vp, _vp]),
    "os_merge_partials": (_i32, [_vp, _vp, _vp, _i64, _i32, _i32, ctypes.c_int, _vp, _vp, _vp,
                                 _vp, _vp]),
    "os_attention_fwd_packed": (_i32, [_vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i32,
                                       _i64, _i64, _i32, _i32, _i32, _i32, _f32, ctypes.c_int, _vp,
                                       _i64, _vp]),
    "os_attention_fwd_packed_workspace_bytes": (_i64, [_i64, _i32, _i32]),
    "os_kv_cache_append": (_i32, [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "os_attention_decode_paged": (_i32, [_vp, _i64, _i64, _i32, _vp, _f32, _vp, _vp, _vp, _i64,
                                         _i64, _vp, _i64, _vp]),
    "os_attention_decode_paged_workspace_bytes": (_i64, [_i32, _vp, ctypes.c_int]),
    "os_kv_cache_evict": (_i32, [_vp, _vp, _i64, _i64, _vp, _i64, _i32, _i32, _i32, _vp, _vp,
                                 _vp, _vp]),
    "os_attention_decode_shared": (_i32, [_vp, _i64, _i64, _i32, _vp, _vp, _i64, _vp, _i32, _vp, _i32,
                                          _f32, _vp, _vp, _vp, _i64, _vp]),
    "os_attention_decode_shared_workspace_bytes": (_i64, [_i32, _vp, _i32, _i32]),
    "os_kv_cache_append_fp8": (_i32, [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "os_kv_cache_read_fp8": (_i32, [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp]),
    "os_attention_decode_paged_fp8": (_i32, [_vp, _i64, _i64, _i32, _vp, _f32, _vp, _vp, _vp, _i64, _vp]),
    "os_attention_decode_paged_fp8_workspace_bytes": (_i64, [_i32, _vp]),
    "os_check_device_error": (_i32, [_vp, ctypes.POINTER(_i32)]),
    "os_attention_set_rescale_policy": (_i32, [_i32]),
    "os_attention_rescale_policy": (_i32, []),
    "os_debug_inject_fault": (_i32, [_i32, _i32, _i64]),
    "os_status_string": (ctypes.c_char_p, [_i32]),
    "os_abi_version": (_i32, []),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)

_lib: Optional[ctypes.CDLL] = None


class OssError(RuntimeError):
    """A liboss call returned a non-OK status."""

    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__(f"{where}: {STATUS_NAMES.get(self.status, self.status)}")


def library_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load liboss.so (built by ``pass_attention_gb300.build_lib``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"liboss is not built ({_LIB_PATH} is missing); build it with "
                "`python -m pass_attention_gb300.build_lib`")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def abi_version() -> int:
    return int(load().os_abi_version())


def _check(status: int, where: str) -> None:
    if status != OS_OK:
        raise OssError(status, where)


def _stream_ptr(stream, device: torch.device) -> int:
    """The CUDA stream to enqueue on: ``stream``, else the current stream of
    the inputs' device. A stream of another device is refused."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (liboss has no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")


def _dense(t: torch.Tensor, name: str) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, the inputs on {device}")


def _out(t, name: str, dtype: torch.dtype, shape, device: torch.device) -> torch.Tensor:
    """A caller-supplied output: a dense CUDA tensor of exactly this dtype and
    shape on the inputs' device (the kernels write every element of it and
    nothing around it, so a short, strided, host or foreign-device buffer is
    refused before the library is called)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (liboss has no CPU path)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the inputs on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# Workspaces of the *_ws entry points, one per (device, stream, kind): calls
# on one stream run one after another and may share one; calls on other
# streams get their own. Each is zero-filled when made, and the calls leave
# what must start at zero at zero again.
_WORKSPACES: dict = {}


def _workspace(device: torch.device, stream_ptr: int, nbytes: int, kind: str = "attn") -> torch.Tensor:
    key = (device.index, stream_ptr, kind)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=device)
        _WORKSPACES[key] = ws
    return ws


# ---------------------------------------------------------------------------
# os_softmax_rows
# ---------------------------------------------------------------------------

def softmax_rows_workspace_bytes(rows: int, cols: int, dtype=torch.float32) -> int:
    """Workspace bytes os_softmax_rows_ws uses for such rows (0: none)."""
    code = 0 if dtype == torch.float32 else _DTYPE_CODES[dtype]
    n = int(load().os_softmax_rows_workspace_bytes(int(rows), int(cols), code))
    if n < 0:
        raise OssError(4, "os_softmax_rows_workspace_bytes")
    return n

def softmax_rows(x: torch.Tensor, scale: float = 1.0, y: Optional[torch.Tensor] = None,
                 m: Optional[torch.Tensor] = None, l: Optional[torch.Tensor] = None,
                 stream=None):
    """Row softmax of ``scale * x`` (fp32 [rows, cols], unit column stride).

    Returns ``(y, m, l)``; see ``os_softmax_rows`` in include/oss.h.
    """
    _need(x, "x", torch.float32, 2)
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    rows, cols = x.shape
    dev = x.device
    if y is None:
        y = torch.empty((rows, cols), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, 2)
    _same_device(dev, y=y)
    if y.stride(1) != 1 or tuple(y.shape) != (rows, cols):
        raise ValueError("y must be [rows, cols] with unit column stride")
    m = _out(torch.empty(rows, dtype=torch.float32, device=dev) if m is None else m,
             "m", torch.float32, (rows,), dev)
    l = _out(torch.empty(rows, dtype=torch.float32, device=dev) if l is None else l,
             "l", torch.float32, (rows,), dev)
    with torch.cuda.device(dev):
        sp = _stream_ptr(stream, dev)
        need = softmax_rows_workspace_bytes(rows, cols)
        ws = _workspace(dev, sp, need, "rows") if need > 0 else None
        st = load().os_softmax_rows_ws(x.data_ptr(), y.data_ptr(), m.data_ptr(), l.data_ptr(), rows,
                                       cols, x.stride(0), y.stride(0), float(scale), _ptr(ws),
                                       need if ws is not None else 0, sp)
    _check(st, "os_softmax_rows_ws")
    return y, m, l


_DTYPE_CODES = {torch.bfloat16: 1, torch.float16: 2}


def softmax_rows_16bit(x: torch.Tensor, scale: float = 1.0, y: Optional[torch.Tensor] = None,
                       m: Optional[torch.Tensor] = None, l: Optional[torch.Tensor] = None,
                       stream=None):
    """Row softmax of ``scale * x`` for bf16 or fp16 rows ([rows, cols], unit
    column stride); y has x's type, m and l are fp32. See
    ``os_softmax_rows_16bit``."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPE_CODES:
        raise TypeError("x must be a bfloat16 or float16 torch.Tensor")
    _need(x, "x", x.dtype, 2)
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    rows, cols = x.shape
    dev = x.device
    if y is None:
        y = torch.empty((rows, cols), dtype=x.dtype, device=dev)
    _need(y, "y", x.dtype, 2)
    _same_device(dev, y=y)
    if y.stride(1) != 1 or tuple(y.shape) != (rows, cols):
        raise ValueError("y must be [rows, cols] with unit column stride")
    m = _out(torch.empty(rows, dtype=torch.float32, device=dev) if m is None else m,
             "m", torch.float32, (rows,), dev)
    l = _out(torch.empty(rows, dtype=torch.float32, device=dev) if l is None else l,
             "l", torch.float32, (rows,), dev)
    with torch.cuda.device(dev):
        sp = _stream_ptr(stream, dev)
        need = softmax_rows_workspace_bytes(rows, cols, x.dtype)
        ws = _workspace(dev, sp, need, "rows") if need > 0 else None
        st = load().os_softmax_rows_16bit_ws(x.data_ptr(), y.data_ptr(), m.data_ptr(), l.data_ptr(),
                                             rows, cols, x.stride(0), y.stride(0), float(scale),
                                             _DTYPE_CODES[x.dtype], _ptr(ws),
                                             need if ws is not None else 0, sp)
    _check(st, "os_softmax_rows_16bit_ws")
    return y, m, l


def softmax_rows_multipass(x: torch.Tensor, passes: int, scale: float = 1.0,
                           y: Optional[torch.Tensor] = None, m: Optional[torch.Tensor] = None,
                           l: Optional[torch.Tensor] = None, stream=None):
    """The 2- or 3-pass comparator of softmax_rows (same outputs; x is read
    from HBM ``passes`` times). See ``os_softmax_rows_multipass``."""
    _need(x, "x", torch.float32, 2)
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    rows, cols = x.shape
    dev = x.device
    if y is None:
        y = torch.empty((rows, cols), dtype=torch.float32, device=dev)
    _need(y, "y", torch.float32, 2)
    _same_device(dev, y=y)
    if y.stride(1) != 1 or tuple(y.shape) != (rows, cols):
        raise ValueError("y must be [rows, cols] with unit column stride")
    m = _out(torch.empty(rows, dtype=torch.float32, device=dev) if m is None else m,
             "m", torch.float32, (rows,), dev)
    l = _out(torch.empty(rows, dtype=torch.float32, device=dev) if l is None else l,
             "l", torch.float32, (rows,), dev)
    with torch.cuda.device(dev):
        st = load().os_softmax_rows_multipass(x.data_ptr(), y.data_ptr(), m.data_ptr(),
                                              l.data_ptr(), rows, cols, x.stride(0), y.stride(0),
                                              float(scale), int(passes), _stream_ptr(stream, dev))
    _check(st, "os_softmax_rows_multipass")
    return y, m, l


def softmax_rows_from_host(x_host: torch.Tensor, scale: float = 1.0, out=None, device="cuda",
                           chunk_rows: Optional[int] = None, x_dev: Optional[torch.Tensor] = None,
                           y_dev: Optional[torch.Tensor] = None):
    """End-to-end call on host memory through os_softmax_rows_from_host: the
    library copies x to the GPU, runs the row softmax and copies y, m and l
    back into (pinned) host tensors, in blocks of ``chunk_rows`` rows (default:
    about 64 MiB of x a block) whose upload, kernel and download overlap.
    Returns host (y, m, l) once the stream has finished them. ``x_dev`` /
    ``y_dev`` are optional device buffers of x's shape to reuse across calls."""
    if not isinstance(x_host, torch.Tensor) or x_host.dim() != 2 or x_host.dtype != torch.float32 \
            or x_host.is_cuda:
        raise ValueError("x_host must be a 2-D float32 host tensor")
    _dense(x_host, "x_host")
    rows, cols = x_host.shape
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if out is None:
        out = (torch.empty((rows, cols), dtype=torch.float32, pin_memory=True),
               torch.empty(rows, dtype=torch.float32, pin_memory=True),
               torch.empty(rows, dtype=torch.float32, pin_memory=True))
    y_host, m_host, l_host = out
    for name, t, shape in (("y_host", y_host, (rows, cols)), ("m_host", m_host, (rows,)),
                           ("l_host", l_host, (rows,))):
        if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.float32 \
                or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a dense float32 host tensor of shape {shape}")
    x_dev = torch.empty((rows, cols), dtype=torch.float32, device=dev) if x_dev is None \
        else _out(x_dev, "x_dev", torch.float32, (rows, cols), dev)
    y_dev = torch.empty((rows, cols), dtype=torch.float32, device=dev) if y_dev is None \
        else _out(y_dev, "y_dev", torch.float32, (rows, cols), dev)
    m_dev = torch.empty(rows, dtype=torch.float32, device=dev)
    l_dev = torch.empty(rows, dtype=torch.float32, device=dev)
    if chunk_rows is not None and chunk_rows < 1:
        raise ValueError("chunk_rows must be at least 1")
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev)
        st = load().os_softmax_rows_from_host(
            x_host.data_ptr(), y_host.data_ptr(), m_host.data_ptr(), l_host.data_ptr(),
            x_dev.data_ptr(), y_dev.data_ptr(), m_dev.data_ptr(), l_dev.data_ptr(), rows, cols,
            ctypes.c_float(scale), 0 if chunk_rows is None else int(chunk_rows), stream.cuda_stream)
        _check(st, "os_softmax_rows_from_host")
        stream.synchronize()
    return out


# ---------------------------------------------------------------------------
# os_attention_fwd
# ---------------------------------------------------------------------------

def attention_fwd_workspace_bytes(B: int, H: int, Sq: int, Sk: int, D: int = 128,
                                  causal: bool = False) -> int:
    """Workspace bytes os_attention_fwd_ws uses for this shape on the current
    device (0: none)."""
    n = int(load().os_attention_fwd_workspace_bytes(B, H, Sq, Sk, D, int(bool(causal))))
    if n < 0:
        raise OssError(4, "os_attention_fwd_workspace_bytes")
    return n


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                  scale: Optional[float] = None, causal: bool = False,
                  o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  stream=None):
    """Fused attention forward on bf16 [B, H, S, D] tensors.

    Returns ``(o, lse)``; see ``os_attention_fwd`` in include/oss.h.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
        _dense(t, n)
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    if tuple(k.shape) != (B, H, Sk, D) or tuple(v.shape) != (B, H, Sk, D):
        raise ValueError("k and v must be [B, H, Sk, D] matching q")
    dev = q.device
    _same_device(dev, k=k, v=v)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    o = _out(torch.empty_like(q) if o is None else o, "o", torch.bfloat16, q.shape, dev)
    lse = _out(torch.empty((B, H, Sq), dtype=torch.float32, device=dev) if lse is None else lse,
               "lse", torch.float32, (B, H, Sq), dev)
    with torch.cuda.device(dev):
        sp = _stream_ptr(stream, dev)
        need = attention_fwd_workspace_bytes(B, H, Sq, Sk, D, causal)
        ws = _workspace(dev, sp, need, "attn") if need > 0 else None
        st = load().os_attention_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                        lse.data_ptr(), B, H, Sq, Sk, D, float(scale),
                                        int(bool(causal)), _ptr(ws), need if ws is not None else 0,
                                        sp)
    _check(st, "os_attention_fwd_ws")
    return o, lse


def attention_fwd_partial(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          part_m: torch.Tensor, part_l: torch.Tensor, part_o: torch.Tensor,
                          index: int, scale: Optional[float] = None, causal: bool = False,
                          stream=None):
    """Partial softmax states of q against one shard k, v (bf16 [B, H, S, D]).

    part_m, part_l: fp32 [B, H, Sq, S_shards]; part_o: fp32 [B, H, Sq,
    S_shards, D]; writes slot ``index``. See ``os_attention_fwd_partial``.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
        _dense(t, n)
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    if tuple(k.shape) != (B, H, Sk, D) or tuple(v.shape) != (B, H, Sk, D):
        raise ValueError("k and v must be [B, H, Sk, D] matching q")
    dev = q.device
    _same_device(dev, k=k, v=v)
    _need(part_m, "part_m", torch.float32, 4)
    stride = part_m.shape[-1]
    _out(part_m, "part_m", torch.float32, (B, H, Sq, stride), dev)
    _out(part_l, "part_l", torch.float32, (B, H, Sq, stride), dev)
    _out(part_o, "part_o", torch.float32, (B, H, Sq, stride, D), dev)
    if not 0 <= int(index) < stride:
        raise ValueError(f"index {index} outside the {stride} partial slots")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with torch.cuda.device(dev):
        st = load().os_attention_fwd_partial(q.data_ptr(), k.data_ptr(), v.data_ptr(), B, H, Sq,
                                             Sk, D, float(scale), int(bool(causal)),
                                             part_m.data_ptr(), part_l.data_ptr(),
                                             part_o.data_ptr(), stride, int(index),
                                             _stream_ptr(stream, dev))
    _check(st, "os_attention_fwd_partial")


def attention_fwd_from_host(q_host, k_host, v_host, scale=None, causal=False, out=None,
                            device="cuda"):
    """End-to-end call on host memory: copy q, k, v to the GPU, run
    os_attention_fwd, copy o and lse back. Returns host (o, lse)."""
    q, k, v = (t.to(device, non_blocking=True) for t in (q_host, k_host, v_host))
    o, lse = attention_fwd(q, k, v, scale, causal)
    if out is None:
        out = (torch.empty(o.shape, dtype=o.dtype, pin_memory=True),
               torch.empty(lse.shape, dtype=lse.dtype, pin_memory=True))
    out[0].copy_(o, non_blocking=True)
    out[1].copy_(lse, non_blocking=True)
    torch.cuda.current_stream().synchronize()
    return out


# ---------------------------------------------------------------------------
# os_attention_decode_splitkv / os_merge_partials
# ---------------------------------------------------------------------------

def attention_decode_splitkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                             kv_len: torch.Tensor, num_splits: int,
                             scale: Optional[float] = None, part_m=None, part_l=None,
                             part_o=None, stream=None):
    """Split-KV decode partials. q [B, H, D], k/v [B, H, Lmax, D] bf16,
    kv_len [B] int32 (device). Returns ``(part_m, part_l, part_o)``."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, 4)
    _need(v, "v", torch.bfloat16, 4)
    _need(kv_len, "kv_len", torch.int32, 1)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (kv_len, "kv_len")):
        _dense(t, n)
    B, H, D = q.shape
    Lmax = k.shape[2]
    if tuple(k.shape) != (B, H, Lmax, D) or tuple(v.shape) != (B, H, Lmax, D):
        raise ValueError("k and v must be [B, H, Lmax, D] matching q")
    if kv_len.numel() != B:
        raise ValueError("kv_len must have B entries")
    dev = q.device
    _same_device(dev, k=k, v=v, kv_len=kv_len)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    S = int(num_splits)
    if S < 1:
        raise ValueError("num_splits must be >= 1")
    part_m = _out(torch.empty((B, H, S), dtype=torch.float32, device=dev) if part_m is None
                  else part_m, "part_m", torch.float32, (B, H, S), dev)
    part_l = _out(torch.empty((B, H, S), dtype=torch.float32, device=dev) if part_l is None
                  else part_l, "part_l", torch.float32, (B, H, S), dev)
    part_o = _out(torch.empty((B, H, S, D), dtype=torch.float32, device=dev) if part_o is None
                  else part_o, "part_o", torch.float32, (B, H, S, D), dev)
    with torch.cuda.device(dev):
        st = load().os_attention_decode_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                kv_len.data_ptr(), B, H, Lmax, D, S, float(scale),
                                                part_m.data_ptr(), part_l.data_ptr(),
                                                part_o.data_ptr(), _stream_ptr(stream, dev))
    _check(st, "os_attention_decode_splitkv")
    return part_m, part_l, part_o


def merge_partials(part_m: torch.Tensor, part_l: torch.Tensor, part_o: torch.Tensor,
                   finalize: bool = True, o_out=None, m_out=None, l_out=None, lse_out=None,
                   stream=None):
    """Merge partials over their split axis. part_m/part_l [..., S],
    part_o [..., S, D] fp32. Returns ``(o, m, l, lse)`` with o bf16 [..., D]
    (finalize) or fp32 [..., D] (unnormalised, finalize=False)."""
    for t, n in ((part_m, "part_m"), (part_l, "part_l"), (part_o, "part_o")):
        if not t.is_cuda or t.dtype != torch.float32:
            raise TypeError(f"{n} must be a CUDA float32 tensor")
        _dense(t, n)
    lead = tuple(part_m.shape[:-1])
    S = part_m.shape[-1]
    D = part_o.shape[-1]
    if tuple(part_l.shape) != tuple(part_m.shape) or tuple(part_o.shape) != lead + (S, D):
        raise ValueError("partials must be [..., S] and [..., S, D]")
    groups = 1
    for n in lead:
        groups *= n
    dev = part_m.device
    _same_device(dev, part_l=part_l, part_o=part_o)
    o_dtype = torch.bfloat16 if finalize else torch.float32
    o_out = _out(torch.empty(lead + (D,), dtype=o_dtype, device=dev) if o_out is None else o_out,
                 "o_out", o_dtype, lead + (D,), dev)
    m_out = _out(torch.empty(lead, dtype=torch.float32, device=dev) if m_out is None else m_out,
                 "m_out", torch.float32, lead, dev)
    l_out = _out(torch.empty(lead, dtype=torch.float32, device=dev) if l_out is None else l_out,
                 "l_out", torch.float32, lead, dev)
    lse_out = _out(torch.empty(lead, dtype=torch.float32, device=dev) if lse_out is None
                   else lse_out, "lse_out", torch.float32, lead, dev)
    with torch.cuda.device(dev):
        st = load().os_merge_partials(part_m.data_ptr(), part_l.data_ptr(), part_o.data_ptr(),
                                      groups, S, D, int(bool(finalize)), o_out.data_ptr(),
                                      _ptr(m_out), _ptr(l_out), _ptr(lse_out),
                                      _stream_ptr(stream, dev))
    _check(st, "os_merge_partials")
    return o_out, m_out, l_out, lse_out


def decode_from_host(q_host, k_host, v_host, kv_len_host, num_splits, scale=None, out=None,
                     device="cuda"):
    """End-to-end split-KV decode on host memory: copy inputs to the GPU, run
    the decode partials and the merge, copy o and lse back."""
    q, k, v, kv = (t.to(device, non_blocking=True) for t in (q_host, k_host, v_host, kv_len_host))
    pm, pl, po = attention_decode_splitkv(q, k, v, kv, num_splits, scale)
    o, _, _, lse = merge_partials(pm, pl, po, finalize=True)
    if out is None:
        out = (torch.empty(o.shape, dtype=o.dtype, pin_memory=True),
               torch.empty(lse.shape, dtype=lse.dtype, pin_memory=True))
    out[0].copy_(o, non_blocking=True)
    out[1].copy_(lse, non_blocking=True)
    torch.cuda.current_stream().synchronize()
    return out


# ---------------------------------------------------------------------------
# the paged key-value cache and packed prompts
# ---------------------------------------------------------------------------

# These calls are made once per layer and token, where the host's time counts:
# each tensor is checked in one expression, and what is wrong with it is found
# out only when that fails.

def _refuse(t, name: str, ndim: int, dtype: torch.dtype, device: torch.device) -> None:
    """Raises what is wrong with a tensor that a quick check refused."""
    _need(t, name, dtype, ndim)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the inputs on {device}")
    raise ValueError(f"{name} must have unit stride in its last dimension")


def _strides(t: torch.Tensor, name: str, ndim: int, dtype: torch.dtype, device: torch.device):
    """Strides of an input that may be a view: a CUDA tensor of this dtype on
    the CUDA device ``device``, with unit stride in its last dimension."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    st = t.stride()
    if t.dtype is not dtype or len(st) != ndim or t.device != device or st[-1] != 1:
        _refuse(t, name, ndim, dtype, device)
    for x in st[:-1]:
        if x & 7:
            # a stride off the 16-byte grid matters only where it is walked
            return tuple(0 if n == 1 else x for n, x in zip(t.shape, st))
    return st


def _pair(k: torch.Tensor, v: torch.Tensor, names, ndim: int, dtype: torch.dtype, device: torch.device):
    """The strides that k and v share."""
    if isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor):
        st = k.stride()
        if len(st) == ndim and st[-1] == 1 and not (st[0] | st[1] | st[ndim - 2]) & 7 and v.stride() == st \
                and k.dtype is dtype and v.dtype is dtype and k.device == device and v.device == device \
                and v.shape == k.shape:
            return st
    sk = _strides(k, names[0], ndim, dtype, device)
    sv = _strides(v, names[1], ndim, dtype, device)
    if v.shape != k.shape or (sv != sk and any(n > 1 and a != b for n, a, b in zip(k.shape, sk, sv))):
        raise ValueError(f"{names[0]} and {names[1]} must have the same shape and strides")
    return sk


def _ints(t: torch.Tensor, name: str, ndim: int, device: torch.device) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.ndim != ndim or t.device != device \
            or (t.stride(-1) != 1 and t.shape[-1] > 1):
        _refuse(t, name, ndim, torch.int32, device)


def _cuda_device(t: torch.Tensor, name: str) -> torch.device:
    """The device of a call's 16-bit tensors."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPE_CODES:
        raise TypeError(f"{name} must be a bfloat16 or float16 torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (liboss has no CPU path)")
    return t.device


def _cache(k_pages, v_pages, page_table, kv_len):
    """``(os_paged_cache, device, batch, heads, head_dim, capacity, page_size)`` of
    these tensors; capacity: the tokens that a row of the page table holds."""
    dev = _cuda_device(k_pages, "k_pages")
    dtype = k_pages.dtype
    st = _pair(k_pages, v_pages, ("k_pages", "v_pages"), 4, dtype, dev)
    _ints(page_table, "page_table", 2, dev)
    _ints(kv_len, "kv_len", 1, dev)
    pages, heads, page_size, d = k_pages.shape
    batch, max_pages = page_table.shape
    if kv_len.shape[0] != batch:
        raise ValueError("kv_len must have one entry for each row of page_table")
    try:
        packed = _PAGED_CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), st[0], st[1], st[2],
                                   page_table.data_ptr(), page_table.stride(0), kv_len.data_ptr(), pages, heads,
                                   page_size, d, _DTYPE_CODES[dtype], batch, max_pages)
    except struct.error:
        raise ValueError("more pages than 32 bits count") from None
    return packed, dev, batch, heads, d, max_pages * page_size, page_size


def _elsewhere(dev: torch.device, stream) -> bool:
    """Whether a call for tensors on ``dev`` has to change the current stream
    or device first (``_on``)."""
    return stream is not None or dev.index != _current_device()


def _on(dev: torch.device, stream):
    """The context in which such a call allocates and launches. Outputs and
    workspaces come from PyTorch's allocator under it, so that their memory is
    ordered with the stream that uses it."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


# The current device, and the raw current stream of a device, without making a
# Stream object. Where PyTorch lacks these names (a build without CUDA has none of
# them), its public calls stand in, which fail when they are made, not at import.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)

# Workspaces of the calls that launch two kernels, kept per (device, stream) up
# to this size. The lock is held from taking one to the end of the launches:
# kernels of two threads' calls on one stream would otherwise alternate on it. A call
# under capture gets its own from the graph's memory.
_KEEP_BYTES = 64 << 20
_LAUNCH_LOCK = threading.Lock()


def _scratch(dev: torch.device, sp: int, nbytes: int) -> torch.Tensor:
    if nbytes > _KEEP_BYTES or _capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    key = (dev.index, sp, "cache")
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _WORKSPACES[key] = ws
    return ws


def attention_fwd_packed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         cu_seqlens_q: torch.Tensor, cu_seqlens_k: Optional[torch.Tensor] = None,
                         scale: Optional[float] = None, causal: bool = True,
                         o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         stream=None):
    """Attention forward over packed sequences: q [tokens_q, Hq, D], k and v
    [tokens_k, Hkv, D] (bf16 or fp16, D 64 or 128, Hq a multiple of Hkv; views
    such as slices of a fused projection are taken as they are, k and v with the
    same strides), cu_seqlens_q and cu_seqlens_k [batch + 1] int32 on the device
    (cu_seqlens_k None: the same). Causal: a sequence's queries are the last of
    its keys' positions. Returns ``(o, lse)``, [tokens_q, Hq, D] and fp32
    [tokens_q, Hq]; rows outside every sequence are left as they were. See
    ``os_attention_fwd_packed``."""
    dev = _cuda_device(q, "q")
    sq = _strides(q, "q", 3, q.dtype, dev)
    sk = _pair(k, v, ("k", "v"), 3, q.dtype, dev)
    tokens_q, hq, d = q.shape
    tokens_k, hkv, dk = k.shape
    if dk != d:
        raise ValueError("q, k and v must have the same head dimension")
    if hkv < 1 or hq < 1 or hq % hkv:
        raise ValueError(f"{hq} query heads cannot share {hkv} key heads")
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens_q
    _ints(cu_seqlens_q, "cu_seqlens_q", 1, dev)
    _ints(cu_seqlens_k, "cu_seqlens_k", 1, dev)
    batch = cu_seqlens_q.shape[0] - 1
    if batch < 1 or cu_seqlens_k.shape[0] != batch + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have batch + 1 entries each")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is not None:
        _out(o, "o", q.dtype, (tokens_q, hq, d), dev)
    if lse is not None:
        _out(lse, "lse", torch.float32, (tokens_q, hq), dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attention_fwd_packed(q, k, v, cu_seqlens_q, cu_seqlens_k, scale, causal, o, lse)
    if o is None:
        o = torch.empty((tokens_q, hq, d), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((tokens_q, hq), dtype=torch.float32, device=dev)
    lib = load()
    need = lib.os_attention_fwd_packed_workspace_bytes(tokens_k, hkv, d)
    if need < 0:
        raise OssError(4, "os_attention_fwd_packed_workspace_bytes")
    sp = _raw_stream(dev.index)
    with _LAUNCH_LOCK:
        ws = _scratch(dev, sp, need)
        st = lib.os_attention_fwd_packed(
            q.data_ptr(), sq[0], sq[1], k.data_ptr(), v.data_ptr(), sk[0], sk[1], o.data_ptr(),
            lse.data_ptr(), cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), batch, tokens_q,
            tokens_k, hq, hkv, d, _DTYPE_CODES[q.dtype], scale, bool(causal), ws.data_ptr(), need, sp)
    _check(st, "os_attention_fwd_packed")
    return o, lse


def kv_cache_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                    page_table: torch.Tensor, kv_len: torch.Tensor,
                    cu_seqlens: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy new tokens' k and v [tokens, Hkv, D] into the pages of a cache:
    k_pages and v_pages [pages, Hkv, page_size, D] (any strides, the same for
    both), page_table [batch, max_pages] and kv_len [batch] int32 on the device.
    kv_len counts the new tokens: those of sequence b, rows cu_seqlens[b] ..
    cu_seqlens[b + 1] - 1, go to its last positions. cu_seqlens None: one token
    for each sequence, none for those of kv_len 0. See ``os_kv_cache_append``."""
    cache, dev, batch, heads, d, _, _ = _cache(k_pages, v_pages, page_table, kv_len)
    sk = _pair(k, v, ("k", "v"), 3, k_pages.dtype, dev)
    tokens, hk, dk = k.shape
    if hk != heads or dk != d:
        raise ValueError(f"k and v must be [tokens, {heads}, {d}] like the cache")
    cu = None
    if cu_seqlens is not None:
        _ints(cu_seqlens, "cu_seqlens", 1, dev)
        if cu_seqlens.shape[0] != batch + 1:
            raise ValueError("cu_seqlens must have batch + 1 entries")
        cu = cu_seqlens.data_ptr()
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return kv_cache_append(k, v, k_pages, v_pages, page_table, kv_len, cu_seqlens)
    st = load().os_kv_cache_append(k.data_ptr(), v.data_ptr(), sk[0], sk[1], tokens, cu, cache,
                                   _raw_stream(dev.index))
    _check(st, "os_kv_cache_append")


def _weights(weights: torch.Tensor, batch: int, heads: int, capacity: int, device: torch.device):
    if not isinstance(weights, torch.Tensor) or weights.dtype is not torch.float32 or weights.dim() != 3 \
            or weights.device != device or (weights.stride(-1) != 1 and weights.shape[-1] > 1):
        _refuse(weights, "weights", 3, torch.float32, device)
    b, h, n = weights.shape
    if b != batch or h != heads or n < capacity:
        raise ValueError(f"weights must be [{batch}, {heads}, n] with n >= max_pages * page_size")
    return weights.stride()


def attention_decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                           page_table: torch.Tensor, kv_len: torch.Tensor,
                           scale: Optional[float] = None, weights: Optional[torch.Tensor] = None,
                           o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                           stream=None):
    """Attention of one new token per sequence, q [batch, Hq, D], over a paged
    cache (see ``kv_cache_append``; append the new token first), Hq a multiple of
    Hkv. ``weights`` (fp32 [batch, Hkv, n], n at least what the page table's rows
    hold) is updated in place: each cached token's attention weight, summed
    over the query heads of its key head, is added to it. Returns ``(o, lse)``,
    [batch, Hq, D] and fp32 [batch, Hq]. See ``os_attention_decode_paged``."""
    cache, dev, batch, heads, d, capacity, _ = _cache(k_pages, v_pages, page_table, kv_len)
    dtype = k_pages.dtype
    sq = _strides(q, "q", 3, dtype, dev)
    bq, hq, dq = q.shape
    if bq != batch or dq != d:
        raise ValueError(f"q must be [{batch}, Hq, {d}] like the cache")
    if heads < 1 or hq < 1 or hq % heads:
        raise ValueError(f"{hq} query heads cannot share {heads} key heads")
    w, sw = None, (0, 0)
    if weights is not None:
        sw = _weights(weights, batch, heads, capacity, dev)
        w = weights.data_ptr()
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is not None:
        _out(o, "o", dtype, (batch, hq, d), dev)
    if lse is not None:
        _out(lse, "lse", torch.float32, (batch, hq), dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attention_decode_paged(q, k_pages, v_pages, page_table, kv_len, scale, weights, o, lse)
    if o is None:
        o = torch.empty((batch, hq, d), dtype=dtype, device=dev)
    if lse is None:
        lse = torch.empty((batch, hq), dtype=torch.float32, device=dev)
    lib = load()
    need = lib.os_attention_decode_paged_workspace_bytes(hq, cache, w is not None)
    if need < 0:
        raise OssError(4, "os_attention_decode_paged_workspace_bytes")
    sp = _raw_stream(dev.index)
    with _LAUNCH_LOCK:
        ws = _scratch(dev, sp, need)
        st = lib.os_attention_decode_paged(q.data_ptr(), sq[0], sq[1], hq, cache, scale, o.data_ptr(),
                                           lse.data_ptr(), w, sw[0], sw[1], ws.data_ptr(), need, sp)
    _check(st, "os_attention_decode_paged")
    return o, lse


def kv_cache_evict(k_pages: torch.Tensor, v_pages: torch.Tensor, weights: torch.Tensor,
                   page_table: torch.Tensor, kv_len: torch.Tensor, new_page_table: torch.Tensor,
                   budget: int, recent: int = 0, kept: Optional[torch.Tensor] = None,
                   new_len: Optional[torch.Tensor] = None,
                   new_weights: Optional[torch.Tensor] = None, stream=None):
    """Keep at most ``budget`` cached tokens of each sequence and key head: the
    last ``recent`` and, of the others, those of the largest ``weights`` (as
    ``attention_decode_paged`` sums them). Their rows are copied, in the order
    of their positions, to the pages that new_page_table [batch, new_max_pages]
    names in the same pools, which nothing else may use; the old pages are only
    read. Returns ``(kept, new_len, new_weights)``: the kept positions [batch,
    Hkv, budget] (-1 behind the last), the new kv_len and the kept tokens'
    weights [batch, Hkv, new_max_pages * page_size] (0 behind the last), ready
    for the next decode. See ``os_kv_cache_evict``."""
    cache, dev, batch, heads, _, capacity, page_size = _cache(k_pages, v_pages, page_table, kv_len)
    sw = _weights(weights, batch, heads, capacity, dev)
    _ints(new_page_table, "new_page_table", 2, dev)
    rows, new_max = new_page_table.shape
    if rows != batch:
        raise ValueError("new_page_table must have one row for each row of page_table")
    budget, recent = int(budget), int(recent)
    room = new_max * page_size
    if not 1 <= budget <= room:
        raise ValueError(f"budget {budget} outside 1 .. {room}, what the new pages hold")
    if not 0 <= recent <= budget:
        raise ValueError(f"recent {recent} outside 0 .. budget")
    if kept is not None:
        _out(kept, "kept", torch.int32, (batch, heads, budget), dev)
    if new_len is not None:
        _out(new_len, "new_len", torch.int32, (batch,), dev)
    if new_weights is not None:
        _out(new_weights, "new_weights", torch.float32, (batch, heads, room), dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return kv_cache_evict(k_pages, v_pages, weights, page_table, kv_len, new_page_table, budget, recent, kept,
                                  new_len, new_weights)
    if kept is None:
        kept = torch.empty((batch, heads, budget), dtype=torch.int32, device=dev)
    if new_len is None:
        new_len = torch.empty(batch, dtype=torch.int32, device=dev)
    if new_weights is None:
        new_weights = torch.empty((batch, heads, room), dtype=torch.float32, device=dev)
    st = load().os_kv_cache_evict(cache, weights.data_ptr(), sw[0], sw[1], new_page_table.data_ptr(),
                                  new_page_table.stride(0), new_max, budget, recent, kept.data_ptr(),
                                  new_len.data_ptr(), new_weights.data_ptr(), _raw_stream(dev.index))
    _check(st, "os_kv_cache_evict")
    return kept, new_len, new_weights


def attention_decode_shared(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                            prefix_table: torch.Tensor, prefix_len: torch.Tensor, page_table: torch.Tensor,
                            kv_len: torch.Tensor, cu_groups: Optional[torch.Tensor] = None,
                            scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, stream=None):
    """``attention_decode_paged`` for sequences that share prefixes: the keys of a
    sequence of group g are the prefix_len[g] tokens in the pages of row g of
    prefix_table [groups, max_prefix_pages], then its own (page_table, kv_len) in
    the same pools. A long prefix is read once for up to 128 rows of its group's queries
    and heads, a short one by every sequence. cu_groups [groups + 1]:
    group g is sequences cu_groups[g] .. cu_groups[g + 1] - 1 (None: one group of all).
    All of them int32 on the device. Returns ``(o, lse)``, [batch, Hq, D] and fp32
    [batch, Hq]. See ``os_attention_decode_shared``."""
    cache, dev, batch, heads, d, _, _ = _cache(k_pages, v_pages, page_table, kv_len)
    dtype = k_pages.dtype
    sq = _strides(q, "q", 3, dtype, dev)
    bq, hq, dq = q.shape
    if bq != batch or dq != d:
        raise ValueError(f"q must be [{batch}, Hq, {d}] like the cache")
    if heads < 1 or hq < 1 or hq % heads:
        raise ValueError(f"{hq} query heads cannot share {heads} key heads")
    _ints(prefix_table, "prefix_table", 2, dev)
    _ints(prefix_len, "prefix_len", 1, dev)
    groups, prefix_pages = prefix_table.shape
    if prefix_len.shape[0] != groups:
        raise ValueError("prefix_len must have one entry for each row of prefix_table")
    cu = None
    if cu_groups is not None:
        _ints(cu_groups, "cu_groups", 1, dev)
        if cu_groups.shape[0] != groups + 1:
            raise ValueError("cu_groups must have one entry more than prefix_table has rows")
        cu = cu_groups.data_ptr()
    elif groups != 1:
        raise ValueError("several groups need cu_groups")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is not None:
        _out(o, "o", dtype, (batch, hq, d), dev)
    if lse is not None:
        _out(lse, "lse", torch.float32, (batch, hq), dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attention_decode_shared(q, k_pages, v_pages, prefix_table, prefix_len, page_table, kv_len, cu_groups,
                                           scale, o, lse)
    if o is None:
        o = torch.empty((batch, hq, d), dtype=dtype, device=dev)
    if lse is None:
        lse = torch.empty((batch, hq), dtype=torch.float32, device=dev)
    lib = load()
    need = lib.os_attention_decode_shared_workspace_bytes(hq, cache, prefix_pages, groups)
    if need < 0:
        raise OssError(4, "os_attention_decode_shared_workspace_bytes")
    sp = _raw_stream(dev.index)
    with _LAUNCH_LOCK:
        ws = _scratch(dev, sp, need)
        st = lib.os_attention_decode_shared(q.data_ptr(), sq[0], sq[1], hq, cache, prefix_table.data_ptr(),
                                            prefix_table.stride(0), prefix_len.data_ptr(), prefix_pages, cu, groups,
                                            scale, o.data_ptr(), lse.data_ptr(), ws.data_ptr(), need, sp)
    _check(st, "os_attention_decode_shared")
    return o, lse


# -- the cache in 8 bits ---------------------------------------------------------------------

# (None on a PyTorch before 2.7: the 8-bit cache is not there, the rest is)
_F8, _E8 = getattr(torch, "float8_e4m3fn", None), getattr(torch, "float8_e8m0fnu", None)


def _scale_strides(t: torch.Tensor, name: str, shape, device: torch.device):
    """Strides of the scales [pages, heads, page_size] of a pool."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _E8 or t.dim() != 3 or t.device != device \
            or t.stride(2) != 1:
        _refuse(t, name, 3, _E8, device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, a scale for each row of the pages")
    st = t.stride()
    if (st[0] | st[1]) & 15:
        # a stride off the 16-byte grid matters only where it is walked
        return tuple(0 if n == 1 else x for n, x in zip(shape, st))
    return st


def _cache_fp8(k_pages, v_pages, k_scales, v_scales, page_table, kv_len, dtype):
    """``(os_paged_cache_fp8, device, batch, heads, head_dim)`` of these tensors, for
    calls whose 16-bit tensors are of ``dtype``."""
    try:
        st, ss, shape, index = k_pages.stride(), k_scales.stride(), k_pages.shape, k_pages.get_device()
        plain = (k_pages.dtype is _F8 and v_pages.dtype is _F8 and k_scales.dtype is _E8 and v_scales.dtype is _E8
                 and page_table.dtype is torch.int32 and kv_len.dtype is torch.int32 and dtype in _DTYPE_CODES
                 and 0 <= index == v_pages.get_device() == k_scales.get_device() == v_scales.get_device()
                 == page_table.get_device() == kv_len.get_device()
                 and len(shape) == 4 and v_pages.shape == shape and v_pages.stride() == st and v_scales.stride() == ss
                 and k_scales.shape == v_scales.shape == shape[:3] and st[3] == ss[2] == 1
                 and not (st[0] | st[1] | st[2] | ss[0] | ss[1]) & 15)
    except (AttributeError, RuntimeError):
        plain = False
    if plain:
        dev, rows, lens = k_pages.device, page_table.shape, kv_len.shape
        ld_table = page_table.stride()
        plain = len(rows) == 2 and len(lens) == 1 and ld_table[1] == 1 and kv_len.stride() == (1,)
    if not plain:
        dev, st, ss = _cache_fp8_checked(k_pages, v_pages, k_scales, v_scales, page_table, kv_len, dtype)
        shape, rows, lens, ld_table = k_pages.shape, page_table.shape, kv_len.shape, page_table.stride()
    pages, heads, page_size, d = shape
    batch, max_pages = rows
    if lens[0] != batch:
        raise ValueError("kv_len must have one entry for each row of page_table")
    try:
        packed = _PAGED_CACHE_FP8.pack(k_pages.data_ptr(), v_pages.data_ptr(), st[0], st[1], st[2],
                                       page_table.data_ptr(), ld_table[0], kv_len.data_ptr(), pages, heads,
                                       page_size, d, _DTYPE_CODES[dtype], batch, max_pages, k_scales.data_ptr(),
                                       v_scales.data_ptr(), ss[0], ss[1])
    except struct.error:
        raise ValueError("more pages than 32 bits count") from None
    return packed, dev, batch, heads, d


def _cache_fp8_checked(k_pages, v_pages, k_scales, v_scales, page_table, kv_len, dtype):
    """The device and strides of a cache that the quick check has not passed: a view
    off the common path, or what is wrong with it is raised."""
    if _F8 is None or _E8 is None:
        raise RuntimeError("the 8-bit cache needs a PyTorch with float8_e4m3fn and float8_e8m0fnu")
    if not isinstance(k_pages, torch.Tensor) or k_pages.dtype is not _F8:
        raise TypeError("k_pages must be a float8_e4m3fn torch.Tensor")
    if not k_pages.is_cuda:
        raise ValueError("k_pages must be a CUDA tensor (liboss has no CPU path)")
    if dtype not in _DTYPE_CODES:
        raise TypeError(f"{dtype} is neither bfloat16 nor float16")
    dev = k_pages.device
    st = _pair(k_pages, v_pages, ("k_pages", "v_pages"), 4, _F8, dev)
    shape = k_pages.shape
    if (st[0] | st[1] | st[2]) & 15:
        # a stride off the grid matters only where it is walked
        st = tuple(0 if n == 1 and x & 15 else x for n, x in zip(shape, st))
    ss = _scale_strides(k_scales, "k_scales", shape[:3], dev)
    sv = _scale_strides(v_scales, "v_scales", shape[:3], dev)
    if sv != ss and any(n > 1 and a != b for n, a, b in zip(shape, ss, sv)):
        raise ValueError("k_scales and v_scales must have the same strides")
    _ints(page_table, "page_table", 2, dev)
    _ints(kv_len, "kv_len", 1, dev)
    return dev, st, ss


def _seqlens(cu_seqlens: torch.Tensor, batch: int, dev: torch.device) -> int:
    _ints(cu_seqlens, "cu_seqlens", 1, dev)
    if cu_seqlens.shape[0] != batch + 1:
        raise ValueError("cu_seqlens must have batch + 1 entries")
    return cu_seqlens.data_ptr()


def kv_cache_append_fp8(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                        k_scales: torch.Tensor, v_scales: torch.Tensor, page_table: torch.Tensor,
                        kv_len: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, stream=None) -> None:
    """``kv_cache_append`` into a cache in 8 bits: k and v [tokens, Hkv, D] (bf16 or
    fp16) are quantised as they are written. k_pages and v_pages [pages, Hkv,
    page_size, D] float8_e4m3fn (any strides, multiples of 16, the same for both),
    k_scales and v_scales [pages, Hkv, page_size] float8_e8m0fnu: a row's values are
    its codes times its scale, the smallest power of two with which they fit. See
    ``os_kv_cache_append_fp8``."""
    dev = _cuda_device(k, "k")
    dtype = k.dtype
    cache, pool_dev, batch, heads, d = _cache_fp8(k_pages, v_pages, k_scales, v_scales, page_table, kv_len, dtype)
    if pool_dev != dev:
        raise ValueError(f"k is on {dev}, the cache on {pool_dev}")
    sk = _pair(k, v, ("k", "v"), 3, dtype, dev)
    tokens, hk, dk = k.shape
    if hk != heads or dk != d:
        raise ValueError(f"k and v must be [tokens, {heads}, {d}] like the cache")
    cu = None if cu_seqlens is None else _seqlens(cu_seqlens, batch, dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return kv_cache_append_fp8(k, v, k_pages, v_pages, k_scales, v_scales, page_table, kv_len, cu_seqlens)
    st = load().os_kv_cache_append_fp8(k.data_ptr(), v.data_ptr(), sk[0], sk[1], tokens, cu, cache,
                                       _raw_stream(dev.index))
    _check(st, "os_kv_cache_append_fp8")


def kv_cache_read_fp8(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                      page_table: torch.Tensor, kv_len: torch.Tensor, cu_seqlens: torch.Tensor, tokens: int,
                      dtype: torch.dtype = torch.bfloat16, k: Optional[torch.Tensor] = None,
                      v: Optional[torch.Tensor] = None, stream=None):
    """Cached tokens of a cache in 8 bits (see ``kv_cache_append_fp8``) as packed rows
    of ``dtype`` (bf16 or fp16), the k and v that ``attention_fwd_packed`` takes: rows
    cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of ``tokens`` get the last positions of
    sequence b, all of them where there are kv_len[b] rows. Returns ``(k, v)`` [tokens,
    Hkv, D]; given ones may be views with the same strides. Rows outside every sequence
    are left as they were. See ``os_kv_cache_read_fp8``."""
    cache, dev, batch, heads, d = _cache_fp8(k_pages, v_pages, k_scales, v_scales, page_table, kv_len, dtype)
    cu = _seqlens(cu_seqlens, batch, dev)
    tokens = int(tokens)
    if tokens < 0:
        raise ValueError("tokens must be >= 0")
    if (k is None) != (v is None):
        raise ValueError("k and v are given together or not at all")
    if k is not None:
        sk = _pair(k, v, ("k", "v"), 3, dtype, dev)
        if tuple(k.shape) != (tokens, heads, d):
            raise ValueError(f"k and v must be [{tokens}, {heads}, {d}]")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return kv_cache_read_fp8(k_pages, v_pages, k_scales, v_scales, page_table, kv_len, cu_seqlens, tokens, dtype,
                                     k, v)
    if k is None:
        k = torch.empty((tokens, heads, d), dtype=dtype, device=dev)
        v = torch.empty_like(k)
        sk = k.stride()
    st = load().os_kv_cache_read_fp8(cache, cu, tokens, k.data_ptr(), v.data_ptr(), sk[0], sk[1], _raw_stream(dev.index))
    _check(st, "os_kv_cache_read_fp8")
    return k, v


def attention_decode_paged_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                               v_scales: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                               scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                               lse: Optional[torch.Tensor] = None, stream=None):
    """``attention_decode_paged`` (without weights) over a cache in 8 bits (see
    ``kv_cache_append_fp8``): q [batch, Hq, D] bf16 or fp16. Returns ``(o, lse)``,
    [batch, Hq, D] of q's type and fp32 [batch, Hq]. See
    ``os_attention_decode_paged_fp8``."""
    dev = _cuda_device(q, "q")
    dtype = q.dtype
    cache, pool_dev, batch, heads, d = _cache_fp8(k_pages, v_pages, k_scales, v_scales, page_table, kv_len, dtype)
    if pool_dev != dev:
        raise ValueError(f"q is on {dev}, the cache on {pool_dev}")
    sq = _strides(q, "q", 3, dtype, dev)
    bq, hq, dq = q.shape
    if bq != batch or dq != d:
        raise ValueError(f"q must be [{batch}, Hq, {d}] like the cache")
    if heads < 1 or hq < 1 or hq % heads:
        raise ValueError(f"{hq} query heads cannot share {heads} key heads")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is not None:
        _out(o, "o", dtype, (batch, hq, d), dev)
    if lse is not None:
        _out(lse, "lse", torch.float32, (batch, hq), dev)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attention_decode_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, page_table, kv_len, scale, o, lse)
    if o is None:
        o = torch.empty((batch, hq, d), dtype=dtype, device=dev)
    if lse is None:
        lse = torch.empty((batch, hq), dtype=torch.float32, device=dev)
    lib = load()
    need = lib.os_attention_decode_paged_fp8_workspace_bytes(hq, cache)
    if need < 0:
        raise OssError(4, "os_attention_decode_paged_fp8_workspace_bytes")
    sp = _raw_stream(dev.index)
    with _LAUNCH_LOCK:
        ws = _scratch(dev, sp, need)
        st = lib.os_attention_decode_paged_fp8(q.data_ptr(), sq[0], sq[1], hq, cache, scale, o.data_ptr(),
                                               lse.data_ptr(), ws.data_ptr(), need, sp)
    _check(st, "os_attention_decode_paged_fp8")
    return o, lse


RESCALE_POLICIES = {"threshold": 0, "on_rise": 1, "always": 2}


def set_rescale_policy(policy) -> None:
    """Rescale policy of this thread's later attention calls: "threshold"
    (default), "on_rise" or "always" (or the os_rescale_policy value). See
    ``os_attention_set_rescale_policy``."""
    code = RESCALE_POLICIES.get(policy, policy)
    _check(load().os_attention_set_rescale_policy(int(code)), "os_attention_set_rescale_policy")


def rescale_policy() -> str:
    code = int(load().os_attention_rescale_policy())
    return {v: k for k, v in RESCALE_POLICIES.items()}[code]


def debug_inject_fault(kind: int, step: int = 0, timeout_ns: int = 0) -> None:
    """Test hook: arm a fault for the next attention_fwd call (kind 1) or
    row softmax call (kind 2) on this thread; kind 0 disarms (see
    ``os_debug_inject_fault`` in include/oss.h)."""
    _check(load().os_debug_inject_fault(int(kind), int(step), int(timeout_ns)),
           "os_debug_inject_fault")


def check_device_error(stream=None) -> int:
    """Synchronise ``stream`` and read/clear the device error word; raises
    OssError(OS_ERR_TIMEOUT) when a kernel gave up on a bounded wait, and
    OssError(OS_ERR_BAD_INDEX) when a call on a paged cache or packed sequences
    met an index outside them."""
    code = _i32(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if stream is None else stream.device
    with torch.cuda.device(dev):
        st = load().os_check_device_error(_stream_ptr(stream, dev), ctypes.byref(code))
    if st != OS_OK:
        # a launch that gave up may have left counters in its workspace:
        # later calls get fresh zero-filled ones
        _WORKSPACES.clear()
    _check(st, f"os_check_device_error (code {code.value:#x})")
    return int(code.value)
