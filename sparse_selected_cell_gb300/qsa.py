"""Thin ctypes binding over libqsa.so (include/qsa.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
CPU fallback: when the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional

import torch

from . import gen

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqsa.so")

QSA_OK, QSA_ERR_ARG, QSA_ERR_UNSUPPORTED, QSA_ERR_CAPACITY, QSA_ERR_CUDA, QSA_ERR_DEVICE_CHECK = range(6)
ATTN_DEFAULT, ATTN_TCGEN05, ATTN_TCGEN05_SM = 0, 1, 2
DEV_BITS = {1: "bad selection count", 2: "union overflow", 4: "bad cell", 8: "bad page-table entry",
            16: "bad union count", 32: "device wait timeout", 64: "bad sequence length", 128: "no page",
            256: "token overflow", 512: "bad axis"}
BF16, F16, F32 = 0, 1, 2          # element types (QSA_BF16, QSA_F16, QSA_F32)

_lib = None
_P, _I, _F, _S, _L = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t, ctypes.c_int64
# The argument structs of the packed calls: one conversion of all arguments (0.3 us) instead of one each (2 to 3 us).
_PAGED_ARGS = struct.Struct("PiPPPPPiiiiiPiifPiPPNPP").pack
_APPEND_ARGS = struct.Struct("PqPqPqiPiiPPiiPqPPPPPiiiiPP").pack
_GATHER_ARGS = struct.Struct("PPPPPiiiPPiPP").pack
_TABLES_ARGS = struct.Struct("PPiPiiiPiPiPPPPPPPP").pack


class QsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({lib().qsa_status_str(status).decode()})")
        self.status = status


def lib():
    """Load libqsa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                               "g.build()'` (no CPU fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        L.qsa_attn_default_variant.argtypes = []
        L.qsa_attn_default_variant.restype = ctypes.c_int
        L.qsa_status_str.argtypes = [ctypes.c_int]
        L.qsa_status_str.restype = ctypes.c_char_p
        L.qsa_union_workspace_bytes.argtypes = [_I, _I]
        L.qsa_union_workspace_bytes.restype = _S
        L.qsa_union_build.argtypes = [_P, _P, _I, _I, _P, _P, _P, _I, _P, _P]
        L.qsa_union_build.restype = ctypes.c_int
        L.qsa_union_attn.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _I, _I, _F, _P, _I, _P, _P]
        L.qsa_union_attn.restype = ctypes.c_int
        L.qsa_prompt_attn.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _F, _P, _P, _S, _I, _I,
                                      _P, _P]
        L.qsa_prompt_attn.restype = ctypes.c_int
        L.qsa_prompt_attn_static.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _F, _P, _I, _I,
                                             _P, _P]
        L.qsa_prompt_attn_static.restype = ctypes.c_int
        L.qsa_fused_attn.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _F, _P, _P, _P]
        L.qsa_fused_attn.restype = ctypes.c_int
        L.qsa_select_attn.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _F, _P, _P, _P]
        L.qsa_select_attn.restype = ctypes.c_int
        L.qsa_decode_attn.argtypes = [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _I, _F, _P, _P, _P]
        L.qsa_decode_attn.restype = ctypes.c_int
        L.qsa_paged_attn.argtypes = [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _I, _F, _P, _I, _P, _P,
                                     _S, _P, _P]
        L.qsa_paged_attn.restype = ctypes.c_int
        L.qsa_paged_attn_workspace_bytes.argtypes = [_I, _I]
        L.qsa_paged_attn_workspace_bytes.restype = _S
        L.qsa_rope_append.argtypes = [_P, _L, _P, _L, _P, _L, _I, _P, _I, _I, _P, _P, _I, _I, _P, _L, _P, _P, _P, _P,
                                      _P, _I, _I, _I, _I, _P, _P]
        L.qsa_rope_append.restype = ctypes.c_int
        L.qsa_rope.argtypes = [_P, _L, _I, _P, _I, _I, _P, _P, _I, _I, _P, _L, _I, _I, _P, _P]
        L.qsa_rope.restype = ctypes.c_int
        L.qsa_cache_gather.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _I, _P, _P]
        L.qsa_cache_gather.restype = ctypes.c_int
        L.qsa_extend_tables.argtypes = [_P, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P]
        L.qsa_extend_tables.restype = ctypes.c_int
        for f in (L.qsa_paged_attn_packed, L.qsa_rope_append_packed, L.qsa_cache_gather_packed, L.qsa_extend_tables_packed):
            f.argtypes = [ctypes.c_char_p]
            f.restype = ctypes.c_int
        L.qsa_wait_selftest.argtypes = [_I, _P, _P]
        L.qsa_wait_selftest.restype = ctypes.c_int
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: torch.Tensor, name: str, dtypes) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_B16 = (torch.bfloat16, torch.int16, torch.uint16)
_H16 = (torch.float16, torch.int16, torch.uint16)


def _attn_inputs(q, k_pool, v_pool, k_scale, v_scale, page_table, out):
    """Device, dtype and shape checks shared by the attention calls; returns out
    (allocated here when not given: float32 [n_q, n_kv*12, 128])."""
    _dev(q, "q", _B16)
    _dev(k_pool, "k_pool", (torch.int8,))
    _dev(v_pool, "v_pool", (torch.int8,))
    _dev(k_scale, "k_scale", _H16)
    _dev(v_scale, "v_scale", _H16)
    _dev(page_table, "page_table", (torch.int32,))
    if q.dim() != 3 or q.shape[2] != gen.HEAD_DIM or q.shape[1] % gen.HEADS_PER_KV != 0:
        raise ValueError(f"q must be [n_q, n_kv*12, 128], got {tuple(q.shape)}")
    shape = (int(q.shape[0]), int(q.shape[1]), gen.HEAD_DIM)
    if out is None:
        return torch.empty(shape, dtype=torch.float32, device=q.device)
    _dev(out, "out", (torch.float32,))
    if tuple(out.shape) != shape:
        raise ValueError(f"out must have shape {shape}, got {tuple(out.shape)}")
    return out


def _check(fn: str, rc: int):
    if rc != QSA_OK:
        raise QsaError(fn, rc)


def default_variant() -> int:
    """The attention variant QSA_ATTN_DEFAULT resolves to in the loaded library."""
    return int(lib().qsa_attn_default_variant())


def workspace_bytes(n_q: int, union_stride: int = gen.UNION_STRIDE) -> int:
    return int(lib().qsa_union_workspace_bytes(int(n_q), int(union_stride)))


def union_build(sel: torch.Tensor, sel_count: torch.Tensor, union_stride: int = gen.UNION_STRIDE,
                out=None, dev_status: Optional[torch.Tensor] = None, stream=None):
    """-> (union_cells int32 [G, stride], union_mask uint8 [G, stride], union_count int32 [G])."""
    _dev(sel, "sel", (torch.int32,))
    _dev(sel_count, "sel_count", (torch.int32,))
    n_q = int(sel_count.shape[0])
    n_groups = (n_q + 7) // 8
    if out is None:
        out = (torch.empty((n_groups, union_stride), dtype=torch.int32, device=sel.device),
               torch.empty((n_groups, union_stride), dtype=torch.uint8, device=sel.device),
               torch.empty((n_groups,), dtype=torch.int32, device=sel.device))
    ucell, umask, ucount = out
    rc = lib().qsa_union_build(_ptr(sel), _ptr(sel_count), n_q, int(sel.shape[1]), _ptr(ucell), _ptr(umask),
                               _ptr(ucount), int(union_stride), _ptr(dev_status), _stream(stream))
    _check("qsa_union_build", rc)
    return ucell, umask, ucount


def union_attn(q, k_pool, v_pool, k_scale, v_scale, page_table, union_cells, union_mask, union_count,
               sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None, variant: int = ATTN_DEFAULT,
               dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Union attention -> out float32 [n_q, n_kv*12, 128]."""
    out = _attn_inputs(q, k_pool, v_pool, k_scale, v_scale, page_table, out)
    n_q, n_heads = int(q.shape[0]), int(q.shape[1])
    n_kv = n_heads // gen.HEADS_PER_KV
    if sm_scale is None:
        sm_scale = gen.HEAD_DIM ** -0.5
    rc = lib().qsa_union_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                              int(page_table.shape[0]), int(k_pool.shape[0]), n_kv, _ptr(union_cells),
                              _ptr(union_mask), _ptr(union_count), int(union_cells.shape[1]), n_q, float(sm_scale),
                              _ptr(out), int(variant), _ptr(dev_status), _stream(stream))
    _check("qsa_union_attn", rc)
    return out


def prompt_attn(q, k_pool, v_pool, k_scale, v_scale, page_table, sel, sel_count,
                sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, union_stride: int = gen.UNION_STRIDE,
                variant: int = ATTN_DEFAULT, dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Union build + union attention in one call, over a caller-owned workspace."""
    out = _attn_inputs(q, k_pool, v_pool, k_scale, v_scale, page_table, out)
    _dev(sel, "sel", (torch.int32,))
    _dev(sel_count, "sel_count", (torch.int32,))
    n_q, n_heads = int(q.shape[0]), int(q.shape[1])
    n_kv = n_heads // gen.HEADS_PER_KV
    need = workspace_bytes(n_q, union_stride)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if sm_scale is None:
        sm_scale = gen.HEAD_DIM ** -0.5
    rc = lib().qsa_prompt_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                               int(page_table.shape[0]), int(k_pool.shape[0]), n_kv, _ptr(sel), _ptr(sel_count),
                               int(sel.shape[1]), n_q, float(sm_scale), _ptr(out), _ptr(workspace),
                               int(workspace.numel() * workspace.element_size()), int(union_stride), int(variant),
                               _ptr(dev_status), _stream(stream))
    _check("qsa_prompt_attn", rc)
    return out


def fused_attn(q, k_pool, v_pool, k_scale, v_scale, page_table, sel, sel_count,
               sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """qsa_fused_attn: the prompt-attention step in one launch, each group's union
    built inside the attention CTA (no workspace) -> out float32 [n_q, n_kv*12, 128]."""
    out = _attn_inputs(q, k_pool, v_pool, k_scale, v_scale, page_table, out)
    _dev(sel, "sel", (torch.int32,))
    _dev(sel_count, "sel_count", (torch.int32,))
    n_q, n_heads = int(q.shape[0]), int(q.shape[1])
    n_kv = n_heads // gen.HEADS_PER_KV
    if sm_scale is None:
        sm_scale = gen.HEAD_DIM ** -0.5
    rc = lib().qsa_fused_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                              int(page_table.shape[0]), int(k_pool.shape[0]), n_kv, _ptr(sel), _ptr(sel_count),
                              int(sel.shape[1]), n_q, float(sm_scale), _ptr(out), _ptr(dev_status), _stream(stream))
    _check("qsa_fused_attn", rc)
    return out


def select_attn(q, k_pool, v_pool, k_scale, v_scale, page_table, sel, sel_count,
                sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Per-position attention without unions (qsa_select_attn) -> out float32 [n_q, n_kv*12, 128]."""
    out = _attn_inputs(q, k_pool, v_pool, k_scale, v_scale, page_table, out)
    _dev(sel, "sel", (torch.int32,))
    _dev(sel_count, "sel_count", (torch.int32,))
    n_q, n_heads = int(q.shape[0]), int(q.shape[1])
    n_kv = n_heads // gen.HEADS_PER_KV
    if sm_scale is None:
        sm_scale = gen.HEAD_DIM ** -0.5
    rc = lib().qsa_select_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                               int(page_table.shape[0]), int(k_pool.shape[0]), n_kv, _ptr(sel), _ptr(sel_count),
                               int(sel.shape[1]), n_q, float(sm_scale), _ptr(out), _ptr(dev_status), _stream(stream))
    _check("qsa_select_attn", rc)
    return out


def decode_attn(q, k_pool, v_pool, k_scale, v_scale, page_tables, sel, sel_count,
                sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None, stream=None,
                n_lpages: Optional[int] = None) -> torch.Tensor:
    """Decode over a batch of sequences (qsa_decode_attn): page_tables int32 [n_q, width], one table per
    query (the first n_lpages entries of its row; n_lpages defaults to the width, which is the stride)
    -> out float32 [n_q, n_kv*12, 128]."""
    _dev(q, "q", _B16)
    _dev(k_pool, "k_pool", (torch.int8,))
    _dev(v_pool, "v_pool", (torch.int8,))
    _dev(k_scale, "k_scale", _H16)
    _dev(v_scale, "v_scale", _H16)
    _dev(page_tables, "page_tables", (torch.int32,))
    _dev(sel, "sel", (torch.int32,))
    _dev(sel_count, "sel_count", (torch.int32,))
    n_q, n_heads = int(q.shape[0]), int(q.shape[1])
    if page_tables.dim() != 2 or int(page_tables.shape[0]) != n_q or not page_tables.is_contiguous():
        raise ValueError("page_tables must be a contiguous [n_q, width] array")
    n_kv = n_heads // gen.HEADS_PER_KV
    if out is None:
        out = torch.empty((n_q, n_heads, gen.HEAD_DIM), dtype=torch.float32, device=q.device)
    _dev(out, "out", (torch.float32,))
    if sm_scale is None:
        sm_scale = gen.HEAD_DIM ** -0.5
    rc = lib().qsa_decode_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(page_tables),
                               int(page_tables.shape[1]),
                               int(page_tables.shape[1]) if n_lpages is None else int(n_lpages),
                               int(k_pool.shape[0]), n_kv,
                               _ptr(sel), _ptr(sel_count), int(sel.shape[1]), n_q, float(sm_scale), _ptr(out),
                               _ptr(dev_status), _stream(stream))
    _check("qsa_decode_attn", rc)
    return out


# ---------------------------------------------------------------- serving a cache
# The operators around the paged cache (include/qsa.h, "Serving a cache").  Single
# tokens make these calls short (the kernels take a few microseconds), so each call
# checks its arguments in one expression and passes raw addresses; only when that
# fails are they gone through one by one, for the message.

_TYPE = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
_I8, _I32, _F64, _BF = torch.int8, torch.int32, torch.float64, torch.bfloat16
_T16 = (torch.bfloat16, torch.float16)
_OUT = (torch.bfloat16, torch.float16, torch.float32)
_SCALE = (torch.float16, torch.int16, torch.uint16)
# torch.cuda.current_device() without its checks, and torch.cuda.current_stream(dev).cuda_stream without the object, where
# this torch has them (one built without CUDA has neither, and imports this module all the same)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _want(t, name: str, dtypes, dev, shape=None, contiguous: bool = True):
    """Raises what is wrong with t, a tensor of one of the dtypes on device index `dev`."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise TypeError(f"{name} must be a tensor on cuda:{dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _here(t, name: str) -> int:
    """The device index of t, which has to be the current one: the library launches there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _ok(t, dtype, dev, shape) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _pool_ok(k, v, ks, vs, dev) -> bool:
    shape, scales = k.shape, ks.shape
    return (k.dtype is _I8 and v.dtype is _I8 and ks.dtype in _SCALE and vs.dtype in _SCALE and len(shape) == 4
            and shape[2] == 64 and shape[3] == 128 and v.shape == shape and scales == shape[:3] and vs.shape == scales
            and k.get_device() == dev and v.get_device() == dev and ks.get_device() == dev and vs.get_device() == dev
            and k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous())


def _want_pool(k_pool, v_pool, k_scale, v_scale, dev):
    _want(k_pool, "k_pool", (_I8,), dev)
    shape = k_pool.shape
    if len(shape) != 4 or shape[2] != gen.PAGE_CELLS or shape[3] != gen.HEAD_DIM:
        raise ValueError(f"k_pool must be [n_ppages, n_kv, 64, 128], got {tuple(shape)}")
    _want(v_pool, "v_pool", (_I8,), dev, shape)
    _want(k_scale, "k_scale", _SCALE, dev, shape[:3])
    _want(v_scale, "v_scale", _SCALE, dev, shape[:3])


def _stream_of(stream, dev) -> int:
    if stream is None:
        return _raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor allocated here for a call on `stream`: on that stream, so that its memory is neither still in use by
    the current one nor handed out again before the call has run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_of(stream, device.index), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _status_of(dev_status, dev) -> int:
    if dev_status is None:
        return 0
    _want(dev_status, "dev_status", (_I32,), dev)
    return dev_status.data_ptr()


def paged_attn_workspace_bytes(n_kv: int, n_heads: int) -> int:
    """Bytes of workspace paged_attn needs for these head counts (whatever the lengths)."""
    return int(lib().qsa_paged_attn_workspace_bytes(int(n_kv), int(n_heads)))


def _refuse_paged_attn(q, k_pool, v_pool, k_scale, v_scale, page_tables, seq_lens, out, lse, workspace):
    dev = _here(q, "q")
    _want(q, "q", _T16, dev)
    _want_pool(k_pool, v_pool, k_scale, v_scale, dev)
    n_kv, shape = k_pool.shape[1], q.shape
    if len(shape) != 3 or shape[2] != gen.HEAD_DIM or n_kv == 0 or shape[1] == 0 or shape[1] % n_kv:
        raise ValueError(f"q must be [n_seq, n_heads, 128] with n_heads a multiple of {n_kv}, got {tuple(shape)}")
    _want(page_tables, "page_tables", (_I32,), dev)
    if page_tables.dim() != 2 or page_tables.shape[0] != shape[0]:
        raise ValueError(f"page_tables must be [{shape[0]}, n_lpages], got {tuple(page_tables.shape)}")
    _want(seq_lens, "seq_lens", (_I32,), dev, shape[:1])
    if out is not None:
        _want(out, "out", _OUT, dev, shape)
    if lse is not None:
        _want(lse, "lse", (torch.float32,), dev, shape[:2])
    if workspace is not None:
        _want(workspace, "workspace", (getattr(workspace, "dtype", None),), dev)


def paged_attn(q, k_pool, v_pool, k_scale, v_scale, page_tables, seq_lens, sm_scale: Optional[float] = None,
               window: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
               stream=None, n_lpages: Optional[int] = None) -> torch.Tensor:
    """One new token per sequence over its whole paged cache, or its last `window` cells (qsa_paged_attn):
    q BF16 or FP16 [n_seq, n_heads, 128], page_tables int32 [n_seq, width], seq_lens int32 [n_seq] -> out
    [n_seq, n_heads, 128] (float32 unless an `out` of another type is given); lse float32 [n_seq, n_heads] is
    written when given.  The first n_lpages entries of a table's row are in use (None: all); short sequences are
    fastest when that is no more than they need.  A workspace that is not given is allocated here; out must not be q."""
    try:
        dev, shape, tables, n_kv = q.get_device(), q.shape, page_tables.shape, k_pool.shape[1]
        good = (dev >= 0 and dev == _current() and q.dtype in _T16 and q.is_contiguous()
                and _pool_ok(k_pool, v_pool, k_scale, v_scale, dev)
                and len(shape) == 3 and shape[2] == 128 and shape[1] > 0 and n_kv > 0 and shape[1] % n_kv == 0
                and page_tables.dtype is _I32 and len(tables) == 2 and tables[0] == shape[0]
                and page_tables.get_device() == dev and page_tables.is_contiguous()
                and _ok(seq_lens, _I32, dev, shape[:1])
                and (out is None or (out.dtype in _OUT and _ok(out, out.dtype, dev, shape)))
                and (lse is None or _ok(lse, torch.float32, dev, shape[:2]))
                and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous())))
    except (AttributeError, IndexError):
        good = False
    if not good:
        _refuse_paged_attn(q, k_pool, v_pool, k_scale, v_scale, page_tables, seq_lens, out, lse, workspace)
        raise ValueError("paged_attn: arguments do not fit together")
    if out is None:
        out = _empty(shape, torch.float32, q.device, stream)
    if workspace is None:
        workspace = _empty(paged_attn_workspace_bytes(n_kv, shape[1]), torch.uint8, q.device, stream)
    rc = (_lib or lib()).qsa_paged_attn_packed(_PAGED_ARGS(
        q.data_ptr(), _TYPE[q.dtype], k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        page_tables.data_ptr(), tables[1], tables[1] if n_lpages is None else n_lpages, k_pool.shape[0], n_kv, shape[1],
        seq_lens.data_ptr(), shape[0], max(-1, min(window, 0x7FFFFFFF)),
        gen.HEAD_DIM ** -0.5 if sm_scale is None else sm_scale, out.data_ptr(), _TYPE[out.dtype],
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, _status_of(dev_status, dev),
        _stream_of(stream, dev)))
    if rc != QSA_OK:
        raise QsaError("qsa_paged_attn", rc)
    return out


def _rows_ok(t, dtype, dev, n_tok, n_heads, stride) -> bool:
    """A [n_tok, n_heads, 128] tensor whose tokens may lie apart (the heads of a token side by side)."""
    return (t.dtype is dtype and t.shape == (n_tok, n_heads, 128) and t.get_device() == dev
            and stride[2] == 1 and (stride[1] == 128 or n_heads == 1))


def _want_rows(t, name: str, dtypes, dev, n_tok=None, n_heads=None):
    _want(t, name, dtypes, dev, contiguous=False)
    shape = t.shape
    if len(shape) != 3 or shape[2] != gen.HEAD_DIM or (n_tok is not None and shape[0] != n_tok) or \
            (n_heads is not None and shape[1] != n_heads):
        raise ValueError(f"{name} must be [{'n_tok' if n_tok is None else n_tok}, "
                         f"{'n_heads' if n_heads is None else n_heads}, 128], got {tuple(shape)}")
    s = t.stride()
    if s[2] != 1 or (s[1] != gen.HEAD_DIM and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must lie side by side")


def _apart(stride, n_tok, n_heads) -> int:
    """Elements from one token to the next (a single token's stride says nothing)."""
    return stride[0] if n_tok > 1 else n_heads * 128


def _rotation_ok(positions, inv_freq, pair_axis, n_tok, dev) -> bool:
    if inv_freq is None:
        return True
    at, pairs = positions.shape, inv_freq.shape
    return (positions.dtype is _I32 and len(at) in (1, 2) and at[-1] == n_tok and positions.get_device() == dev
            and positions.is_contiguous() and len(pairs) == 1 and _ok(inv_freq, _F64, dev, pairs)
            and (pair_axis is None or _ok(pair_axis, _I32, dev, pairs)))


def _want_rotation(positions, inv_freq, pair_axis, n_tok, dev):
    if inv_freq is None:
        return
    _want(positions, "positions", (_I32,), dev)
    if positions.dim() not in (1, 2) or positions.shape[-1] != n_tok:
        raise ValueError(f"positions must be [n_axes, {n_tok}] or [{n_tok}], got {tuple(positions.shape)}")
    _want(inv_freq, "inv_freq", (_F64,), dev)
    if inv_freq.dim() != 1:
        raise ValueError(f"inv_freq must be [n_pairs], got {tuple(inv_freq.shape)}")
    if pair_axis is not None:
        _want(pair_axis, "pair_axis", (_I32,), dev, inv_freq.shape)


def _rotation(positions, inv_freq, pair_axis, n_tok):
    """(positions, n_axes, pos_stride, inv_freq, pair_axis, n_pairs) of a rotation; inv_freq None: none."""
    if inv_freq is None:
        return 0, 0, 0, 0, 0, 0
    at = positions.shape
    return (positions.data_ptr(), at[0] if len(at) == 2 else 1, n_tok, inv_freq.data_ptr(),
            0 if pair_axis is None else pair_axis.data_ptr(), inv_freq.shape[0])


def rope(x, positions, inv_freq, pair_axis: Optional[torch.Tensor] = None, interleaved: bool = False,
         out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotary positions with one or several axes (qsa_rope): x BF16 or FP16 [n_tok, n_heads, 128], positions int32
    [n_axes, n_tok] (or [n_tok]), inv_freq float64 [n_pairs], pair_axis int32 [n_pairs] (None: axis 0) -> out (may be x)."""
    dev = _here(x, "x")
    _want_rows(x, "x", _T16, dev)
    n_tok, n_heads = x.shape[0], x.shape[1]
    _want_rotation(positions, inv_freq, pair_axis, n_tok, dev)
    if out is None:
        out = _empty((n_tok, n_heads, gen.HEAD_DIM), x.dtype, x.device, stream)
    _want_rows(out, "out", (x.dtype,), dev, n_tok, n_heads)
    rc = lib().qsa_rope(x.data_ptr(), _apart(x.stride(), n_tok, n_heads), _TYPE[x.dtype],
                        *_rotation(positions, inv_freq, pair_axis, n_tok), bool(interleaved), out.data_ptr(),
                        _apart(out.stride(), n_tok, n_heads), n_heads, n_tok, _status_of(dev_status, dev),
                        _stream_of(stream, dev))
    if rc != QSA_OK:
        raise QsaError("qsa_rope", rc)
    return out


def _refuse_rope_append(q, k, v, positions, inv_freq, pair_axis, k_pool, v_pool, k_scale, v_scale, slots, q_out):
    dev = _here(k, "k")
    _want_rows(k, "k", _T16, dev)
    n_tok, n_kv = k.shape[0], k.shape[1]
    _want_rows(v, "v", (k.dtype,), dev, n_tok, n_kv)
    _want_pool(k_pool, v_pool, k_scale, v_scale, dev)
    if k_pool.shape[1] != n_kv:
        raise ValueError(f"k has {n_kv} heads, the cache {k_pool.shape[1]}")
    _want_rotation(positions, inv_freq, pair_axis, n_tok, dev)
    _want(slots, "slots", (_I32,), dev, (n_tok,))
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        return
    _want_rows(q, "q", (k.dtype,), dev, n_tok)
    if q_out is not None:
        _want_rows(q_out, "q_out", (k.dtype,), dev, n_tok, q.shape[1])


def rope_append(q, k, v, positions, inv_freq, pair_axis, k_pool, v_pool, k_scale, v_scale, slots,
                interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Rotates a step's queries and keys and writes keys and values to their slots of the cache as INT8 rows with FP16
    scales (qsa_rope_append): q [n_tok, n_heads, 128] (None: keys and values only), k and v [n_tok, n_kv, 128], all BF16
    or all FP16, tokens any multiple of 8 elements apart; positions, inv_freq, pair_axis as in rope (inv_freq None: no
    rotation); slots int32 [n_tok], < 0 = not written -> the rotated q (q_out, which may be q)."""
    try:
        dev, dtype, ks, vs = k.get_device(), k.dtype, k.stride(), v.stride()
        n_tok, n_kv = k.shape[0], k.shape[1]
        n_heads = 0
        good = (dev >= 0 and dev == _current() and dtype in _T16 and _rows_ok(k, dtype, dev, n_tok, n_kv, ks)
                and _rows_ok(v, dtype, dev, n_tok, n_kv, vs) and _pool_ok(k_pool, v_pool, k_scale, v_scale, dev)
                and k_pool.shape[1] == n_kv and _rotation_ok(positions, inv_freq, pair_axis, n_tok, dev)
                and _ok(slots, _I32, dev, (n_tok,)))
        if q is not None:
            n_heads, qs = q.shape[1], q.stride()
            good = (good and _rows_ok(q, dtype, dev, n_tok, n_heads, qs)
                    and (q_out is None or _rows_ok(q_out, dtype, dev, n_tok, n_heads, q_out.stride())))
        elif q_out is not None:
            good = False
    except (AttributeError, IndexError):
        good = False
    if not good:
        _refuse_rope_append(q, k, v, positions, inv_freq, pair_axis, k_pool, v_pool, k_scale, v_scale, slots, q_out)
        raise ValueError("rope_append: arguments do not fit together")
    qp = op = qs_ = os_ = 0
    if q is not None:
        if q_out is None:
            q_out = _empty((n_tok, n_heads, gen.HEAD_DIM), dtype, k.device, stream)
        qp, op, qs_, os_ = q.data_ptr(), q_out.data_ptr(), _apart(qs, n_tok, n_heads), _apart(q_out.stride(), n_tok, n_heads)
    rc = (_lib or lib()).qsa_rope_append_packed(_APPEND_ARGS(
        qp, qs_, k.data_ptr(), _apart(ks, n_tok, n_kv), v.data_ptr(), _apart(vs, n_tok, n_kv), _TYPE[dtype],
        *_rotation(positions, inv_freq, pair_axis, n_tok), bool(interleaved), op, os_, k_pool.data_ptr(), v_pool.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), slots.data_ptr(), k_pool.shape[0], n_heads, n_kv, n_tok,
        _status_of(dev_status, dev), _stream_of(stream, dev)))
    if rc != QSA_OK:
        raise QsaError("qsa_rope_append", rc)
    return q_out


def _refuse_cache_gather(k_pool, v_pool, k_scale, v_scale, slots, dtype, k_out, v_out):
    dev = _here(k_pool, "k_pool")
    _want_pool(k_pool, v_pool, k_scale, v_scale, dev)
    _want(slots, "slots", (_I32,), dev)
    if slots.dim() != 1:
        raise ValueError(f"slots must be [n_cell], got {tuple(slots.shape)}")
    shape = (slots.shape[0], k_pool.shape[1], gen.HEAD_DIM)
    if k_out is not None:
        _want(k_out, "k_out", _OUT, dev, shape)
    if v_out is not None:
        _want(v_out, "v_out", _OUT if k_out is None else (k_out.dtype,), dev, shape)
    if k_out is None and v_out is None and dtype not in _OUT:
        raise TypeError(f"dtype {dtype} is none of {_OUT}")


def cache_gather(k_pool, v_pool, k_scale, v_scale, slots, dtype: torch.dtype = torch.bfloat16,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                 dev_status: Optional[torch.Tensor] = None, stream=None):
    """Cells read back as the values they stand for (qsa_cache_gather): slots int32 [n_cell] -> (k, v)
    [n_cell, n_kv, 128] of `dtype`, or of the given outputs' type."""
    try:
        dev, cells, n_kv = k_pool.get_device(), slots.shape, k_pool.shape[1]
        shape = (cells[0], n_kv, 128)
        kind = dtype if k_out is None and v_out is None else v_out.dtype if k_out is None else k_out.dtype
        good = (dev >= 0 and dev == _current() and _pool_ok(k_pool, v_pool, k_scale, v_scale, dev) and len(cells) == 1
                and _ok(slots, _I32, dev, cells) and kind in _OUT
                and (k_out is None or _ok(k_out, kind, dev, shape)) and (v_out is None or _ok(v_out, kind, dev, shape)))
    except (AttributeError, IndexError):
        good = False
    if not good:
        _refuse_cache_gather(k_pool, v_pool, k_scale, v_scale, slots, dtype, k_out, v_out)
        raise ValueError("cache_gather: arguments do not fit together")
    if k_out is None:
        k_out = _empty(shape, kind, k_pool.device, stream)
    if v_out is None:
        v_out = _empty(shape, kind, k_pool.device, stream)
    rc = (_lib or lib()).qsa_cache_gather_packed(_GATHER_ARGS(
        k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), slots.data_ptr(), shape[0],
        k_pool.shape[0], n_kv, k_out.data_ptr(), v_out.data_ptr(), _TYPE[kind], _status_of(dev_status, dev),
        _stream_of(stream, dev)))
    if rc != QSA_OK:
        raise QsaError("qsa_cache_gather", rc)
    return k_out, v_out


class StepTables(NamedTuple):
    """What extend_tables writes beside the page tables (all int32)."""
    slots: torch.Tensor           # [n_tok] physical cell of each new token, -1 = none
    positions: torch.Tensor       # [n_tok] its cell in its sequence
    token_seq: torch.Tensor       # [n_tok] its sequence, -1 behind the last token
    seq_lens: torch.Tensor        # [n_seq] lengths after the step
    cu_tokens: torch.Tensor       # [n_seq + 1] first token of each sequence, then the total
    free_head: torch.Tensor       # [1] pages of the free list that are taken now


def _refuse_extend_tables(seq_lens, new_lens, page_tables, free_pages, n_tok, n_ppages, free_head, out):
    dev = _here(seq_lens, "seq_lens")
    if seq_lens.dim() != 1:
        raise ValueError(f"seq_lens must be [n_seq], got {tuple(seq_lens.shape)}")
    n_seq = seq_lens.shape[0]
    _want(seq_lens, "seq_lens", (_I32,), dev)
    _want(new_lens, "new_lens", (_I32,), dev, (n_seq,))
    _want(page_tables, "page_tables", (_I32,), dev)
    if page_tables.dim() != 2 or page_tables.shape[0] != n_seq:
        raise ValueError(f"page_tables must be [{n_seq}, n_lpages], got {tuple(page_tables.shape)}")
    if not (0 <= n_tok < 1 << 31 and 0 <= n_ppages < 1 << 31):
        raise ValueError("n_tok and n_ppages must be non-negative 32-bit numbers")
    _want(free_pages, "free_pages", (_I32,), dev)
    if free_head is not None:
        _want(free_head, "free_head", (_I32,), dev, (1,))
    for t, name, n in zip(out or (), StepTables._fields, (n_tok, n_tok, n_tok, n_seq, n_seq + 1, 1)):
        _want(t, f"out: {name}", (_I32,), dev, (n,))


def extend_tables(seq_lens, new_lens, page_tables, free_pages, n_tok: int, n_ppages: int,
                  free_head: Optional[torch.Tensor] = None, out=None, dev_status: Optional[torch.Tensor] = None,
                  stream=None) -> StepTables:
    """Page tables extended in place and slots mapped for a step's new tokens (qsa_extend_tables): seq_lens and new_lens
    int32 [n_seq], page_tables int32 [n_seq, n_lpages], free_pages int32 [n_free] of which *free_head are taken, n_tok =
    length of the token arrays (at least the new tokens of all sequences).  `out`: six tensors as in StepTables to reuse."""
    try:
        dev, lens, tables = seq_lens.get_device(), seq_lens.shape, page_tables.shape
        n_seq, toks = lens[0], (n_tok,)
        good = (dev >= 0 and dev == _current() and len(lens) == 1 and _ok(seq_lens, _I32, dev, lens)
                and _ok(new_lens, _I32, dev, lens) and len(tables) == 2 and tables[0] == n_seq
                and _ok(page_tables, _I32, dev, tables) and _ok(free_pages, _I32, dev, free_pages.shape)
                and (free_head is None or _ok(free_head, _I32, dev, (1,)))
                and 0 <= n_tok < 1 << 31 and 0 <= n_ppages < 1 << 31)
        if out is not None:
            slots, positions, token_seq, lens_out, cu, head_out = out
            good = (good and _ok(slots, _I32, dev, toks) and _ok(positions, _I32, dev, toks)
                    and _ok(token_seq, _I32, dev, toks) and _ok(lens_out, _I32, dev, lens)
                    and _ok(cu, _I32, dev, (n_seq + 1,)) and _ok(head_out, _I32, dev, (1,)))
    except (AttributeError, IndexError):
        good = False
    if not good:
        _refuse_extend_tables(seq_lens, new_lens, page_tables, free_pages, n_tok, n_ppages, free_head, out)
        raise ValueError("extend_tables: arguments do not fit together")
    if out is None:
        slots, positions, token_seq, lens_out, cu, head_out = (
            _empty(n, _I32, seq_lens.device, stream) for n in (n_tok, n_tok, n_tok, n_seq, n_seq + 1, 1))
    rc = (_lib or lib()).qsa_extend_tables_packed(_TABLES_ARGS(
        seq_lens.data_ptr(), new_lens.data_ptr(), n_seq, page_tables.data_ptr(), tables[1], tables[1], n_ppages,
        free_pages.data_ptr(), free_pages.numel(), 0 if free_head is None else free_head.data_ptr(), n_tok,
        slots.data_ptr(), positions.data_ptr(), token_seq.data_ptr(), lens_out.data_ptr(), cu.data_ptr(),
        head_out.data_ptr(), _status_of(dev_status, dev), _stream_of(stream, dev)))
    if rc != QSA_OK:
        raise QsaError("qsa_extend_tables", rc)
    return StepTables(slots, positions, token_seq, lens_out, cu, head_out)


def wait_selftest(limit_us: int, dev_status: torch.Tensor, stream=None) -> None:
    """qsa_wait_selftest: one bounded wait that runs out after limit_us and sets QSA_DEV_WAIT_TIMEOUT."""
    _dev(dev_status, "dev_status", (torch.int32,))
    _check("qsa_wait_selftest", lib().qsa_wait_selftest(int(limit_us), _ptr(dev_status), _stream(stream)))


STATIC_SCRATCH_BYTES = 32 << 20   # QSA_STATIC_SCRATCH_BYTES


def prompt_attn_static(q, k_pool, v_pool, k_scale, v_scale, page_table, sel, sel_count,
                       sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       union_stride: int = gen.UNION_STRIDE, variant: int = ATTN_DEFAULT,
                       dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """qsa_prompt_attn_static: the prompt-attention step over the library's static
    device scratch (no workspace, no allocation inside the call).  Only `out`, when
    not given, is allocated here, by the caller's side of the binding."""
    out = _attn_inputs(q, k_pool, v_pool, k_scale, v_scale, page_table, out)
    _dev(sel, "sel", (torch.int32,))
    _dev(sel_count, "sel_count", (torch.int32,))
    n_q, n_heads = int(q.shape[0]), int(q.shape[1])
    n_kv = n_heads // gen.HEADS_PER_KV
    if sm_scale is None:
        sm_scale = gen.HEAD_DIM ** -0.5
    rc = lib().qsa_prompt_attn_static(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
                                      _ptr(page_table), int(page_table.shape[0]), int(k_pool.shape[0]), n_kv,
                                      _ptr(sel), _ptr(sel_count), int(sel.shape[1]), n_q, float(sm_scale), _ptr(out),
                                      int(union_stride), int(variant), _ptr(dev_status), _stream(stream))
    _check("qsa_prompt_attn_static", rc)
    return out


def to_device(wl: "gen.Workload", device="cuda") -> dict:
    """Copy a generator workload's host arrays into device tensors (marshalling only)."""
    t = lambda a, dt=None: torch.from_numpy(a if dt is None else a.view(dt)).to(device)
    import numpy as np
    return dict(q=t(wl.q, np.int16), k_pool=t(wl.k_pool), v_pool=t(wl.v_pool),
                k_scale=t(wl.k_scale.view(np.int16)), v_scale=t(wl.v_scale.view(np.int16)),
                page_table=t(wl.page_table), sel=t(wl.sel), sel_count=t(wl.sel_count))


def decode_status(word: int) -> list:
    return [name for bit, name in DEV_BITS.items() if word & bit]
