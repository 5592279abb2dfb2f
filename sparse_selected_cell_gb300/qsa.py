"""Thin ctypes binding over libqsa.so (include/qsa.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
CPU fallback: when the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
import os
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
# tokens make these calls short, so the checks below are written out for speed:
# one device comparison per tensor, raw addresses into ctypes, no wrappers.

_TYPE = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
_I32 = torch.int32


def _want(t, name: str, dtype, dev, shape=None, contiguous: bool = True) -> int:
    """The address of t, a tensor of the given dtype (or one of several) on device `dev`."""
    if not isinstance(t, torch.Tensor) or t.device != dev:
        raise TypeError(f"{name} must be a tensor on {dev}")
    if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _here(t, name: str) -> torch.device:
    """The device of t, which has to be the current one: the library launches there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.device
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {dev}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _raw_stream(stream, dev) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)   # current_stream(dev).cuda_stream without the object
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _status_ptr(dev_status, dev) -> Optional[int]:
    return None if dev_status is None else _want(dev_status, "dev_status", _I32, dev)


_SCALE = (torch.float16, torch.int16, torch.uint16)


def _pool_ptrs(k_pool, v_pool, k_scale, v_scale, dev):
    """Addresses of the four arrays of a cache, then (n_ppages, n_kv)."""
    kp = _want(k_pool, "k_pool", torch.int8, dev)
    shape = k_pool.shape
    if len(shape) != 4 or shape[2] != gen.PAGE_CELLS or shape[3] != gen.HEAD_DIM:
        raise ValueError(f"k_pool must be [n_ppages, n_kv, 64, 128], got {tuple(shape)}")
    return (kp, _want(v_pool, "v_pool", torch.int8, dev, shape), _want(k_scale, "k_scale", _SCALE, dev, shape[:3]),
            _want(v_scale, "v_scale", _SCALE, dev, shape[:3]), shape[0], shape[1])


def paged_attn_workspace_bytes(n_kv: int, n_heads: int) -> int:
    """Bytes of workspace paged_attn needs for these head counts (whatever the lengths)."""
    return int(lib().qsa_paged_attn_workspace_bytes(int(n_kv), int(n_heads)))


def paged_attn(q, k_pool, v_pool, k_scale, v_scale, page_tables, seq_lens, sm_scale: Optional[float] = None,
               window: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """One new token per sequence over its whole paged cache, or its last `window` cells (qsa_paged_attn):
    q BF16 or FP16 [n_seq, n_heads, 128], page_tables int32 [n_seq, n_lpages], seq_lens int32 [n_seq] -> out
    [n_seq, n_heads, 128] (float32 unless an `out` of another type is given); lse float32 [n_seq, n_heads] is
    written when given.  A workspace that is not given is allocated here."""
    dev = _here(q, "q")
    qp = _want(q, "q", (torch.bfloat16, torch.float16), dev)
    kp, vp, ksp, vsp, n_ppages, n_kv = _pool_ptrs(k_pool, v_pool, k_scale, v_scale, dev)
    shape = q.shape
    if len(shape) != 3 or shape[2] != gen.HEAD_DIM or n_kv == 0 or shape[1] == 0 or shape[1] % n_kv:
        raise ValueError(f"q must be [n_seq, n_heads, 128] with n_heads a multiple of {n_kv}, got {tuple(shape)}")
    n_seq, n_heads = shape[0], shape[1]
    tp = _want(page_tables, "page_tables", _I32, dev)
    if page_tables.dim() != 2 or page_tables.shape[0] != n_seq:
        raise ValueError(f"page_tables must be [{n_seq}, n_lpages], got {tuple(page_tables.shape)}")
    width = page_tables.shape[1]
    lp = _want(seq_lens, "seq_lens", _I32, dev, (n_seq,))
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=dev)
    op = _want(out, "out", (torch.float32, torch.bfloat16, torch.float16), dev, shape)
    sp = None if lse is None else _want(lse, "lse", torch.float32, dev, (n_seq, n_heads))
    if workspace is None:
        workspace = torch.empty(paged_attn_workspace_bytes(n_kv, n_heads), dtype=torch.uint8, device=dev)
    wp = _want(workspace, "workspace", workspace.dtype, dev)
    rc = lib().qsa_paged_attn(qp, _TYPE[q.dtype], kp, vp, ksp, vsp, tp, width, width, n_ppages, n_kv, n_heads, lp, n_seq,
                              min(int(window), 0x7FFFFFFF), gen.HEAD_DIM ** -0.5 if sm_scale is None else sm_scale, op,
                              _TYPE[out.dtype], sp, wp, workspace.nbytes, _status_ptr(dev_status, dev),
                              _raw_stream(stream, dev))
    if rc != QSA_OK:
        raise QsaError("qsa_paged_attn", rc)
    return out


def _rows(t, name: str, dtype, dev, n_tok=None, n_heads=None):
    """Address and token stride of a [n_tok, n_heads, 128] tensor whose tokens may lie apart."""
    p = _want(t, name, dtype, dev, contiguous=False)
    shape = t.shape
    if len(shape) != 3 or shape[2] != gen.HEAD_DIM or (n_tok is not None and shape[0] != n_tok) or \
            (n_heads is not None and shape[1] != n_heads):
        raise ValueError(f"{name} must be [{n_tok or 'n_tok'}, {n_heads or 'n_heads'}, 128], got {tuple(shape)}")
    s = t.stride()
    if s[2] != 1 or (s[1] != gen.HEAD_DIM and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must lie side by side")
    return p, s[0] if shape[0] > 1 else shape[1] * gen.HEAD_DIM


def _rotation(positions, inv_freq, pair_axis, n_tok, dev):
    """(positions, n_axes, pos_stride, inv_freq, pair_axis, n_pairs) of a rotation; inv_freq None: none."""
    if inv_freq is None:
        return None, 0, 0, None, None, 0
    pp = _want(positions, "positions", _I32, dev)
    if positions.dim() not in (1, 2) or positions.shape[-1] != n_tok:
        raise ValueError(f"positions must be [n_axes, {n_tok}] or [{n_tok}], got {tuple(positions.shape)}")
    n_pairs = inv_freq.numel()
    fp = _want(inv_freq, "inv_freq", torch.float64, dev, (n_pairs,))
    ap = None if pair_axis is None else _want(pair_axis, "pair_axis", _I32, dev, (n_pairs,))
    return pp, positions.shape[0] if positions.dim() == 2 else 1, n_tok, fp, ap, n_pairs


def rope(x, positions, inv_freq, pair_axis: Optional[torch.Tensor] = None, interleaved: bool = False,
         out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rotary positions with one or several axes (qsa_rope): x BF16 or FP16 [n_tok, n_heads, 128], positions int32
    [n_axes, n_tok] (or [n_tok]), inv_freq float64 [n_pairs], pair_axis int32 [n_pairs] (None: axis 0) -> out (may be x)."""
    dev = _here(x, "x")
    xp, xs = _rows(x, "x", (torch.bfloat16, torch.float16), dev)
    n_tok, n_heads = x.shape[0], x.shape[1]
    rot = _rotation(positions, inv_freq, pair_axis, n_tok, dev)
    if out is None:
        out = torch.empty((n_tok, n_heads, gen.HEAD_DIM), dtype=x.dtype, device=dev)
    op, os_ = _rows(out, "out", x.dtype, dev, n_tok, n_heads)
    rc = lib().qsa_rope(xp, xs, _TYPE[x.dtype], *rot, bool(interleaved), op, os_, n_heads, n_tok,
                        _status_ptr(dev_status, dev), _raw_stream(stream, dev))
    if rc != QSA_OK:
        raise QsaError("qsa_rope", rc)
    return out


def rope_append(q, k, v, positions, inv_freq, pair_axis, k_pool, v_pool, k_scale, v_scale, slots,
                interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Rotates a step's queries and keys and writes keys and values to their slots of the cache as INT8 rows with FP16
    scales (qsa_rope_append): q [n_tok, n_heads, 128] (None: keys and values only), k and v [n_tok, n_kv, 128], all BF16
    or all FP16, tokens any multiple of 8 elements apart; positions, inv_freq, pair_axis as in rope (inv_freq None: no
    rotation); slots int32 [n_tok], < 0 = not written -> the rotated q (q_out, which may be q)."""
    dev = _here(k, "k")
    kp_, ks_ = _rows(k, "k", (torch.bfloat16, torch.float16), dev)
    n_tok, n_kv, dtype = k.shape[0], k.shape[1], k.dtype
    vp_, vs_ = _rows(v, "v", dtype, dev, n_tok, n_kv)
    kp, vp, ksp, vsp, n_ppages, pool_kv = _pool_ptrs(k_pool, v_pool, k_scale, v_scale, dev)
    if pool_kv != n_kv:
        raise ValueError(f"k has {n_kv} heads, the cache {pool_kv}")
    rot = _rotation(positions, inv_freq, pair_axis, n_tok, dev)
    sp = _want(slots, "slots", _I32, dev, (n_tok,))
    qp = op = None
    qs = os_ = n_heads = 0
    if q is not None:
        qp, qs = _rows(q, "q", dtype, dev, n_tok)
        n_heads = q.shape[1]
        if q_out is None:
            q_out = torch.empty((n_tok, n_heads, gen.HEAD_DIM), dtype=dtype, device=dev)
        op, os_ = _rows(q_out, "q_out", dtype, dev, n_tok, n_heads)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rc = lib().qsa_rope_append(qp, qs, kp_, ks_, vp_, vs_, _TYPE[dtype], *rot, bool(interleaved), op, os_, kp, vp, ksp,
                               vsp, sp, n_ppages, n_heads, n_kv, n_tok, _status_ptr(dev_status, dev),
                               _raw_stream(stream, dev))
    if rc != QSA_OK:
        raise QsaError("qsa_rope_append", rc)
    return q_out


def cache_gather(k_pool, v_pool, k_scale, v_scale, slots, dtype: torch.dtype = torch.bfloat16,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                 dev_status: Optional[torch.Tensor] = None, stream=None):
    """Cells read back as the values they stand for (qsa_cache_gather): slots int32 [n_cell] -> (k, v)
    [n_cell, n_kv, 128] of `dtype`, or of the given outputs' type."""
    dev = _here(k_pool, "k_pool")
    kp, vp, ksp, vsp, n_ppages, n_kv = _pool_ptrs(k_pool, v_pool, k_scale, v_scale, dev)
    sp = _want(slots, "slots", _I32, dev)
    if slots.dim() != 1:
        raise ValueError(f"slots must be [n_cell], got {tuple(slots.shape)}")
    shape = (slots.shape[0], n_kv, gen.HEAD_DIM)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype if v_out is None else v_out.dtype, device=dev)
    if v_out is None:
        v_out = torch.empty(shape, dtype=k_out.dtype, device=dev)
    ko = _want(k_out, "k_out", (torch.bfloat16, torch.float16, torch.float32), dev, shape)
    vo = _want(v_out, "v_out", k_out.dtype, dev, shape)
    rc = lib().qsa_cache_gather(kp, vp, ksp, vsp, sp, shape[0], n_ppages, n_kv, ko, vo, _TYPE[k_out.dtype],
                                _status_ptr(dev_status, dev), _raw_stream(stream, dev))
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


def extend_tables(seq_lens, new_lens, page_tables, free_pages, n_tok: int, n_ppages: int,
                  free_head: Optional[torch.Tensor] = None, out=None, dev_status: Optional[torch.Tensor] = None,
                  stream=None) -> StepTables:
    """Page tables extended in place and slots mapped for a step's new tokens (qsa_extend_tables): seq_lens and new_lens
    int32 [n_seq], page_tables int32 [n_seq, n_lpages], free_pages int32 [n_free] of which *free_head are taken, n_tok =
    length of the token arrays (at least the new tokens of all sequences).  `out`: six tensors as in StepTables to reuse."""
    dev = _here(seq_lens, "seq_lens")
    n_seq = seq_lens.shape[0]
    sl, nl = _want(seq_lens, "seq_lens", _I32, dev, (n_seq,)), _want(new_lens, "new_lens", _I32, dev, (n_seq,))
    tp = _want(page_tables, "page_tables", _I32, dev)
    if page_tables.dim() != 2 or page_tables.shape[0] != n_seq:
        raise ValueError(f"page_tables must be [{n_seq}, n_lpages], got {tuple(page_tables.shape)}")
    width = page_tables.shape[1]
    if not (0 <= n_tok < 1 << 31 and 0 <= n_ppages < 1 << 31):
        raise ValueError("n_tok and n_ppages must be non-negative 32-bit numbers")
    fp = _want(free_pages, "free_pages", _I32, dev)
    if out is None:
        out = [torch.empty(n, dtype=_I32, device=dev) for n in (n_tok, n_tok, n_tok, n_seq, n_seq + 1, 1)]
    slots, positions, token_seq, lens_out, cu, head_out = out
    rc = lib().qsa_extend_tables(
        sl, nl, n_seq, tp, width, width, n_ppages, fp, free_pages.numel(),
        None if free_head is None else _want(free_head, "free_head", _I32, dev, (1,)), n_tok,
        _want(slots, "slots", _I32, dev, (n_tok,)), _want(positions, "positions", _I32, dev, (n_tok,)),
        _want(token_seq, "token_seq", _I32, dev, (n_tok,)), _want(lens_out, "seq_lens_out", _I32, dev, (n_seq,)),
        _want(cu, "cu_tokens", _I32, dev, (n_seq + 1,)), _want(head_out, "free_head_out", _I32, dev, (1,)),
        _status_ptr(dev_status, dev), _raw_stream(stream, dev))
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
