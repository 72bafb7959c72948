"""GB300 (sm_103a) scaled dot-product attention forward: Python binding.

This module only marshals arguments to the C ABI declared in include/attn.h
(``libattn.so`` next to this file): every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and streams.  There is
no CPU path: when the library is missing, every call raises.

    attn_fwd(q, k, v, out=None, scale=None, causal=False, kv_len=None, stream=None)
    attn_fwd_packed(q, k, v, cu_seqlens, scale=None, causal=False, return_lse=False, ...)
    attn_rope(q, k, positions, freqs, ...), attn_rope_append(q, k, v, kcache, vcache, freqs, ...)
    attn_fwd_paged(q, kpages, vpages, page_table, cache_len, ...), attn_rope_append_paged(...), attn_norm_rope(...)
    attn_pages_step(page_table, cache_len, n_pages, page_size, ...), attn_pages_compact(...), attn_pages_copy(...)
    attn_decode(q, kcache, vcache, out=None, kv_len=None, stream=None)
    attn_decode_tree(q, kcache, vcache, parents, cache_len=None, draft_len=None, ...)
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
from typing import Optional

ATTN_F32 = 0
ATTN_BF16 = 1

ATTN_OK = 0
ATTN_EINVAL = -1
ATTN_EUNSUPPORTED = -2
ATTN_ECUDA = -3
ATTN_ENOMEM = -4
ATTN_ETIMEOUT = -5
ATTN_ECONFLICT = -6

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn.so")

# The exported functions, as declared in include/attn.h: name -> (restype, argtypes)
_vp, _i, _f, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
SIGNATURES = {
    "attn_fwd": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _i, _vp]),
    "attn_fwd_gqa": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _i, _vp]),
    "attn_fwd_chunked": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _i, _vp]),
    "attn_fwd_host": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _i, _vp]),
    "attn_fwd_debug": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _i, _vp]),
    "attn_decode": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _vp]),
    "attn_decode_gqa": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _i, _vp]),
    "attn_decode_noalloc": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _vp]),
    "attn_decode_splits": (_i, [_i, _i, _i, _i]),
    "attn_fwd_packed": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _i, _f, _i, _i, _vp, _ll, _vp]),
    "attn_fwd_packed_workspace": (_ll, [_i, _i, _i, _i, _i]),
    "attn_decode_tree": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _f, _i, _vp, _ll, _vp]),
    "attn_decode_tree_workspace": (_ll, [_i, _i, _i, _i, _i, _i, _i]),
    "attn_fwd_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _i, _vp, _i, _ll, _vp, _vp, _i, _f, _i, _vp, _ll,
                            _vp]),
    "attn_fwd_paged_workspace": (_ll, [_i, _i, _i, _i, _i, _i, _i, _i, _i]),
    "attn_rope": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _i, _i, _i, _f, _i, _vp]),
    "attn_rope_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _i, _vp, _vp, _vp, _vp,
                              _i, _i, _f, _i, _vp]),
    "attn_norm_rope": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _i, _i, _f, _vp, _vp, _f, _i, _vp]),
    "attn_rope_append_paged": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _i, _vp, _i, _ll, _vp, _vp, _i,
                                    _vp, _vp, _i, _i, _f, _vp, _vp, _f, _i, _vp]),
    "attn_pages_step": (_i, [_vp, _vp, _i, _i, _ll, _i, _i, _vp, _vp, _vp, _i, _vp, _ll, _vp, _vp, _vp, _vp, _ll, _vp]),
    "attn_pages_compact": (_i, [_vp, _vp, _i, _i, _ll, _i, _i, _vp, _vp, _ll, _vp, _vp, _vp, _ll, _vp]),
    "attn_pages_copy": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _i, _i, _vp]),
    "attn_pages_workspace": (_ll, [_i, _i]),
    "attn_device_status": (_i, [_vp]),
    "attn_last_error": (ctypes.c_char_p, []),
    "attn_release": (None, []),
    "attn_selftest_wait_timeout": (_i, [ctypes.c_longlong, _vp]),
}

_lib = None


class AttnError(RuntimeError):
    """A non-zero status from the library; ``code`` is the ATTN_E* value."""

    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code


def lib(path: Optional[str] = None):
    """The loaded C library (ctypes handle with typed signatures)."""
    global _lib
    if path is not None:
        return _bind(ctypes.CDLL(path))
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m transformer_scaled_dot_fwd_gb300.build`")
        _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


def _bind(handle):
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


def attn_last_error() -> str:
    return (lib().attn_last_error() or b"").decode(errors="replace")


def _check(rc: int):
    if rc != ATTN_OK:
        raise AttnError(rc, attn_last_error())


def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    if t.dtype == torch.float32:
        return ATTN_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check_tensor(name, t, ndim):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")


def _kv_len_arg(kv_len, B, device):
    torch = _torch()
    if kv_len is None:
        return None
    if not (kv_len.is_cuda and kv_len.dtype == torch.int32 and kv_len.shape == (B,)
            and kv_len.is_contiguous() and kv_len.device == device):
        raise ValueError("kv_len must be a contiguous int32 CUDA tensor of shape (B,) on q's device")
    return kv_len


def attn_fwd(q, k, v, out=None, scale: Optional[float] = None, causal: bool = False,
             kv_len=None, stream=None):
    """Prefill attention of (B, H, Sq, D) queries against (B, H_kv, Skv, D)
    keys/values, H_kv dividing H (H_kv < H: grouped-query attention, calls
    attn_fwd_gqa).

    Returns ``out`` (allocated like q when not given).  See include/attn.h.
    """
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, 4)
    B, H, Sq, D = q.shape
    H_kv, Skv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, H_kv, Skv, D) or tuple(v.shape) != (B, H_kv, Skv, D) or H % H_kv:
        raise ValueError("k and v must be (B, H_kv, Skv, D) matching q, with H_kv dividing H")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    if out is None:
        out = _torch().empty_like(q)
    _check_tensor("out", out, 4)
    if tuple(out.shape) != tuple(q.shape) or out.dtype != q.dtype:
        raise ValueError("out must match q's shape and dtype")
    kl = _kv_len_arg(kv_len, B, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if H_kv == H:
        rc = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, Sq, Skv, D, float(scale),
                            int(bool(causal)), _ptr(kl), _dtype_code(q), _stream_handle(stream))
    else:
        rc = lib().attn_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, H_kv, Sq, Skv, D,
                                float(scale), int(bool(causal)), _ptr(kl), _dtype_code(q),
                                _stream_handle(stream))
    _check(rc)
    return out


def attn_fwd_host(q, k, v, out=None, scale: Optional[float] = None, causal: bool = False,
                  kv_len=None, stream=None):
    """attn_fwd with q, k, v, out in host memory (contiguous CPU tensors; pinned
    ones copy fastest): the library copies each chunk of heads in, computes it
    and copies it out, overlapping the three.  kv_len is a CPU int32 tensor of
    shape (B,) or a sequence of B ints.  Returns ``out`` (allocated like q,
    pinned if q is, when not given) once it holds the result.  See
    include/attn.h.
    """
    torch = _torch()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous 4-D CPU tensor")
    B, H, Sq, D = q.shape
    H_kv, Skv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, H_kv, Skv, D) or tuple(v.shape) != (B, H_kv, Skv, D) or H % H_kv:
        raise ValueError("k and v must be (B, H_kv, Skv, D) matching q, with H_kv dividing H")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=q.is_pinned())
    if out.is_cuda or not out.is_contiguous() or tuple(out.shape) != tuple(q.shape) or out.dtype != q.dtype:
        raise ValueError("out must be a contiguous CPU tensor matching q")
    kl = None
    if kv_len is not None:
        kl = torch.as_tensor(kv_len, dtype=torch.int32).contiguous()
        if kl.is_cuda or tuple(kl.shape) != (B,):
            raise ValueError("kv_len must be B ints on the host")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    rc = lib().attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, H_kv, Sq, Skv, D, float(scale),
                             int(bool(causal)), _ptr(kl), _dtype_code(q), _stream_handle(stream))
    _check(rc)
    return out


def attn_fwd_chunked(q, kcache, vcache, out=None, lse=None, scale: Optional[float] = None,
                     cache_len=None, return_lse: bool = False, stream=None):
    """Prefill of a chunk of (B, H, Sq, D) queries against a (B, H_kv, Skv, D)
    KV cache whose last positions hold the chunk's own keys/values: query i
    of sequence b sits at position cache_len[b] - Sq + i (causal).  Returns
    ``out``, or ``(out, lse)`` with the (B, H, Sq) fp32 log-sum-exp when
    ``return_lse`` (or an ``lse`` tensor) is given.  See include/attn.h.
    """
    for name, t in (("q", q), ("kcache", kcache), ("vcache", vcache)):
        _check_tensor(name, t, 4)
    B, H, Sq, D = q.shape
    H_kv, Skv = kcache.shape[1], kcache.shape[2]
    if (tuple(kcache.shape) != (B, H_kv, Skv, D) or tuple(vcache.shape) != (B, H_kv, Skv, D)
            or H % H_kv):
        raise ValueError("kcache and vcache must be (B, H_kv, Skv, D) matching q, with H_kv dividing H")
    if not (q.dtype == kcache.dtype == vcache.dtype):
        raise TypeError("q, kcache, vcache must share one dtype")
    torch = _torch()
    if out is None:
        out = torch.empty_like(q)
    _check_tensor("out", out, 4)
    if lse is None and return_lse:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check_tensor("lse", lse, 3)
        if tuple(lse.shape) != (B, H, Sq) or lse.dtype != torch.float32:
            raise ValueError("lse must be a float32 (B, H, Sq) tensor")
    cl = _kv_len_arg(cache_len, B, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    rc = lib().attn_fwd_chunked(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(out), _ptr(lse), B, H, H_kv,
                                Sq, Skv, D, float(scale), _ptr(cl), _dtype_code(q), _stream_handle(stream))
    _check(rc)
    return (out, lse) if lse is not None else out


def attn_fwd_debug(q, k, v, out=None, weights=None, scale: Optional[float] = None, causal: bool = False,
                   kv_len=None, return_weights: bool = False, stream=None):
    """General attention for inspection: q (B, H, Sq, Dk), k (B, H_kv, Skv, Dk),
    v (B, H_kv, Skv, Dv); returns out (B, H, Sq, Dv), or (out, weights) with
    the (B, H, Sq, Skv) fp32 attention weights.  See include/attn.h."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, 4)
    B, H, Sq, Dk = q.shape
    H_kv, Skv, Dv = k.shape[1], k.shape[2], v.shape[3]
    if tuple(k.shape) != (B, H_kv, Skv, Dk) or tuple(v.shape[:3]) != (B, H_kv, Skv) or H % H_kv:
        raise ValueError("k must be (B, H_kv, Skv, Dk) and v (B, H_kv, Skv, Dv), with H_kv dividing H")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    torch = _torch()
    if out is None:
        out = torch.empty((B, H, Sq, Dv), dtype=q.dtype, device=q.device)
    _check_tensor("out", out, 4)
    if weights is None and return_weights:
        weights = torch.empty((B, H, Sq, Skv), dtype=torch.float32, device=q.device)
    if weights is not None:
        _check_tensor("weights", weights, 4)
    kl = _kv_len_arg(kv_len, B, q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(Dk)
    rc = lib().attn_fwd_debug(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(weights), B, H, H_kv, Sq, Skv,
                              Dk, Dv, float(scale), int(bool(causal)), _ptr(kl), _dtype_code(q),
                              _stream_handle(stream))
    _check(rc)
    return (out, weights) if weights is not None else out


def attn_decode(q, kcache, vcache, out=None, kv_len=None, stream=None):
    """One query per (batch, head): q (B, H, D) against a (B, H_kv, Skv, D)
    cache, H_kv dividing H (H_kv < H: grouped-query decode, attn_decode_gqa).

    Returns ``out`` (B, H, D).  See include/attn.h.
    """
    _check_tensor("q", q, 3)
    _check_tensor("kcache", kcache, 4)
    _check_tensor("vcache", vcache, 4)
    B, H, D = q.shape
    H_kv, Skv = kcache.shape[1], kcache.shape[2]
    if (tuple(kcache.shape) != (B, H_kv, Skv, D) or tuple(vcache.shape) != (B, H_kv, Skv, D)
            or H % H_kv):
        raise ValueError("kcache and vcache must be (B, H_kv, Skv, D) matching q, with H_kv dividing H")
    if not (q.dtype == kcache.dtype == vcache.dtype):
        raise TypeError("q, kcache, vcache must share one dtype")
    if out is None:
        out = _torch().empty_like(q)
    _check_tensor("out", out, 3)
    kl = _kv_len_arg(kv_len, B, q.device)
    if H_kv == H:
        rc = lib().attn_decode(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(out), B, H, Skv, D, _ptr(kl),
                               _dtype_code(q), _stream_handle(stream))
    else:
        rc = lib().attn_decode_gqa(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(out), B, H, H_kv, Skv, D,
                                   _ptr(kl), _dtype_code(q), _stream_handle(stream))
    _check(rc)
    return out


def attn_decode_noalloc(q, kcache, vcache, out, kv_len=None, stream=None):
    """attn_decode without any device allocation (see include/attn.h): the
    caller supplies ``out``; the scratch is a fixed array inside the library."""
    _check_tensor("q", q, 3)
    _check_tensor("kcache", kcache, 4)
    _check_tensor("vcache", vcache, 4)
    _check_tensor("out", out, 3)
    B, H, D = q.shape
    Skv = kcache.shape[2]
    if tuple(kcache.shape) != (B, H, Skv, D) or tuple(vcache.shape) != (B, H, Skv, D):
        raise ValueError("kcache and vcache must be (B, H, Skv, D) matching q")
    if tuple(out.shape) != (B, H, D) or not (q.dtype == kcache.dtype == vcache.dtype == out.dtype):
        raise ValueError("out must be (B, H, D) and every tensor must share q's dtype")
    kl = _kv_len_arg(kv_len, B, q.device)
    rc = lib().attn_decode_noalloc(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(out), B, H, Skv, D, _ptr(kl),
                                   _dtype_code(q), _stream_handle(stream))
    _check(rc)
    return out


def attn_decode_splits(B: int, H: int, Skv: int, D: int) -> int:
    return lib().attn_decode_splits(B, H, Skv, D)


# The serving entry points below are called once per layer and token, so the usual
# call, whose arguments are all in order and on the current device and stream, goes
# through the compiled binding.  It answers None for any other, and the Python
# below refuses that one with its reason or runs it.  A call for another device or stream
# than the current one re-enters with that one current: outputs and
# workspaces then belong to the stream the work runs on, and the caching
# allocator orders their reuse with it.

_native = None


class _NoBinding:
    """Stands for a binding that is not there: leaves every call to the checked path."""

    def _none(self, *args):
        return None

    packed = rope = rope_append = tree = paged = norm_rope = append_paged = _none
    pages_step = pages_compact = pages_copy = _none


def _load_native():
    """The compiled binding (csrc/binding.cpp), with the library's functions bound."""
    global _native
    import importlib.util
    import warnings
    handle = lib()
    path = os.path.join(_HERE, f"_binding.torch{_torch().__version__}.so")
    try:
        spec = importlib.util.spec_from_file_location(__name__ + "._binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"no compiled binding for this torch ({e}): the serving entry points take their checked path, some "
                      "10 us more a call; run `python -m transformer_scaled_dot_fwd_gb300.build`", RuntimeWarning)
        _native = _NoBinding()
        return _native
    module.bind(*(ctypes.cast(getattr(handle, name), ctypes.c_void_p).value for name in (
        "attn_fwd_packed", "attn_fwd_packed_workspace", "attn_rope", "attn_rope_append", "attn_decode_tree",
        "attn_decode_tree_workspace")))
    module.bind_paged(*(ctypes.cast(getattr(handle, name), ctypes.c_void_p).value for name in (
        "attn_fwd_paged", "attn_fwd_paged_workspace", "attn_norm_rope", "attn_rope_append_paged",
        "attn_pages_step", "attn_pages_compact", "attn_pages_copy", "attn_pages_workspace")))
    _native = module
    return module


def _elsewhere(device, stream):
    """Context to re-enter a call in when device or stream are not current."""
    torch = _torch()
    if stream is None:
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream must be on q's device {device} (it is on {stream.device})")
    return torch.cuda.stream(stream)


def _current(device):
    """cudaStream_t of the device's current stream."""
    return _torch().cuda.current_stream(device).cuda_stream


def _scale(scale, D):
    """The default, 1 / sqrt(D), where none is given (a D of 0 is the library's to refuse)."""
    return scale if scale is not None else 1.0 / math.sqrt(D) if D else 1.0


def _workspace(nbytes, device):
    """``nbytes`` of device memory for one call on the device's current stream, given
    back with the last reference: the allocator reuses it in stream order."""
    return _torch().empty(nbytes, dtype=_torch().uint8, device=device) if nbytes > 0 else None


def _rows(name, t, T, D, dtype, device):
    """(heads, token stride, head stride) of a (T, heads, D) tensor whose head rows
    are contiguous."""
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or st[2] != 1 or shape[0] != T or shape[2] != D:
        raise ValueError(f"{name} must be ({T}, heads, {D}) with contiguous rows of {D} elements (got {tuple(shape)})")
    if t.dtype != dtype:
        raise TypeError(f"{name} must share q's dtype {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on q's device {device}")
    return shape[1], st[0], st[1]


def _out_rows(name, t, T, heads, D, dtype, device):
    """(tensor, token stride, head stride) of a (T, heads, D) output, made when not given."""
    if t is None:
        return _torch().empty((T, heads, D), dtype=dtype, device=device), heads * D, D
    given, ts, hs = _rows(name, t, T, D, dtype, device)
    if given != heads:
        raise ValueError(f"{name} must be ({T}, {heads}, {D}) (got {tuple(t.shape)})")
    return t, ts, hs


def _first(q, ndim):
    """(shape, strides, dtype code, device) of a call's q."""
    shape, st = q.shape, q.stride()
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if len(shape) != ndim or st[-1] != 1:
        raise ValueError(f"q must be {ndim}-D with contiguous rows of D elements")
    return shape, st, _dtype_code(q), q.device


def _ints(name, t, shape, device):
    """data_ptr of an optional int32 tensor."""
    if t is None:
        return None
    if not (t.dtype == _torch().int32 and t.device == device and t.shape == shape and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on q's device")
    return t.data_ptr()


def _caches(kcache, vcache, dtype, device, D):
    """(B, H_kv, Skv) of a pair of contiguous caches."""
    shape = kcache.shape
    if len(shape) != 4 or vcache.shape != shape or shape[3] != D:
        raise ValueError(f"kcache and vcache must be (B, H_kv, Skv, {D})")
    if kcache.dtype != dtype or vcache.dtype != dtype:
        raise TypeError("q, kcache, vcache must share one dtype")
    if kcache.device != device or vcache.device != device:
        raise ValueError("the caches must be on q's device")
    if not (kcache.is_contiguous() and vcache.is_contiguous()):
        raise ValueError("kcache and vcache must be contiguous")
    return shape[0], shape[1], shape[2]


def _freqs_arg(freqs, D):
    torch = _torch()
    if not (isinstance(freqs, torch.Tensor) and freqs.dtype == torch.float64 and freqs.dim() == 1
            and not freqs.is_cuda and freqs.is_contiguous()) or 2 * freqs.shape[0] > D:
        raise ValueError("freqs must be a contiguous 1-D float64 CPU tensor of rotary_dim / 2 <= D / 2 values")
    return freqs.data_ptr(), 2 * freqs.shape[0]


# host int64 arrays of strides (a bytes object serves as the pointer)
_LL6, _LL8, _LL10, _LL16 = (struct.Struct(f"{n}q").pack for n in (6, 8, 10, 16))


@functools.lru_cache(maxsize=4096)
def _packed_workspace(T, n_seq, H, H_kv, dtype):
    return lib().attn_fwd_packed_workspace(T, n_seq, H, H_kv, dtype)


@functools.lru_cache(maxsize=4096)
def _tree_workspace(B, H, H_kv, T, Skv, D, dtype, device):
    return lib().attn_decode_tree_workspace(B, H, H_kv, T, Skv, D, dtype)


def attn_fwd_packed(q, k, v, cu_seqlens, out=None, lse=None, scale: Optional[float] = None, causal: bool = False,
                    return_lse: bool = False, stream=None):
    """Prefill attention of packed sequences: q (T, H, D), k and v (T, H_kv, D),
    sequence s being tokens [cu_seqlens[s], cu_seqlens[s + 1]) (int32, on the
    device).  Rows may be strided (slices of a fused projection).  Returns
    ``out`` (T, H, D), or ``(out, lse)`` with the (T, H) fp32 log-sum-exp when
    ``return_lse`` (or an ``lse`` tensor) is given.  Rows outside every sequence
    are not written.  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).packed(q, k, v, cu_seqlens, out, lse, scale, causal, return_lse)
        if done is not None:
            return done
    torch = _torch()
    (T, H, D), sq, code, device = _first(q, 3)
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_fwd_packed(q, k, v, cu_seqlens, out, lse, scale, causal, return_lse)
    dtype = q.dtype
    H_kv, kt, kh = _rows("k", k, T, D, dtype, device)
    Hv, vt, vh = _rows("v", v, T, D, dtype, device)
    if Hv != H_kv or H_kv < 1 or H % H_kv:
        raise ValueError("k and v must be (T, H_kv, D) matching q, with H_kv dividing H")
    if cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be 1-D with at least one value")
    n_seq = cu_seqlens.shape[0] - 1
    cu = _ints("cu_seqlens", cu_seqlens, (n_seq + 1,), device)
    out, ot, oh = _out_rows("out", out, T, H, D, dtype, device)
    if lse is None:
        if return_lse:
            lse = torch.empty((T, H), dtype=torch.float32, device=device)
    elif not (lse.dtype == torch.float32 and lse.shape == (T, H) and lse.is_contiguous() and lse.device == device):
        raise ValueError("lse must be a contiguous float32 (T, H) tensor on q's device")
    need = _packed_workspace(T, n_seq, H, H_kv, code)
    ws = _workspace(need, device)
    rc = lib().attn_fwd_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                               None if lse is None else lse.data_ptr(), T, H, H_kv, D,
                               _LL8(sq[0], sq[1], kt, kh, vt, vh, ot, oh), cu, n_seq, _scale(scale, D),
                               1 if causal else 0, code, _ptr(ws), need, _current(device))
    if rc:
        _check(rc)
    return out if lse is None else (out, lse)


def attn_decode_tree(q, kcache, vcache, parents, cache_len=None, draft_len=None, out=None,
                     scale: Optional[float] = None, stream=None):
    """Attention of a tree of T <= 128 drafted tokens per sequence over a KV cache:
    q (B, H, T, D) (any strides, contiguous head rows), caches (B, H_kv, Skv, D).
    Sequence b's last draft_len[b] (default T) of its cache_len[b] (default Skv)
    cache rows are the drafted tokens; ``parents`` int32 (B, T), or (T,) for one
    tree, holds each token's parent among them, -1 for none.  A token sees the
    committed cache, its ancestors and itself.  Returns ``out`` like q; rows
    without a token are zeros.  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).tree(q, kcache, vcache, parents, cache_len, draft_len, out, scale)
        if done is not None:
            return done
    torch = _torch()
    (B, H, T, D), sq, code, device = _first(q, 4)
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_decode_tree(q, kcache, vcache, parents, cache_len, draft_len, out, scale)
    Bc, H_kv, Skv = _caches(kcache, vcache, q.dtype, device, D)
    if Bc != B or H_kv < 1 or H % H_kv:
        raise ValueError("kcache and vcache must be (B, H_kv, Skv, D) matching q, with H_kv dividing H")
    one = parents.dim() == 1
    par = _ints("parents", parents, (T,) if one else (B, T), device)
    cl = _ints("cache_len", cache_len, (B,), device)
    dl = _ints("draft_len", draft_len, (B,), device)
    if out is None:
        out = torch.empty_like(q)
        so = out.stride()
    else:
        so = out.stride()
        if out.shape != q.shape or out.dtype != q.dtype or out.device != device or so[3] != 1:
            raise ValueError("out must match q's shape, dtype and device, with contiguous rows")
    need = _tree_workspace(B, H, H_kv, T, Skv, D, code, device.index) if B and 0 < T <= 128 else 0
    ws = _workspace(need, device)
    rc = lib().attn_decode_tree(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), out.data_ptr(), B, H, H_kv, T, Skv,
                                D, _LL6(sq[0], sq[1], sq[2], so[0], so[1], so[2]), par, 0 if one else T, cl, dl,
                                _scale(scale, D), code, _ptr(ws), need if need > 0 else 0, _current(device))
    if rc:
        _check(rc)
    return out


def _pages(kpages, vpages, dtype, device, D, layered=False):
    """(n_pages, H_kv, page_size, strides of both in order) of a pair of page pools."""
    shape, n = kpages.shape, 5 if layered else 4
    if len(shape) != n or vpages.shape != shape or shape[-1] != D:
        raise ValueError(f"kpages and vpages must be ({'layers, ' if layered else ''}n_pages, H_kv, page_size, {D})")
    if kpages.dtype != dtype or vpages.dtype != dtype:
        raise TypeError("kpages and vpages must share one dtype" if layered else "q, kpages, vpages must share one dtype")
    if kpages.device != device or vpages.device != device:
        raise ValueError("the pages must be on one device" if layered else "the pages must be on q's device")
    ks, vs = kpages.stride(), vpages.stride()
    if ks[-1] != 1 or vs[-1] != 1:
        raise ValueError("kpages and vpages must have contiguous rows of D elements")
    return shape[-4], shape[-3], shape[-2], ks[:-1] + vs[:-1]


def _table(page_table, device):
    """(rows, max_pages, row stride, data_ptr) of a page table."""
    if not (page_table.dtype == _torch().int32 and page_table.device == device and page_table.dim() == 2
            and (page_table.stride(1) == 1 or page_table.shape[1] <= 1)):
        raise ValueError("page_table must be an int32 tensor of shape (sequences, max_pages) with contiguous rows on the "
                         "pages' device")
    return page_table.shape[0], page_table.shape[1], page_table.stride(0), page_table.data_ptr()


@functools.lru_cache(maxsize=4096)
def _paged_workspace(T, n_seq, H, H_kv, D, max_pages, page_size, ragged, dtype, device):
    return lib().attn_fwd_paged_workspace(T, n_seq, H, H_kv, D, max_pages, page_size, ragged, dtype)


def attn_fwd_paged(q, kpages, vpages, page_table, cache_len=None, cu_seqlens=None, out=None, lse=None,
                   scale: Optional[float] = None, return_lse: bool = False, stream=None):
    """Attention of new tokens over a paged KV cache: q (T, H, D), pages (n_pages,
    H_kv, page_size, D) (any strides, contiguous rows), ``page_table`` int32
    (sequences, max_pages).  Sequence s has tokens [cu_seqlens[s], cu_seqlens[s + 1])
    (T / sequences each without cu_seqlens, one each in a decode step), the last of
    its cache_len[s] keys (default: all its table holds); each sees the keys up to its own.
    Returns ``out`` (T, H, D), or ``(out, lse)`` with the (T, H) fp32 log-sum-exp
    when ``return_lse`` (or an ``lse`` tensor) is given.  Rows outside every sequence
    are not written.  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).paged(q, kpages, vpages, page_table, cache_len, cu_seqlens, out, lse, scale,
                                                 return_lse)
        if done is not None:
            return done
    torch = _torch()
    (T, H, D), sq, code, device = _first(q, 3)
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_fwd_paged(q, kpages, vpages, page_table, cache_len, cu_seqlens, out, lse, scale, return_lse)
    n_pages, H_kv, P, ps = _pages(kpages, vpages, q.dtype, device, D)
    if H_kv < 1 or H % H_kv:
        raise ValueError("kpages and vpages must be (n_pages, H_kv, page_size, D), with H_kv dividing H")
    n_seq, M, ts, table = _table(page_table, device)
    cu = _ints("cu_seqlens", cu_seqlens, (n_seq + 1,), device)
    cl = _ints("cache_len", cache_len, (n_seq,), device)
    if cu is None and (n_seq == 0 and T or n_seq and T % n_seq):
        raise ValueError(f"without cu_seqlens q's {T} tokens must be a multiple of the {n_seq} sequences")
    out, ot, oh = _out_rows("out", out, T, H, D, q.dtype, device)
    if lse is None:
        if return_lse:
            lse = torch.empty((T, H), dtype=torch.float32, device=device)
    elif not (lse.dtype == torch.float32 and lse.shape == (T, H) and lse.is_contiguous() and lse.device == device):
        raise ValueError("lse must be a contiguous float32 (T, H) tensor on q's device")
    need = _paged_workspace(T, n_seq, H, H_kv, D, M, P, 0 if cu is None else 1, code, device.index)
    ws = _workspace(need, device)
    rc = lib().attn_fwd_paged(q.data_ptr(), kpages.data_ptr(), vpages.data_ptr(), out.data_ptr(),
                              None if lse is None else lse.data_ptr(), T, H, H_kv, D,
                              _LL10(sq[0], sq[1], ot, oh, *ps), n_pages, P, table, M, ts, cu, cl, n_seq,
                              _scale(scale, D), code, _ptr(ws), need if need > 0 else 0, _current(device))
    if rc:
        _check(rc)
    return out if lse is None else (out, lse)


def attn_rope_frequencies(rotary_dim: int, theta: float = 10000.0, scaling: Optional[str] = None,
                          factor: float = 1.0, original_len: int = 8192, low: float = 1.0, high: float = 4.0):
    """Rotary frequencies in radians per position, a CPU float64 tensor of
    rotary_dim / 2 values w_p = theta^(-2p / rotary_dim), for attn_rope and
    attn_rope_append.  ``scaling`` stretches them for contexts ``factor`` times
    longer:

    "linear"      every w_p / factor (positions interpolated)
    "ntk"         theta grows by factor^(r / (r - 2)), r = rotary_dim: the highest
                  frequency stays, the lowest is divided by ``factor``
    "wavelength"  by the turns t_p = original_len * w_p / 2 pi that pair p makes
                  over the original context: w_p / factor below ``low`` turns, w_p
                  above ``high``, and a linear blend in t_p between them
    """
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and >= 0 (got {rotary_dim})")
    if not (theta > 0 and factor > 0):
        raise ValueError("theta and factor must be positive")
    torch = _torch()
    if scaling == "ntk" and rotary_dim > 2:
        theta = theta * factor ** (rotary_dim / (rotary_dim - 2))
    w = [theta ** (-2.0 * p / rotary_dim) for p in range(rotary_dim // 2)]
    if scaling == "linear":
        w = [x / factor for x in w]
    elif scaling == "wavelength":
        if not (original_len > 0 and high > low):
            raise ValueError("wavelength scaling needs original_len > 0 and high > low")
        blend = [min(1.0, max(0.0, (original_len * x / (2 * math.pi) - low) / (high - low))) for x in w]
        w = [x * ((1 - s) / factor + s) for x, s in zip(w, blend)]
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r} (linear, ntk, wavelength)")
    return torch.tensor(w, dtype=torch.float64)


def attn_rope(q, k, positions, freqs, q_out=None, k_out=None, interleaved: bool = False, inverse: bool = False,
              mscale: float = 1.0, stream=None):
    """Rotary positions: turn the first 2 * len(freqs) elements of every head row
    of q (T, H, D) and k (T, H_kv, D) by position * frequency.  k may be None.
    Returns ``(q_out, k_out)`` (``q_out`` alone without k); pass ``q_out=q`` to
    turn in place.  ``positions`` is int32 (T,), ``freqs`` from
    attn_rope_frequencies.  ``inverse`` turns back, which is also the gradient.
    Rows may be strided (slices of a fused projection).  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).rope(q, k, positions, freqs, q_out, k_out, interleaved, inverse, mscale)
        if done is not None:
            return done
    torch = _torch()
    (T, H, D), sq, code, device = _first(q, 3)
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_rope(q, k, positions, freqs, q_out, k_out, interleaved, inverse, mscale)
    dtype = q.dtype
    fr, rd = _freqs_arg(freqs, D)
    pos = _ints("positions", positions, (T,), device)
    if positions is None:
        raise ValueError("positions must be given")
    q_out, ot, oh = _out_rows("q_out", q_out, T, H, D, dtype, device)
    H_kv = kt = kh = kot = koh = 0
    if k is not None:
        H_kv, kt, kh = _rows("k", k, T, D, dtype, device)
        k_out, kot, koh = _out_rows("k_out", k_out, T, H_kv, D, dtype, device)
    elif k_out is not None:
        raise ValueError("k_out without k")
    rc = lib().attn_rope(q.data_ptr(), None if k is None else k.data_ptr(), q_out.data_ptr(),
                         None if k is None else k_out.data_ptr(), T, H, H_kv, D,
                         _LL8(sq[0], sq[1], kt, kh, ot, oh, kot, koh), pos, fr, rd, 1 if interleaved else 0,
                         1 if inverse else 0, mscale, code, _current(device))
    if rc:
        _check(rc)
    return q_out if k is None else (q_out, k_out)


def attn_rope_append(q, k, v, kcache, vcache, freqs, cu_seqlens=None, cache_len=None, positions=None, q_out=None,
                     k_out=None, interleaved: bool = False, mscale: float = 1.0, stream=None):
    """attn_rope of new tokens, with the turned keys and the values written to
    their rows of a (B, H_kv, Skv, D) cache: token i of sequence b (tokens
    [cu_seqlens[b], cu_seqlens[b + 1]), n of them; T / B each without cu_seqlens)
    goes to row cache_len[b] - n + i, which is also its position unless
    ``positions`` is given.  Returns ``q_out``, or ``(q_out, k_out)`` when a
    ``k_out`` (T, H_kv, D) is given for the turned keys.  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).rope_append(q, k, v, kcache, vcache, freqs, cu_seqlens, cache_len, positions,
                                                       q_out, k_out, interleaved, mscale)
        if done is not None:
            return done
    torch = _torch()
    (T, H, D), sq, code, device = _first(q, 3)
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_rope_append(q, k, v, kcache, vcache, freqs, cu_seqlens, cache_len, positions, q_out, k_out,
                                    interleaved, mscale)
    dtype = q.dtype
    H_kv, kt, kh = _rows("k", k, T, D, dtype, device)
    Hv, vt, vh = _rows("v", v, T, D, dtype, device)
    B, Hc, Skv = _caches(kcache, vcache, dtype, device, D)
    if Hv != H_kv or Hc != H_kv:
        raise ValueError("k and v must be (T, H_kv, D), kcache and vcache (B, H_kv, Skv, D)")
    fr, rd = _freqs_arg(freqs, D)
    cu = _ints("cu_seqlens", cu_seqlens, (B + 1,), device)
    cl = _ints("cache_len", cache_len, (B,), device)
    pos = _ints("positions", positions, (T,), device)
    q_out, ot, oh = _out_rows("q_out", q_out, T, H, D, dtype, device)
    kot = koh = 0
    if k_out is not None:
        k_out, kot, koh = _out_rows("k_out", k_out, T, H_kv, D, dtype, device)
    rc = lib().attn_rope_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(),
                                None if k_out is None else k_out.data_ptr(), kcache.data_ptr(), vcache.data_ptr(),
                                T, H, H_kv, D, _LL10(sq[0], sq[1], kt, kh, vt, vh, ot, oh, kot, koh), B, Skv, cu, cl,
                                pos, fr, rd, 1 if interleaved else 0, mscale, code, _current(device))
    if rc:
        _check(rc)
    return q_out if k_out is None else (q_out, k_out)


def _weight(name, w, D, dtype, device):
    """data_ptr of an optional (D,) weight."""
    if w is None:
        return None
    if not (w.shape == (D,) and w.device == device and w.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous ({D},) tensor on q's device")
    if w.dtype != dtype:
        raise TypeError(f"{name} must share q's dtype {dtype}")
    return w.data_ptr()


def attn_norm_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
                   interleaved: bool = False, mscale: float = 1.0, stream=None):
    """RMS norm of each head row of q (T, H, D) and k (T, H_kv, D), times the (D,)
    weights (a tensor without one is not normed), then attn_rope's turn of the result, in one
    pass and with one rounding.  k may be None.  Returns ``(q_out, k_out)`` (``q_out``
    alone without k); pass ``q_out=q`` to work in place.  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).norm_rope(q, k, positions, freqs, q_weight, k_weight, eps, q_out, k_out,
                                                     interleaved, mscale)
        if done is not None:
            return done
    torch = _torch()
    (T, H, D), sq, code, device = _first(q, 3)
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_norm_rope(q, k, positions, freqs, q_weight, k_weight, eps, q_out, k_out, interleaved, mscale)
    dtype = q.dtype
    fr, rd = _freqs_arg(freqs, D)
    pos = _ints("positions", positions, (T,), device)
    if positions is None:
        raise ValueError("positions must be given")
    wq, wk = _weight("q_weight", q_weight, D, dtype, device), _weight("k_weight", k_weight, D, dtype, device)
    q_out, ot, oh = _out_rows("q_out", q_out, T, H, D, dtype, device)
    H_kv = kt = kh = kot = koh = 0
    if k is not None:
        H_kv, kt, kh = _rows("k", k, T, D, dtype, device)
        k_out, kot, koh = _out_rows("k_out", k_out, T, H_kv, D, dtype, device)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out or k_weight without k")
    rc = lib().attn_norm_rope(q.data_ptr(), None if k is None else k.data_ptr(), q_out.data_ptr(),
                              None if k is None else k_out.data_ptr(), T, H, H_kv, D,
                              _LL8(sq[0], sq[1], kt, kh, ot, oh, kot, koh), pos, fr, rd, 1 if interleaved else 0, mscale,
                              wq, wk, eps, code, _current(device))
    if rc:
        _check(rc)
    return q_out if k is None else (q_out, k_out)


def attn_rope_append_paged(q, k, v, kpages, vpages, page_table, freqs, cache_len=None, cu_seqlens=None, positions=None,
                           q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None,
                           interleaved: bool = False, mscale: float = 1.0, stream=None):
    """attn_rope (or, with weights, attn_norm_rope) of new tokens, with the turned keys
    and the values written to the pages (n_pages, H_kv, page_size, D) of a cache: token i of
    sequence s (tokens [cu_seqlens[s], cu_seqlens[s + 1]), n of them; T / sequences
    each without cu_seqlens) is key j = cache_len[s] - n + i, in row j % page_size of
    page page_table[s, j // page_size]; j is also its position unless ``positions`` is given.
    Returns ``q_out``, or ``(q_out, k_out)`` when a ``k_out`` (T, H_kv, D) is given
    for the turned keys.  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).append_paged(q, k, v, kpages, vpages, page_table, freqs, cache_len, cu_seqlens,
                                                        positions, q_weight, k_weight, eps, q_out, k_out, interleaved, mscale)
        if done is not None:
            return done
    torch = _torch()
    (T, H, D), sq, code, device = _first(q, 3)
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_rope_append_paged(q, k, v, kpages, vpages, page_table, freqs, cache_len, cu_seqlens, positions,
                                          q_weight, k_weight, eps, q_out, k_out, interleaved, mscale)
    dtype = q.dtype
    H_kv, kt, kh = _rows("k", k, T, D, dtype, device)
    Hv, vt, vh = _rows("v", v, T, D, dtype, device)
    n_pages, Hp, P, ps = _pages(kpages, vpages, dtype, device, D)
    if Hv != H_kv or Hp != H_kv:
        raise ValueError("k and v must be (T, H_kv, D), kpages and vpages (n_pages, H_kv, page_size, D)")
    n_seq, M, tst, table = _table(page_table, device)
    fr, rd = _freqs_arg(freqs, D)
    cu = _ints("cu_seqlens", cu_seqlens, (n_seq + 1,), device)
    cl = _ints("cache_len", cache_len, (n_seq,), device)
    pos = _ints("positions", positions, (T,), device)
    if cu is None and n_seq == 0 and T:
        raise ValueError(f"without cu_seqlens q's {T} tokens must be a multiple of the {n_seq} sequences")
    wq, wk = _weight("q_weight", q_weight, D, dtype, device), _weight("k_weight", k_weight, D, dtype, device)
    q_out, ot, oh = _out_rows("q_out", q_out, T, H, D, dtype, device)
    kot = koh = 0
    if k_out is not None:
        k_out, kot, koh = _out_rows("k_out", k_out, T, H_kv, D, dtype, device)
    rc = lib().attn_rope_append_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(),
                                      None if k_out is None else k_out.data_ptr(), kpages.data_ptr(), vpages.data_ptr(),
                                      T, H, H_kv, D, _LL16(sq[0], sq[1], kt, kh, vt, vh, ot, oh, kot, koh, *ps), n_pages, P,
                                      table, M, tst, cu, cl, n_seq, pos, fr, rd, 1 if interleaved else 0, mscale, wq, wk, eps,
                                      code, _current(device))
    if rc:
        _check(rc)
    return q_out if k_out is None else (q_out, k_out)


def _given(out, shapes, device):
    """``out``, int32 tensors of the given shapes, or new ones."""
    torch = _torch()
    if out is None:
        return [torch.empty(s, dtype=torch.int32, device=device) for s in shapes]
    out = list(out)
    if len(out) != len(shapes):
        raise ValueError(f"out must hold {len(shapes)} tensors")
    for t, s in zip(out, shapes):
        if not (t.dtype == torch.int32 and t.device == device and t.shape == s and t.is_contiguous()):
            raise ValueError(f"out must hold contiguous int32 tensors of shapes {', '.join(str(tuple(s)) for s in shapes)} on "
                             "page_table's device")
    return out


def attn_pages_step(page_table, cache_len, n_pages: int, page_size: int, parents=None, new_len=None, pinned=None, out=None,
                    stream=None):
    """The next table of pages.  Row b goes on from row ``parents[b]`` of ``page_table``
    int32 (sequences, max_pages) (itself by default; an index that is no row starts an
    empty sequence) and is to hold ``new_len[b]`` tokens (by default its parent's
    ``cache_len``): pages beyond are dropped, missing ones are taken from those that no row
    holds and that are not ``pinned`` int32 (n_pages,).  Full pages are shared, a partly
    filled one has one holder and is copied for the others.  Returns ``(table, lengths,
    copies, free)``: new tensors, or the four of ``out``; ``copies`` (rows, 3) is for
    attn_pages_copy, ``free`` (1,) counts the free pages left (negative: missing; then
    call again from the old table with fewer or shorter rows, before copying and
    appending, as a page given later comes without the tokens it was to hold).
    See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).pages_step(page_table, cache_len, n_pages, page_size, parents, new_len, pinned, out)
        if done is not None:
            return done
    torch = _torch()
    device = page_table.device
    if not page_table.is_cuda:
        raise ValueError("page_table must be a CUDA tensor")
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_pages_step(page_table, cache_len, n_pages, page_size, parents, new_len, pinned, out)
    n_seq, M, ts, table = _table(page_table, device)
    n_out = n_seq if parents is None else parents.shape[0]
    cl = _ints("cache_len", cache_len, (n_seq,), device)
    par = _ints("parents", parents, (n_out,), device)
    new = _ints("new_len", new_len, (n_out,), device)
    pin = _ints("pinned", pinned, (n_pages,), device)
    r = _given(out, [(n_out, M), (n_out,), (n_out, 3), (1,)], device)
    need = lib().attn_pages_workspace(n_out, n_pages)
    ws = _workspace(need, device)
    rc = lib().attn_pages_step(table, cl, n_seq, M, ts, n_pages, page_size, par, new, pin, n_out, r[0].data_ptr(), M,
                               r[1].data_ptr(), r[2].data_ptr(), r[3].data_ptr(), _ptr(ws), max(need, 0), _current(device))
    if rc:
        _check(rc)
    return tuple(r)


def attn_pages_compact(page_table, cache_len, n_pages: int, page_size: int, pinned=None, out=None, stream=None):
    """Moves the pages that the rows of ``page_table`` hold together at the front of the
    pool (``pinned`` ones stay where they are).  Returns ``(table, copies, free)``: new
    tensors, or the three of ``out``; ``copies`` ((n_pages + 1) // 2, 3) is for
    attn_pages_copy, ``free`` (1,) counts the free pages.  See include/attn.h.
    """
    if stream is None:
        done = (_native or _load_native()).pages_compact(page_table, cache_len, n_pages, page_size, pinned, out)
        if done is not None:
            return done
    torch = _torch()
    device = page_table.device
    if not page_table.is_cuda:
        raise ValueError("page_table must be a CUDA tensor")
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_pages_compact(page_table, cache_len, n_pages, page_size, pinned, out)
    n_seq, M, ts, table = _table(page_table, device)
    cl = _ints("cache_len", cache_len, (n_seq,), device)
    pin = _ints("pinned", pinned, (n_pages,), device)
    r = _given(out, [(n_seq, M), ((n_pages + 1) // 2, 3), (1,)], device)
    need = lib().attn_pages_workspace(n_seq, n_pages)
    ws = _workspace(need, device)
    rc = lib().attn_pages_compact(table, cl, n_seq, M, ts, n_pages, page_size, pin, r[0].data_ptr(), M, r[1].data_ptr(),
                                  r[2].data_ptr(), _ptr(ws), max(need, 0), _current(device))
    if rc:
        _check(rc)
    return tuple(r)


def attn_pages_copy(kpages, vpages, copies, stream=None) -> None:
    """Copies pages within both pools, (n_pages, H_kv, page_size, D) or (layers, n_pages,
    H_kv, page_size, D) of any strides: for each (from, to, rows) of ``copies`` int32 (n, 3)
    the first ``rows`` rows of page ``to`` become those of page ``from``; pairs with an index
    that is no page are passed over.  See include/attn.h.
    """
    if stream is None and (_native or _load_native()).pages_copy(kpages, vpages, copies):
        return
    torch = _torch()
    device = kpages.device
    if not kpages.is_cuda:
        raise ValueError("kpages must be a CUDA tensor")
    if stream is not None or device.index != torch.cuda.current_device():
        with _elsewhere(device, stream):
            return attn_pages_copy(kpages, vpages, copies)
    code = _dtype_code(kpages)
    layered = kpages.dim() == 5
    D = kpages.shape[-1]
    n_pages, H_kv, P, st = _pages(kpages, vpages, kpages.dtype, device, D, layered)
    layers = kpages.shape[0] if layered else 1
    if not layered:
        st = (0, *st[:3], 0, *st[3:])
    if not (copies.dtype == torch.int32 and copies.device == device and copies.dim() == 2 and copies.shape[1] == 3
            and copies.is_contiguous()):
        raise ValueError("copies must be a contiguous int32 tensor of shape (n, 3) on the pages' device")
    rc = lib().attn_pages_copy(kpages.data_ptr(), vpages.data_ptr(), layers, n_pages, H_kv, P, D, _LL8(*st),
                               copies.data_ptr(), copies.shape[0], code, _current(device))
    if rc:
        _check(rc)


def attn_device_status(stream=None) -> None:
    """Synchronise the stream and raise AttnError if a kernel reported a timed-out
    wait (ATTN_ETIMEOUT) or a shared prefill work counter (ATTN_ECONFLICT)."""
    _check(lib().attn_device_status(_stream_handle(stream)))


def attn_selftest_wait_timeout(limit_cycles: int = 1_000_000, stream=None) -> None:
    """Enqueue the diagnostic kernel whose wait runs out (see include/attn.h)."""
    _check(lib().attn_selftest_wait_timeout(int(limit_cycles), _stream_handle(stream)))


def attn_release() -> None:
    lib().attn_release()


__all__ = [
    "attn_fwd", "attn_fwd_chunked", "attn_fwd_debug", "attn_fwd_host", "attn_decode", "attn_decode_noalloc", "attn_decode_splits", "attn_fwd_packed", "attn_decode_tree",
    "attn_fwd_paged", "attn_norm_rope", "attn_rope_append_paged",
    "attn_pages_step", "attn_pages_compact", "attn_pages_copy",
    "attn_rope",
    "attn_rope_append", "attn_rope_frequencies", "attn_device_status", "attn_release",
    "attn_last_error", "attn_selftest_wait_timeout", "lib", "AttnError", "SIGNATURES", "LIB_PATH",
    "ATTN_F32", "ATTN_BF16", "ATTN_OK", "ATTN_EINVAL", "ATTN_EUNSUPPORTED", "ATTN_ECUDA",
    "ATTN_ENOMEM", "ATTN_ETIMEOUT", "ATTN_ECONFLICT",
]
