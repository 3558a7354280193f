"""Python binding of the MoDA C ABI (``libmoda.so``, header ``include/moda.h``).

Argument marshalling only: every function forwards torch CUDA tensors' device
pointers and the current CUDA stream to the C entry point of the same name.
All arithmetic runs in the library's CUDA kernels. There is no CPU fallback:
importing this package fails if the library has not been built
(``python depth_kv_attention_b200/csrc/build.py``).

Layouts (contiguous): q/out/dout [B,T,Hq,d]; k/v [B,T,Hkv,d];
kd/vd [B,T,Ld,Hkv,d]; lse [B,Hq,T] fp32. The paged sequence cache packs the
new tokens of all sequences along one axis: q/out [N,Hq,d], kd/vd [N,Ld,Hkv,d],
lse [N,Hq], pages [num_pages,Hkv,page_size,d].
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

import torch

__all__ = [
    "MODA_OK", "ModaError", "lib", "LIB_PATH", "moda_abi_version", "moda_status_string",
    "moda_fwd", "moda_fwd_sel", "moda_bwd", "moda_bwd_sel", "moda_bwd_workspace_bytes", "moda_bwd_noalloc", "moda_pack_depth",
    "moda_pack_depth_bytes", "moda_fwd_packed", "moda_depth_write", "moda_device_status",
    "moda_debug_set_wait_limit", "moda_debug_exp2_poly", "moda_fwd_from_host",
    "moda_fwd_host_staging_bytes", "moda_fwd_q8", "moda_depth_quantize_q8", "moda_depth_write_q8",
    "moda_depth_slot_layout", "depth_slot_view", "moda_paged_append", "moda_paged_append_q8", "moda_fwd_paged",
    "moda_fwd_paged_q8", "moda_fwd_paged_workspace_bytes",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoda.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python depth_kv_attention_b200/csrc/build.py` "
        "(the MoDA path has no CPU fallback)")
lib = ctypes.CDLL(LIB_PATH)

MODA_OK = 0
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}
_IMPL = {"auto": 0, "simt": 1, "tc": 2, "tc2": 3}
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


def _sig(name, res, args):
    fn = getattr(lib, name)
    fn.restype = res
    fn.argtypes = args
    return fn


_DIMS = [_i] * 6  # B, T, Hq, Hkv, d, Ld
_c_abi_version = _sig("moda_abi_version", _i, [])
_c_status_string = _sig("moda_status_string", ctypes.c_char_p, [_i])
_c_fwd_ex = _sig("moda_fwd_ex", _i, [_vp] * 5 + _DIMS + [_i, _f, _vp, _vp, _vp, _i])
_c_fwd = _sig("moda_fwd", _i, [_vp] * 5 + _DIMS + [_i, _f, _vp, _vp, _vp])
_c_fwd_sel = _sig("moda_fwd_sel", _i, [_vp] * 6 + _DIMS + [_i, _f, _vp, _vp, _vp, _i])
_c_bwd_ws = _sig("moda_bwd_workspace_bytes", _sz, _DIMS + [_i])
_c_bwd_ex = _sig("moda_bwd_ex", _i, [_vp] * 8 + _DIMS + [_i, _f] + [_vp] * 5 + [_vp, _sz, _vp, _i])
_c_bwd = _sig("moda_bwd", _i, [_vp] * 8 + _DIMS + [_i, _f] + [_vp] * 5 + [_vp, _sz, _vp])
_c_bwd_sel = _sig("moda_bwd_sel", _i, [_vp] * 9 + _DIMS + [_i, _f] + [_vp] * 5 + [_vp, _sz, _vp, _i])
_c_pack_bytes = _sig("moda_pack_depth_bytes", _sz, [_i] * 5 + [_i])
_c_pack = _sig("moda_pack_depth", _i, [_vp, _vp] + [_i] * 5 + [_i, _vp, _vp])
_c_fwd_packed = _sig("moda_fwd_packed", _i, [_vp] * 4 + _DIMS + [_i, _f, _vp, _vp, _vp])
_c_depth_write = _sig("moda_depth_write", _i, [_vp, _vp] + [_i] * 6 + [_i, _vp, _vp, _vp])
_c_dev_status = _sig("moda_device_status", _i, [_vp])
_c_wait_limit = _sig("moda_debug_set_wait_limit", _i, [ctypes.c_uint32])
_c_exp2_poly = _sig("moda_debug_exp2_poly", _i, [_vp, _vp, _i, _vp])
_c_bwd_noalloc = _sig("moda_bwd_noalloc", _i, [_vp] * 8 + _DIMS + [_i, _f] + [_vp] * 5 + [_vp])
_c_host_bytes = _sig("moda_fwd_host_staging_bytes", _sz, _DIMS + [_i])
_c_slot_layout = _sig("moda_depth_slot_layout", _i, [_i] * 6 + [ctypes.POINTER(ctypes.c_longlong),
                                                                  ctypes.POINTER(ctypes.c_longlong)])
_c_fwd_q8 = _sig("moda_fwd_q8", _i, [_vp] * 7 + _DIMS + [_i, _f, _vp, _vp, _vp, _i])
_c_quant_q8 = _sig("moda_depth_quantize_q8", _i, [_vp, _vp] + [_i] * 5 + [_i] + [_vp] * 4 + [_vp])
_c_write_q8 = _sig("moda_depth_write_q8", _i, [_vp, _vp] + [_i] * 6 + [_i] + [_vp] * 4 + [_vp])
_c_fwd_host = _sig("moda_fwd_host", _i, [_vp] * 5 + _DIMS + [_i, _f, _vp, _vp, _vp, _sz, _vp])
_ll = ctypes.c_longlong
_APPEND = [_vp] * 3 + [_ll] * 3 + [_vp, _i, _i, _i] + [_vp] * 3 + [_i] * 9
_c_append = _sig("moda_paged_append", _i, _APPEND + [_vp] * 5 + [_i, _i, _vp])
_c_append_q8 = _sig("moda_paged_append_q8", _i, _APPEND + [_vp] * 7 + [_i, _i, _vp])
_c_paged_ws = _sig("moda_fwd_paged_workspace_bytes", _sz, [_i] * 10)
_PAGED = [_vp] * 5 + [_i] * 12 + [_f, _vp, _vp, _vp, _sz, _vp, _i]
_c_fwd_paged = _sig("moda_fwd_paged", _i, [_vp] * 3 + _PAGED)
_c_fwd_paged_q8 = _sig("moda_fwd_paged_q8", _i, [_vp] * 5 + _PAGED)


class ModaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {moda_status_string(code)} ({code})")


def moda_abi_version() -> int:
    return _c_abi_version()


def moda_status_string(code: int) -> str:
    return _c_status_string(code).decode()


def _check(code: int, where: str) -> None:
    if code != MODA_OK:
        raise ModaError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dims(q, k, kd):
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    Ld = 0 if kd is None else kd.shape[2]
    return B, T, Hq, Hkv, d, Ld


def _check_tensors(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("MoDA tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("MoDA tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("MoDA tensors must be on one device")


def moda_fwd(q, k, v, kd=None, vd=None, scale: float | None = None, out=None, lse=None,
             impl: str = "auto", stream=None):
    """MoDA forward (``moda_fwd_ex``). Returns (out, lse)."""
    if kd is not None and kd.shape[2] == 0:
        kd = vd = None
    _check_tensors(q, k, v, kd, vd, out, lse)
    B, T, Hq, Hkv, d, Ld = _dims(q, k, kd)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        _check(_c_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(kd), _ptr(vd), B, T, Hq, Hkv, d, Ld,
                         _DTYPE[q.dtype], scale, _ptr(out), _ptr(lse), _stream(stream), _IMPL[impl]),
               "moda_fwd")
    return out, lse


def _check_sel(depth_sel, B, T):
    if depth_sel is None:
        return
    if depth_sel.dtype != torch.int64 or tuple(depth_sel.shape) != (B, T):
        raise ValueError("depth_sel must be an int64 [B, T] tensor of depth-slot bit masks")


def moda_fwd_sel(q, k, v, kd, vd, depth_sel, scale: float | None = None, out=None, lse=None,
                 impl: str = "auto", stream=None):
    """MoDA forward with per-token depth-slot selection (``moda_fwd_sel``).

    ``depth_sel``: int64 [B, T] bit masks (bit i set = the token's depth slot
    i takes part), or None for every slot. Returns (out, lse)."""
    _check_tensors(q, k, v, kd, vd, depth_sel, out, lse)
    B, T, Hq, Hkv, d, Ld = _dims(q, k, kd)
    _check_sel(depth_sel, B, T)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        _check(_c_fwd_sel(_ptr(q), _ptr(k), _ptr(v), _ptr(kd), _ptr(vd), _ptr(depth_sel), B, T, Hq,
                          Hkv, d, Ld, _DTYPE[q.dtype], scale, _ptr(out), _ptr(lse), _stream(stream),
                          _IMPL[impl]), "moda_fwd_sel")
    return out, lse


def moda_bwd_sel(q, k, v, kd, vd, depth_sel, out, lse, dout, scale: float | None = None,
                 grads=None, workspace=None, impl: str = "auto", stream=None):
    """Gradients of ``moda_fwd_sel`` (``moda_bwd_sel``), same ``depth_sel``.
    Returns (dq, dk, dv, dkd, dvd)."""
    _check_tensors(q, k, v, kd, vd, depth_sel, out, lse, dout)
    B, T, Hq, Hkv, d, Ld = _dims(q, k, kd)
    _check_sel(depth_sel, B, T)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(kd), torch.empty_like(vd))
    dq, dk, dv, dkd, dvd = grads
    need = moda_bwd_workspace_bytes(B, T, Hq, Hkv, d, Ld, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    with torch.cuda.device(q.device):
        _check(_c_bwd_sel(_ptr(q), _ptr(k), _ptr(v), _ptr(kd), _ptr(vd), _ptr(depth_sel), _ptr(out),
                          _ptr(lse), _ptr(dout), B, T, Hq, Hkv, d, Ld, _DTYPE[q.dtype], scale,
                          _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dkd), _ptr(dvd), _ptr(workspace),
                          workspace.numel(), _stream(stream), _IMPL[impl]), "moda_bwd_sel")
    return dq, dk, dv, dkd, dvd


def moda_bwd_workspace_bytes(B, T, Hq, Hkv, d, Ld, dtype) -> int:
    return _c_bwd_ws(B, T, Hq, Hkv, d, Ld, _DTYPE[dtype])


def moda_bwd(q, k, v, kd, vd, out, lse, dout, scale: float | None = None, grads=None,
             workspace=None, impl: str = "auto", stream=None):
    """MoDA backward (``moda_bwd_ex``). Returns (dq, dk, dv, dkd, dvd)."""
    if kd is not None and kd.shape[2] == 0:
        kd = vd = None
    _check_tensors(q, k, v, kd, vd, out, lse, dout)
    B, T, Hq, Hkv, d, Ld = _dims(q, k, kd)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 None if kd is None else torch.empty_like(kd),
                 None if vd is None else torch.empty_like(vd))
    dq, dk, dv, dkd, dvd = grads
    need = moda_bwd_workspace_bytes(B, T, Hq, Hkv, d, Ld, q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=q.device, dtype=torch.uint8)
    with torch.cuda.device(q.device):
        _check(_c_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(kd), _ptr(vd), _ptr(out), _ptr(lse),
                         _ptr(dout), B, T, Hq, Hkv, d, Ld, _DTYPE[q.dtype], scale, _ptr(dq),
                         _ptr(dk), _ptr(dv), _ptr(dkd), _ptr(dvd), _ptr(workspace),
                         workspace.numel(), _stream(stream), _IMPL[impl]), "moda_bwd")
    return dq, dk, dv, dkd, dvd


def moda_bwd_noalloc(q, k, v, kd, vd, out, lse, dout, scale: float | None = None, grads=None,
                     stream=None):
    """``moda_bwd_noalloc``: the backward without a workspace argument, for
    callers that cannot allocate device memory (the library's fixed scratch
    array holds the row statistics). Output tensors come from ``grads`` or
    are created here by torch (the C call itself allocates nothing).
    Returns (dq, dk, dv, dkd, dvd)."""
    if kd is not None and kd.shape[2] == 0:
        kd = vd = None
    _check_tensors(q, k, v, kd, vd, out, lse, dout)
    B, T, Hq, Hkv, d, Ld = _dims(q, k, kd)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 None if kd is None else torch.empty_like(kd),
                 None if vd is None else torch.empty_like(vd))
    dq, dk, dv, dkd, dvd = grads
    with torch.cuda.device(q.device):
        _check(_c_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(kd), _ptr(vd), _ptr(out), _ptr(lse),
                              _ptr(dout), B, T, Hq, Hkv, d, Ld, _DTYPE[q.dtype], scale, _ptr(dq),
                              _ptr(dk), _ptr(dv), _ptr(dkd), _ptr(dvd), _stream(stream)),
               "moda_bwd_noalloc")
    return dq, dk, dv, dkd, dvd


def moda_pack_depth_bytes(B, T, Hkv, d, Ld, dtype) -> int:
    return _c_pack_bytes(B, T, Hkv, d, Ld, _DTYPE[dtype])


def moda_pack_depth(kd, vd, packed=None, stream=None):
    """Repack kd, vd [B,T,Ld,Hkv,d] into [2,B,Hkv,T*Ld,d] (``moda_pack_depth``)."""
    _check_tensors(kd, vd, packed)
    B, T, Ld, Hkv, d = kd.shape
    n = moda_pack_depth_bytes(B, T, Hkv, d, Ld, kd.dtype)
    if packed is None:
        packed = torch.empty(n // kd.element_size(), device=kd.device, dtype=kd.dtype)
    with torch.cuda.device(kd.device):
        _check(_c_pack(_ptr(kd), _ptr(vd), B, T, Hkv, d, Ld, _DTYPE[kd.dtype], _ptr(packed),
                       _stream(stream)), "moda_pack_depth")
    return packed


def moda_fwd_packed(q, k, v, packed, Ld: int, scale: float | None = None, out=None, lse=None,
                    stream=None):
    """MoDA forward reading depth from ``moda_pack_depth``'s layout."""
    _check_tensors(q, k, v, packed, out, lse)
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        _check(_c_fwd_packed(_ptr(q), _ptr(k), _ptr(v), _ptr(packed) if Ld else None, B, T, Hq,
                             Hkv, d, Ld, _DTYPE[q.dtype], scale, _ptr(out), _ptr(lse),
                             _stream(stream)), "moda_fwd_packed")
    return out, lse


def moda_depth_write(k, v, kd, vd, slot: int, stream=None):
    """The write step (``moda_depth_write``): k, v [B,T,Hkv,d] into slot
    ``slot`` of the depth cache kd, vd [B,T,Ld,Hkv,d], in place. Returns (kd, vd)."""
    _check_tensors(k, v, kd, vd)
    B, T, Hkv, d = k.shape
    Ld = kd.shape[2]
    if tuple(v.shape) != (B, T, Hkv, d) or tuple(kd.shape) != (B, T, Ld, Hkv, d) or kd.shape != vd.shape:
        raise ValueError("moda_depth_write: k, v [B,T,Hkv,d] and kd, vd [B,T,Ld,Hkv,d] expected")
    if not (k.dtype == v.dtype == kd.dtype == vd.dtype):
        raise ValueError("moda_depth_write: one dtype expected")
    with torch.cuda.device(k.device):
        _check(_c_depth_write(_ptr(k), _ptr(v), B, T, Hkv, d, Ld, slot, _DTYPE[k.dtype], _ptr(kd),
                              _ptr(vd), _stream(stream)), "moda_depth_write")
    return kd, vd


def moda_depth_quantize_q8(kd, vd, out=None, stream=None):
    """8-bit depth cache of kd, vd [B,T,Ld,Hkv,d] (``moda_depth_quantize_q8``).
    Returns (kd8, vd8, kd_scale, vd_scale): int8 codes [B,T,Ld,Hkv,d] and fp32
    row scales [B,T,Ld,Hkv]; ``out`` may supply those four tensors."""
    _check_tensors(kd, vd)
    B, T, Ld, Hkv, d = kd.shape
    if out is None:
        out = (torch.empty(kd.shape, dtype=torch.int8, device=kd.device),
               torch.empty(kd.shape, dtype=torch.int8, device=kd.device),
               torch.empty(kd.shape[:-1], dtype=torch.float32, device=kd.device),
               torch.empty(kd.shape[:-1], dtype=torch.float32, device=kd.device))
    _check_tensors(*out)
    with torch.cuda.device(kd.device):
        _check(_c_quant_q8(_ptr(kd), _ptr(vd), B, T, Hkv, d, Ld, _DTYPE[kd.dtype], *(_ptr(t) for t in out),
                           _stream(stream)), "moda_depth_quantize_q8")
    return out


def moda_depth_write_q8(k, v, kd8, vd8, kd_scale, vd_scale, slot: int, stream=None):
    """The write step into an 8-bit depth cache (``moda_depth_write_q8``): k, v
    [B,T,Hkv,d] quantised into slot ``slot`` of kd8, vd8 and their scales, in
    place. Returns (kd8, vd8, kd_scale, vd_scale)."""
    _check_tensors(k, v, kd8, vd8, kd_scale, vd_scale)
    B, T, Hkv, d = k.shape
    Ld = kd8.shape[2]
    if kd8.dtype != torch.int8 or kd_scale.dtype != torch.float32 or tuple(kd8.shape) != (B, T, Ld, Hkv, d):
        raise ValueError("moda_depth_write_q8: int8 kd8 [B,T,Ld,Hkv,d] and fp32 scales [B,T,Ld,Hkv] expected")
    with torch.cuda.device(k.device):
        _check(_c_write_q8(_ptr(k), _ptr(v), B, T, Hkv, d, Ld, slot, _DTYPE[k.dtype], _ptr(kd8), _ptr(vd8),
                           _ptr(kd_scale), _ptr(vd_scale), _stream(stream)), "moda_depth_write_q8")
    return kd8, vd8, kd_scale, vd_scale


def moda_fwd_q8(q, k, v, kd8, vd8, kd_scale, vd_scale, scale: float | None = None, out=None, lse=None,
                impl: str = "auto", stream=None):
    """MoDA forward over an 8-bit depth cache (``moda_fwd_q8``). Returns (out, lse)."""
    if kd8 is not None and kd8.shape[2] == 0:
        kd8 = vd8 = kd_scale = vd_scale = None
    _check_tensors(q, k, v, kd8, vd8, kd_scale, vd_scale, out, lse)
    B, T, Hq, Hkv, d, Ld = _dims(q, k, kd8)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, T), device=q.device, dtype=torch.float32)
    with torch.cuda.device(q.device):
        _check(_c_fwd_q8(_ptr(q), _ptr(k), _ptr(v), _ptr(kd8), _ptr(vd8), _ptr(kd_scale), _ptr(vd_scale),
                         B, T, Hq, Hkv, d, Ld, _DTYPE[q.dtype], scale, _ptr(out), _ptr(lse),
                         _stream(stream), _IMPL[impl]), "moda_fwd_q8")
    return out, lse


def moda_depth_slot_layout(B, T, Hkv, d, Ld, slot):
    """(offset, strides) of depth slot ``slot`` inside a native cache
    [B,T,Ld,Hkv,d], in elements (``moda_depth_slot_layout``)."""
    off = ctypes.c_longlong()
    st = (ctypes.c_longlong * 4)()
    _check(_c_slot_layout(B, T, Hkv, d, Ld, slot, ctypes.byref(off), st), "moda_depth_slot_layout")
    return off.value, tuple(st)


def depth_slot_view(kd, slot: int):
    """Slot ``slot`` of a depth cache kd [B,T,Ld,Hkv,d] as a strided
    [B, T, Hkv, d] view (no copy), per ``moda_depth_slot_layout``: a producer
    that writes its K or V into this view (e.g. a projection GEMM with
    ``out=view.view(B*T, Hkv*d)``-style leading dimension Ld*Hkv*d) fills the
    cache in place."""
    B, T, Ld, Hkv, d = kd.shape
    off, st = moda_depth_slot_layout(B, T, Hkv, d, Ld, slot)
    return kd.as_strided((B, T, Hkv, d), st, kd.storage_offset() + off)


def _on(device):
    """Guard that makes ``device`` current; free when it is already."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_cache(where, q, k_pages, v_pages, scales, block_table, cu_q, ctx_lens, kd, vd, *others):
    """Shapes, types and places of the arguments that both paged operators
    share. Returns (N, B, Hq, Hkv, d, num_pages, page_size, max_blocks)."""
    if q.dim() != 3 or k_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError(f"{where}: packed tokens [N,H,d], pages [num_pages,Hkv,page_size,d] and a block table "
                         "[B,max_blocks] expected")
    N, Hq, d = q.shape
    num_pages, Hkv, page_size, dp = k_pages.shape
    B, max_blocks = block_table.shape
    if dp != d or v_pages.shape != k_pages.shape or cu_q.shape != (B + 1,) or ctx_lens.shape != (B,):
        raise ValueError(f"{where}: shapes of pages, cu_q [B+1] or ctx_lens [B] do not match")
    if not (cu_q.dtype == ctx_lens.dtype == block_table.dtype == torch.int32):
        raise ValueError(f"{where}: int32 cu_q, ctx_lens and block_table expected")
    if q.dtype not in _DTYPE:
        raise ValueError(f"{where}: bf16 or fp32 expected")
    want = q.dtype if scales is None else torch.int8
    if k_pages.dtype != want or v_pages.dtype != want:
        raise ValueError(f"{where}: pages of {want} expected")
    if scales is not None:
        for t in scales:
            if t.dtype != torch.float32 or t.shape != (num_pages, Hkv):
                raise ValueError(f"{where}: fp32 scales [num_pages,Hkv] expected")
    if (kd is None) != (vd is None):
        raise ValueError(f"{where}: kd and vd come together")
    if kd is not None and (kd.dim() != 4 or kd.shape[0] != N or kd.shape[2:] != (Hkv, d) or kd.shape != vd.shape
                           or kd.dtype != q.dtype or vd.dtype != q.dtype):
        raise ValueError(f"{where}: kd, vd [N,Ld,Hkv,d] of the tokens' type expected")
    dev = q.device
    for t in (k_pages, v_pages, block_table, cu_q, ctx_lens, kd, vd, *(scales or ()), *others):
        if t is not None and not (t.is_contiguous() and t.device == dev):
            raise ValueError(f"{where}: contiguous tensors on one device expected")
    if not q.is_cuda:
        raise ValueError("MoDA tensors must be CUDA tensors")
    return N, B, Hq, Hkv, d, num_pages, page_size, max_blocks


def _token_stride(where, t, device):
    """Elements from token to token of t [N,H,d] with dense heads (a dimension
    of one element may carry any stride)."""
    N, H, d = t.shape
    if t.device != device or (d > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != d):
        raise ValueError(f"{where}: dense heads on one device expected (any stride from token to token)")
    return t.stride(0) if N > 1 else H * d


def _append(where, fn, q, k, v, pages, scales, block_table, cu_q, ctx_lens, rope, interleaved, q_out, kd, vd, slot,
            stream):
    N, B, Hk, Hkv, d, num_pages, page_size, max_blocks = _check_cache(
        where, k, pages[0], pages[1], scales, block_table, cu_q, ctx_lens, kd, vd, rope, q_out)
    if Hk != Hkv or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError(f"{where}: k, v [N,Hkv,d] of one type expected")
    Hq = Hkv
    if q is not None:
        Hq = q.shape[1] if q.dim() == 3 else 0
        if q.shape != (N, Hq, d) or q.dtype != k.dtype:
            raise ValueError(f"{where}: q [N,Hq,d] of the type of k expected")
        if q_out is None:
            q_out = torch.empty((N, Hq, d), device=q.device, dtype=q.dtype)
        elif q_out.shape != q.shape or q_out.dtype != q.dtype:
            raise ValueError(f"{where}: q_out like q expected")
    elif q_out is not None:
        raise ValueError(f"{where}: q_out without q")
    strides = [0 if t is None else _token_stride(where, t, k.device) for t in (q, k, v)]
    if rope is not None and (rope.dtype != torch.float32 or rope.dim() != 2):
        raise ValueError(f"{where}: fp32 rope [positions, rot_dim] expected")
    if N == 0:
        return q_out
    with _on(k.device):
        _check(fn(_addr(q), k.data_ptr(), v.data_ptr(), *strides, _addr(rope),
                  0 if rope is None else rope.shape[0], 0 if rope is None else rope.shape[1], int(interleaved),
                  cu_q.data_ptr(), ctx_lens.data_ptr(), block_table.data_ptr(), N, B, Hq, Hkv, d, num_pages, page_size,
                  max_blocks, _DTYPE[k.dtype], pages[0].data_ptr(), pages[1].data_ptr(),
                  *(t.data_ptr() for t in scales or ()), _addr(q_out), _addr(kd), _addr(vd),
                  0 if kd is None else kd.shape[1], slot, _stream_addr(stream)), where)
    return q_out


def _stream_addr(stream):
    # the raw handle: making a Stream object costs as much as a launch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def moda_paged_append(q, k, v, k_pages, v_pages, block_table, cu_q, ctx_lens, rope=None, interleaved: bool = False,
                      q_out=None, kd=None, vd=None, slot: int = 0, stream=None):
    """Append new tokens to the paged sequence cache (``moda_paged_append``):
    k [N,Hkv,d], rotated by each token's position, and v into k_pages, v_pages
    [num_pages,Hkv,page_size,d], in place; with kd, vd [N,Ld,Hkv,d] also into
    depth slot ``slot``. q (may be None), k and v need dense heads only, so
    column blocks of one projection's output serve as they are. ``rope`` [positions, rot_dim]
    holds cos | sin rows; None leaves q and k unrotated. Returns the rotated q
    (``q_out`` when given; None without q)."""
    return _append("moda_paged_append", _c_append, q, k, v, (k_pages, v_pages), None, block_table, cu_q, ctx_lens,
                   rope, interleaved, q_out, kd, vd, slot, stream)


def moda_paged_append_q8(q, k, v, k_pages, v_pages, k_scale, v_scale, block_table, cu_q, ctx_lens, rope=None,
                         interleaved: bool = False, q_out=None, kd=None, vd=None, slot: int = 0, stream=None):
    """``moda_paged_append`` into 8-bit pages (``moda_paged_append_q8``): int8
    codes k_pages, v_pages and fp32 power-of-two scales [num_pages,Hkv], in
    place. kd, vd stay in the tokens' type."""
    return _append("moda_paged_append_q8", _c_append_q8, q, k, v, (k_pages, v_pages), (k_scale, v_scale), block_table,
                   cu_q, ctx_lens, rope, interleaved, q_out, kd, vd, slot, stream)


@functools.lru_cache(maxsize=256)
def _paged_ws(*dims):
    return _c_paged_ws(*dims)


def moda_fwd_paged_workspace_bytes(N, B, max_q, Hq, Hkv, d, num_pages, page_size, dtype, q8: bool = False) -> int:
    return _c_paged_ws(N, B, max_q, Hq, Hkv, d, num_pages, page_size, _DTYPE[dtype], int(q8))


def _fwd_paged(where, fn, q, pages, scales, block_table, cu_q, ctx_lens, max_q, kd, vd, Ld, scale, out, lse,
               workspace, impl, stream):
    N, B, Hq, Hkv, d, num_pages, page_size, max_blocks = _check_cache(
        where, q, pages[0], pages[1], scales, block_table, cu_q, ctx_lens, kd, vd, q, out, lse, workspace)
    cap = 0 if kd is None else kd.shape[1]
    if Ld is None:
        Ld = cap
    if not 0 <= Ld <= cap:
        raise ValueError(f"{where}: Ld must lie in [0, slots of kd]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError(f"{where}: out like q expected")
    if lse is None:
        lse = torch.empty((N, Hq), device=q.device, dtype=torch.float32)
    elif lse.shape != (N, Hq) or lse.dtype != torch.float32:
        raise ValueError(f"{where}: fp32 lse [N,Hq] expected")
    if N == 0:
        return out, lse
    dt = _DTYPE[q.dtype]
    need = _paged_ws(N, B, max_q, Hq, Hkv, d, num_pages, page_size, dt, scales is not None)
    with _on(q.device):
        if workspace is None and need:
            # from the pool of the stream it is used on
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
        _check(fn(q.data_ptr(), pages[0].data_ptr(), pages[1].data_ptr(), *(t.data_ptr() for t in scales or ()),
                  _addr(kd) if Ld else None, _addr(vd) if Ld else None, cu_q.data_ptr(), ctx_lens.data_ptr(),
                  block_table.data_ptr(), N, B, max_q, Hq, Hkv, d, Ld, cap, num_pages, page_size, max_blocks, dt,
                  scale, out.data_ptr(), lse.data_ptr(), _addr(workspace),
                  0 if workspace is None else workspace.numel() * workspace.element_size(), _stream_addr(stream),
                  _IMPL[impl]), where)
    return out, lse


def moda_fwd_paged(q, k_pages, v_pages, block_table, cu_q, ctx_lens, max_q: int, kd=None, vd=None,
                   Ld: int | None = None, scale: float | None = None, out=None, lse=None, workspace=None,
                   impl: str = "auto", stream=None):
    """MoDA read step over the paged sequence cache (``moda_fwd_paged``): q
    [N,Hq,d] of the new tokens against their sequences' pages and, under the
    same softmax, slots 0..Ld-1 (default all) of their own depth rows kd, vd
    [N,slots,Hkv,d]. ``max_q``: about the most new tokens of any sequence.
    ``workspace``: a uint8 CUDA tensor of moda_fwd_paged_workspace_bytes, made
    here when not given. Returns (out [N,Hq,d], lse [N,Hq])."""
    return _fwd_paged("moda_fwd_paged", _c_fwd_paged, q, (k_pages, v_pages), None, block_table, cu_q, ctx_lens, max_q,
                      kd, vd, Ld, scale, out, lse, workspace, impl, stream)


def moda_fwd_paged_q8(q, k_pages, v_pages, k_scale, v_scale, block_table, cu_q, ctx_lens, max_q: int, kd=None,
                      vd=None, Ld: int | None = None, scale: float | None = None, out=None, lse=None, workspace=None,
                      impl: str = "auto", stream=None):
    """``moda_fwd_paged`` over 8-bit pages (``moda_fwd_paged_q8``): int8 codes
    and fp32 scales [num_pages,Hkv], as moda_paged_append_q8 writes them."""
    return _fwd_paged("moda_fwd_paged_q8", _c_fwd_paged_q8, q, (k_pages, v_pages), (k_scale, v_scale), block_table,
                      cu_q, ctx_lens, max_q, kd, vd, Ld, scale, out, lse, workspace, impl, stream)


def moda_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return _c_dev_status(_stream(stream))


def moda_debug_set_wait_limit(spins: int) -> None:
    _check(_c_wait_limit(spins), "moda_debug_set_wait_limit")


def moda_debug_exp2_poly(x, y=None, stream=None):
    """Apply the forward kernel's FMA-pipe exp2 to a CUDA fp32 tensor."""
    _check_tensors(x, y)
    if y is None:
        y = torch.empty_like(x)
    with torch.cuda.device(x.device):
        _check(_c_exp2_poly(_ptr(x), _ptr(y), x.numel(), _stream(stream)), "moda_debug_exp2_poly")
    return y


def moda_fwd_host_staging_bytes(B, T, Hq, Hkv, d, Ld, dtype) -> int:
    return _c_host_bytes(B, T, Hq, Hkv, d, Ld, _DTYPE[dtype])


def moda_fwd_from_host(q, k, v, kd=None, vd=None, scale: float | None = None, device="cuda",
                       out_host=None, lse_host=None, staging=None, stream=None):
    """End-to-end forward from HOST tensors through ``moda_fwd_host``: the C
    call enqueues the host->device copies of the inputs into the device
    ``staging`` buffer, the forward and the device->host copies of out and
    lse; this function then waits for the stream.

    ``out_host`` / ``lse_host`` (pinned CPU tensors) are filled in place when
    given, else created (pinned). ``staging`` (a CUDA uint8 tensor of at
    least ``moda_fwd_host_staging_bytes`` bytes) is created when not given.
    Returns (out_host, lse_host)."""
    if kd is not None and kd.shape[2] == 0:
        kd = vd = None
    for t in (q, k, v, kd, vd, out_host, lse_host):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("moda_fwd_from_host takes contiguous host tensors")
    B, T, Hq, Hkv, d, Ld = _dims(q, k, kd)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dev = torch.device(device)
    need = moda_fwd_host_staging_bytes(B, T, Hq, Hkv, d, Ld, q.dtype)
    if staging is None:
        staging = torch.empty(need, dtype=torch.uint8, device=dev)
    if out_host is None:
        out_host = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if lse_host is None:
        lse_host = torch.empty((B, Hq, T), dtype=torch.float32, pin_memory=True)
    with torch.cuda.device(staging.device):
        st = _stream(stream)
        _check(_c_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(kd), _ptr(vd), B, T, Hq, Hkv, d, Ld,
                           _DTYPE[q.dtype], scale, _ptr(out_host), _ptr(lse_host), _ptr(staging),
                           staging.numel(), st), "moda_fwd_host")
        _check(_c_dev_status(st), "moda_fwd_host (stream)")
    return out_host, lse_host
