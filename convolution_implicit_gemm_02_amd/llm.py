"""ctypes binding of the decoder-step operators (include/cbs_llm.h), same entry-point names.

    norm = llm.make_rms_desc(4096, dtype=llm.CBS_BF16, out_dtype=llm.CBS_I8)
    llm.cbs_rms_norm(norm, x, weight, codes, residual=r, residual_out=r, out_scale=scale)
    llm.cbs_w4_linear(llm.make_w4_desc(4096, 6144, 128, dtype=llm.CBS_I8), codes, w_codes, w_scales, qkv, x_scale=scale)

Calls whose arguments are in order go through the extension module _llm_bind (csrc/llm_bind.cpp), all others through the checks
here, which say what is wrong.

Device buffers are torch tensors, which give sizes and strides (the innermost axis has to be dense); streams are
``torch.cuda.Stream`` objects, raw handles or None (torch's current stream).  Types, shapes and devices are checked
before the call (ValueError); what the library itself refuses raises CbsError.  Calls only enqueue: lengths, page
tables and slots stay on the GPU, so a call can be captured into a graph.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _llm_bind
from .cbs import (CBS_EDEVICE, CBS_EINVAL, CBS_ELAUNCH, CBS_ENOMEM, CBS_EUNSUPPORTED, CBS_F32, CBS_I8, CBS_OK, CbsError, _check,  # noqa: F401
                  lib)

CBS_F16 = 3
CBS_BF16 = 4
CBS_RMS_MAX_DIM = 65536

_I, _L, _F, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_TORCH = {CBS_F32: torch.float32, CBS_F16: torch.float16, CBS_BF16: torch.bfloat16, CBS_I8: torch.int8}


class cbs_rms_desc(ctypes.Structure):
    _fields_ = [("dim", _I), ("dtype", _I), ("out_dtype", _I), ("weight_dtype", _I), ("eps", _F)]


class cbs_w4_desc(ctypes.Structure):
    _fields_ = [("k", _I), ("n", _I), ("group", _I), ("dtype", _I), ("out_dtype", _I), ("scale_dtype", _I)]


class cbs_kv_desc(ctypes.Structure):
    _fields_ = [("heads", _I), ("head_dim", _I), ("page_size", _I), ("dtype", _I), ("cache_dtype", _I), ("read_dtype", _I)]


class cbs_attn_desc(ctypes.Structure):
    _fields_ = [("heads", _I), ("kv_heads", _I), ("head_dim", _I), ("page_size", _I), ("dtype", _I), ("cache_dtype", _I), ("causal", _I), ("window", _I),
                ("scale", _F), ("max_seqs", _I)]


class cbs_rms_args(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "residual", "weight", "out", "residual_out", "out_scale")] + \
               [(n, _L) for n in ("rows", "x_stride", "residual_stride", "out_stride", "residual_out_stride")]


class cbs_w4_args(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("x", "x_scale", "codes", "scales", "zeros", "out")] + [(n, _L) for n in ("rows", "x_stride", "out_stride")]


class cbs_kv_args(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k", "v", "slots", "k_cache", "v_cache", "k_scale", "v_scale")] + \
               [(n, _L) for n in ("tokens", "pages", "k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride")]


class cbs_attn_args(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("q", "q_start", "kv_len", "table", "k_cache", "v_cache", "k_scale", "v_scale", "out")] + \
               [(n, _L) for n in ("tokens", "pages", "q_token_stride", "q_head_stride", "out_token_stride", "out_head_stride", "table_stride")] + \
               [(n, _I) for n in ("seqs", "columns", "max_new", "max_kv")]


# Every symbol the header declares, with (restype, argtypes).  A call's arguments go as packed bytes of the structure.
_SIGNATURES = {
    "cbs_rms_norm": (_I, [ctypes.POINTER(cbs_rms_desc), ctypes.c_char_p, _P]),
    "cbs_w4_linear": (_I, [ctypes.POINTER(cbs_w4_desc), ctypes.c_char_p, _P]),
    "cbs_kv_write": (_I, [ctypes.POINTER(cbs_kv_desc), ctypes.c_char_p, _P]),
    "cbs_kv_read": (_I, [ctypes.POINTER(cbs_kv_desc), ctypes.c_char_p, _P]),
    "cbs_attn_create": (_I, [ctypes.POINTER(cbs_attn_desc), ctypes.POINTER(_P)]),
    "cbs_attn_run": (_I, [_P, ctypes.c_char_p, _P]),
    "cbs_attn_destroy": (None, [_P]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.restype, _fn.argtypes = _res, _args

_llm_bind.setup(*(ctypes.cast(getattr(lib, _name), _P).value for _name in ("cbs_rms_norm", "cbs_w4_linear", "cbs_kv_write", "cbs_kv_read", "cbs_attn_run")))

# The argument structures: pointers and 64-bit counts, then 32-bit ones, without padding.
_pack_rms = struct.Struct("=6Q5q").pack
_pack_w4 = struct.Struct("=6Q3q").pack
_pack_kv = struct.Struct("=7Q6q").pack
_pack_attn = struct.Struct("=9Q7q4i").pack


def make_rms_desc(dim, dtype=CBS_BF16, out_dtype=None, weight_dtype=None, eps=1e-6) -> cbs_rms_desc:
    return cbs_rms_desc(dim, dtype, dtype if out_dtype is None else out_dtype, dtype if weight_dtype is None else weight_dtype, float(eps))


def make_w4_desc(k, n, group=128, dtype=CBS_BF16, out_dtype=CBS_BF16, scale_dtype=CBS_F16) -> cbs_w4_desc:
    return cbs_w4_desc(k, n, group, dtype, out_dtype, scale_dtype)


def make_kv_desc(heads, head_dim, page_size, dtype=CBS_BF16, cache_dtype=CBS_I8, read_dtype=None) -> cbs_kv_desc:
    return cbs_kv_desc(heads, head_dim, page_size, dtype, cache_dtype, dtype if read_dtype is None else read_dtype)


def make_attn_desc(heads, kv_heads, head_dim, page_size, dtype=CBS_BF16, cache_dtype=CBS_I8, causal=True, window=0, scale=None, max_seqs=1) -> cbs_attn_desc:
    return cbs_attn_desc(heads, kv_heads, head_dim, page_size, dtype, cache_dtype, int(causal), window, float(head_dim) ** -0.5 if scale is None else float(scale),
                         max_seqs)


def _stream(stream, dev) -> int:
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    return stream if isinstance(stream, int) else int(stream.cuda_stream)


def _ptr(t, what, dtype, shape, dev):
    """Address of a tensor of this type and shape on GPU `dev`, dense in its last axis."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or (t.stride(-1) != 1 and t.shape[-1] > 1):
        _wrong(t, what, dtype, shape, dev)
    return t.data_ptr()


def _dense(t, what, dtype, shape, dev):
    """The same for a tensor that is dense in every axis."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _wrong(t, what, dtype, shape, dev, True)
    return t.data_ptr()


def _wrong(t, what, dtype, shape, dev, dense=False):
    said = "%s %s, strides %s on %s" % (t.dtype, tuple(t.shape), t.stride(), t.device)
    raise ValueError("%s: %s; wanted %s %s, dense %s, on cuda:%d" % (what, said, dtype, tuple(shape), "throughout" if dense else "in its last axis", dev))


def _device(t, what) -> int:
    if not t.is_cuda:
        raise ValueError("%s is not on a GPU (device %s)" % (what, t.device))
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError("%s is on cuda:%d, which is not the current device" % (what, dev))
    return dev


def cbs_rms_norm(desc: cbs_rms_desc, x, weight, out, residual=None, residual_out=None, out_scale=None, stream=None) -> None:
    """x, residual, residual_out, out: [rows][dim]; weight: [dim]; out_scale: float32 [rows], for int8 output."""
    if stream is None:
        status = _llm_bind.rms_norm(desc, x, weight, out, residual, residual_out, out_scale)
        if status >= 0:
            return _check(status, "cbs_rms_norm")
    dev = _device(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x: wanted [rows][dim], got %s" % (tuple(shape),))
    rows, dim = shape
    if dim != desc.dim:
        raise ValueError("x: rows of %d, the descriptor has %d" % (dim, desc.dim))
    kind = _TORCH.get(desc.dtype)
    _check(lib.cbs_rms_norm(desc, _pack_rms(
        _ptr(x, "x", kind, shape, dev), 0 if residual is None else _ptr(residual, "residual", kind, shape, dev),
        _dense(weight, "weight", _TORCH.get(desc.weight_dtype), (dim,), dev), _ptr(out, "out", _TORCH.get(desc.out_dtype), shape, dev),
        0 if residual_out is None else _ptr(residual_out, "residual_out", kind, shape, dev),
        0 if out_scale is None else _dense(out_scale, "out_scale", torch.float32, (rows,), dev),
        rows, x.stride(0), 0 if residual is None else residual.stride(0), out.stride(0), 0 if residual_out is None else residual_out.stride(0)),
        _stream(stream, dev)), "cbs_rms_norm")


def cbs_w4_linear(desc: cbs_w4_desc, x, codes, scales, out, zeros=None, x_scale=None, stream=None) -> None:
    """x: [rows][k]; codes: uint8 [n][round_up(ceil(k / 2), 16)]; scales, zeros (uint8): [ceil(k / group)][n]; out: [rows][n]; x_scale: float32 [rows], for
    int8 rows."""
    if stream is None:
        status = _llm_bind.w4_linear(desc, x, codes, scales, out, zeros, x_scale)
        if status >= 0:
            return _check(status, "cbs_w4_linear")
    dev = _device(x, "x")
    k, n = desc.k, desc.n
    if len(x.shape) != 2 or desc.group < 1:
        raise ValueError("x: wanted [rows][k], got %s; group %d" % (tuple(x.shape), desc.group))
    rows = x.shape[0]
    per = (-(-k // desc.group), n)
    _check(lib.cbs_w4_linear(desc, _pack_w4(
        _ptr(x, "x", _TORCH.get(desc.dtype), (rows, k), dev), 0 if x_scale is None else _dense(x_scale, "x_scale", torch.float32, (rows,), dev),
        _dense(codes, "codes", torch.uint8, (n, (k + 31) // 32 * 16), dev), _dense(scales, "scales", _TORCH.get(desc.scale_dtype), per, dev),
        0 if zeros is None else _dense(zeros, "zeros", torch.uint8, per, dev), _ptr(out, "out", _TORCH.get(desc.out_dtype), (rows, n), dev),
        rows, x.stride(0), out.stride(0)), _stream(stream, dev)), "cbs_w4_linear")


def _kv(fast, fn, name, desc, kind, k, v, slots, k_cache, v_cache, k_scale, v_scale, stream):
    if stream is None:
        status = fast(desc, k, v, slots, k_cache, v_cache, k_scale, v_scale)
        if status >= 0:
            return _check(status, name)
    dev = _device(slots, "slots")
    heads, dim, page = desc.heads, desc.head_dim, desc.page_size
    tokens, pages = slots.shape[0], k_cache.shape[0]
    shape, kept = (tokens, heads, dim), _TORCH.get(desc.cache_dtype)
    _check(fn(desc, _pack_kv(
        _ptr(k, "k", kind, shape, dev), _ptr(v, "v", kind, shape, dev), _dense(slots, "slots", torch.int64, (tokens,), dev),
        _dense(k_cache, "k_cache", kept, (pages, heads, page, dim), dev), _dense(v_cache, "v_cache", kept, (pages, heads, dim, page), dev),
        0 if k_scale is None else _dense(k_scale, "k_scale", torch.float32, (pages, heads, page), dev),
        0 if v_scale is None else _dense(v_scale, "v_scale", torch.float32, (pages, heads, page), dev),
        tokens, pages, k.stride(0), k.stride(1), v.stride(0), v.stride(1)), _stream(stream, dev)), name)


def cbs_kv_write(desc: cbs_kv_desc, k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, stream=None) -> None:
    """k, v: [tokens][heads][head_dim]; slots: int64 [tokens]; k_cache: [pages][heads][page_size][head_dim]; v_cache: [pages][heads][head_dim][page_size];
    scales: float32 [pages][heads][page_size], for an int8 cache."""
    _kv(_llm_bind.kv_write, lib.cbs_kv_write, "cbs_kv_write", desc, _TORCH.get(desc.dtype), k, v, slots, k_cache, v_cache, k_scale, v_scale, stream)


def cbs_kv_read(desc: cbs_kv_desc, slots, k_cache, v_cache, k, v, k_scale=None, v_scale=None, stream=None) -> None:
    """The other way: into k and v, of desc.read_dtype."""
    _kv(_llm_bind.kv_read, lib.cbs_kv_read, "cbs_kv_read", desc, _TORCH.get(desc.read_dtype), k, v, slots, k_cache, v_cache, k_scale, v_scale, stream)


class Attn:
    """Handle of the attention operator (a cbs_attn*), destroyed on garbage collection."""

    def __init__(self, handle: int, desc: cbs_attn_desc):
        self.handle = handle
        self.desc = cbs_attn_desc.from_buffer_copy(desc)
        self.heads, self.kv_heads, self.head_dim, self.page_size = desc.heads, desc.kv_heads, desc.head_dim, desc.page_size
        self.kind, self.kept = _TORCH[desc.dtype], _TORCH[desc.cache_dtype]

    def __del__(self):
        if getattr(self, "handle", 0) and lib is not None:
            lib.cbs_attn_destroy(self.handle)
            self.handle = 0


def cbs_attn_create(desc: cbs_attn_desc) -> Attn:
    h = _P()
    _check(lib.cbs_attn_create(desc, ctypes.byref(h)), "cbs_attn_create")
    return Attn(h.value, desc)


def cbs_attn_destroy(attn: Attn) -> None:
    if attn.handle:
        lib.cbs_attn_destroy(attn.handle)
        attn.handle = 0


def cbs_attn_run(attn: Attn, q, q_start, kv_len, table, k_cache, v_cache, out, k_scale=None, v_scale=None, max_new=None, max_kv=None, stream=None) -> None:
    """q, out: [tokens][heads][head_dim]; q_start: int32 [seqs + 1]; kv_len: int32 [seqs]; table: int32 [seqs][columns]; caches and scales as in
    cbs_kv_write.  max_new, max_kv: most new tokens and most tokens of a sequence, which choose how the work is split: say them where
    they are known.  None: as many as there can be, but one new token where there are as many as sequences (32 of them over 8192
    tokens of int8: 90 us, and 340 as if one could have all)."""
    if stream is None:
        status = _llm_bind.attn_run(attn.handle, attn.desc, q, q_start, kv_len, table, k_cache, v_cache, out, k_scale, v_scale, max_new, max_kv)
        if status >= 0:
            return _check(status, "cbs_attn_run")
    dev = _device(q, "q")
    heads, dim, page = attn.heads, attn.head_dim, attn.page_size
    seqs, columns = table.shape
    tokens, pages = q.shape[0], k_cache.shape[0]
    shape, cache, per = (tokens, heads, dim), (pages, attn.kv_heads), (pages, attn.kv_heads, page)
    _check(lib.cbs_attn_run(attn.handle, _pack_attn(
        _ptr(q, "q", attn.kind, shape, dev), _dense(q_start, "q_start", torch.int32, (seqs + 1,), dev), _dense(kv_len, "kv_len", torch.int32, (seqs,), dev),
        _ptr(table, "table", torch.int32, (seqs, columns), dev), _dense(k_cache, "k_cache", attn.kept, cache + (page, dim), dev),
        _dense(v_cache, "v_cache", attn.kept, cache + (dim, page), dev), 0 if k_scale is None else _dense(k_scale, "k_scale", torch.float32, per, dev),
        0 if v_scale is None else _dense(v_scale, "v_scale", torch.float32, per, dev), _ptr(out, "out", attn.kind, shape, dev),
        tokens, pages, q.stride(0), q.stride(1), out.stride(0), out.stride(1), table.stride(0), seqs, columns,
        (1 if tokens == seqs else tokens) if max_new is None else max_new, min(columns * page, 2**31 - 1) if max_kv is None else max_kv), _stream(stream, dev)), "cbs_attn_run")
