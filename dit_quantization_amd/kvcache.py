"""Python binding of include/kvcache.h: paged 8-bit caches of keys and values,
quantized as they are written, and read back (argument marshalling only, as in
dit_quantization_amd.int4; the entry points live in the same libnvfp4.so and
there is no fallback path).

A cache is the tuple (key codes, key scales, value codes, value scales): codes
int8 or float8_e4m3fn [pages, page_size, heads, dim], scales float32 [pages,
page_size, heads]; a value is scale * code.  Only the first dimension may be
strided (keys and values in one allocation).  Rows of keys and values are
tokens of a packed batch: rows cu[b] to cu[b + 1] - 1 belong to sequence b and
are its positions starts[b], starts[b] + 1, ...; position p lies in page
page_table[b, p // page_size].  Tensors live on the current device and calls
run on torch's current stream.

    cache = kvcache.new(pages, 64, heads, dim, dtype=torch.float8_e4m3fn)
    kvcache.write(k, v, cache, page_table, cu, starts)                # k, v [T, heads, dim]
    k, v = kvcache.read(cache, page_table, cu_all, tokens=total)      # bf16, everything the sequences hold
"""
import ctypes
import struct

import torch

from . import int4 as _i4
from . import nvfp4 as _nv

_P, _I, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class Tensor(ctypes.Structure):
    """kv8_tensor of include/kvcache.h."""
    _fields_ = [("codes", _P), ("scales", _P), ("code_stride", _I64), ("scale_stride", _I64), ("rows", _P),
                ("token_stride", _I64), ("head_stride", _I64), ("dim", _I64)]


class Places(ctypes.Structure):
    """kv8_places of include/kvcache.h."""
    _fields_ = [("page_table", _P), ("cu", _P), ("starts", _P), ("seqs", _I64), ("table_width", _I64),
                ("tokens", _I64), ("heads", _I64), ("pages", _I64), ("page_size", _I64)]


_TP, _PP = ctypes.POINTER(Tensor), ctypes.POINTER(Places)
SIGNATURES = {
    "kv8_write": (_I, [_TP, _TP, _PP, _I, _I, _P]),
    "kv8_read": (_I, [_TP, _TP, _PP, _I, _I, _P]),
}

_lib = None


def lib():
    """The loaded C library with this module's signatures (raises if it has not been built)."""
    global _lib
    if _lib is None:
        L = _nv.lib()
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def new(pages, page_size, heads, dim, value_dim=None, dtype=torch.int8, device="cuda"):
    """A cache of zeros (code 0, scale 0)."""
    _i4._code(_i4._BYTES, dtype, "cache")
    out = []
    for d in (dim, dim if value_dim is None else value_dim):
        out.append(torch.zeros(pages, page_size, heads, d, dtype=torch.uint8, device=device).view(dtype))
        out.append(torch.zeros(pages, page_size, heads, dtype=torch.float32, device=device))
    return tuple(out)


def _page_stride(t, page, what):
    """Elements from page to page of a tensor of pages of `page` elements, which are contiguous."""
    inner = 1
    for size, stride in zip(t.shape[:0:-1], t.stride()[:0:-1]):
        if size > 1 and stride != inner:
            raise ValueError(f"{what}: only the first dimension may be strided")
        inner *= size
    return t.stride(0) if t.shape[0] > 1 else page


def _refuse_cache(cache):
    got = ", ".join(f"{t.dtype} {tuple(t.shape)}" for t in cache)
    raise ValueError("a cache is (codes, scales) of keys and of values: int8 or float8_e4m3fn codes [pages, page_size, "
                     f"heads, dim] of one type that agree but for dim, float32 scales [pages, page_size, heads]; got {got}")


def _rows(t, shape, dtype, c, s, places, what):
    """The Tensor of a cache's tensor c with its scales s and of rows t [tokens, heads, dim]."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what} must be a {dtype} tensor of shape {tuple(shape)}; got {t.dtype} {tuple(t.shape)}")
    tokens, heads, dim = shape
    token, head, one = t.stride()
    if one != 1 and dim > 1:
        raise ValueError(f"{what}'s heads must be contiguous")
    page = places[1] * places[2]
    return _TENSOR(_PACK(c.data_ptr(), s.data_ptr(),
                         page * dim if c.is_contiguous() else _page_stride(c, page * dim, "codes"),
                         page if s.is_contiguous() else _page_stride(s, page, "scales"), t.data_ptr(),
                         token if tokens > 1 else 0, head if heads > 1 else 0, dim))


# (What every call does is kept short, as in int4: a decode step's call costs
# the host more than the GPU.)
_PACK, _PACK_PLACES = struct.Struct("8q").pack, struct.Struct("9q").pack
_TENSOR, _PLACES = Tensor.from_buffer_copy, Places.from_buffer_copy
_F32, _I32 = torch.float32, torch.int32


def _call(fn, cache, k, v, page_table, cu, starts):
    """Checks a cache, rows of keys and values [tokens, heads, dim] and the tables, and calls fn."""
    kc, ks, vc, vs = cache
    held, vheld = kc.shape, vc.shape
    qt = _i4._BYTES.get(kc.dtype)
    places = held[:3]
    if (qt is None or len(held) != 4 or len(vheld) != 4 or vheld[:3] != places or vc.dtype != kc.dtype
            or ks.shape != places or vs.shape != places or ks.dtype != _F32 or vs.dtype != _F32):
        _refuse_cache(cache)
    dtype, tokens = k.dtype, k.shape[0]
    pages, size, heads = places
    keys = _rows(k, (tokens, heads, held[3]), dtype, kc, ks, places, "keys")
    values = _rows(v, (tokens, heads, vheld[3]), dtype, vc, vs, places, "values")
    table = page_table.shape
    if page_table.dtype != _I32 or len(table) != 2 or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 tensor [sequences, pages of a sequence]")
    seqs, width = table
    if cu.dtype != _I32 or cu.shape != (seqs + 1,) or not cu.is_contiguous():
        raise ValueError(f"cu must be a contiguous int32 tensor of shape {(seqs + 1,)}")
    first = None
    if starts is not None:
        if starts.dtype != _I32 or starts.shape != (seqs,) or not starts.is_contiguous():
            raise ValueError(f"starts must be a contiguous int32 tensor of shape {(seqs,)}")
        first = starts.data_ptr()
    stream = _i4._stream(k, v, kc, ks, vc, vs)
    _i4._stream(page_table, cu, starts)
    at = _PLACES(_PACK_PLACES(page_table.data_ptr(), cu.data_ptr(), first or 0, seqs, width, tokens, heads, pages, size))
    _i4._done(fn, getattr(_lib or lib(), fn)(keys, values, at, _i4._FLOATS[dtype], qt, stream))


def write(k, v, cache, page_table, cu, starts=None):
    """Quantizes keys and values [tokens, heads, dim] (fp32 or bf16) into the cache.

    starts: int32 [sequences], the positions of the sequences' first rows (None:
    0).  Rows that belong to no sequence, and positions without a page (past the
    table, or a page number that is no page of the cache, as -1), are not
    written."""
    _i4._code(_i4._FLOATS, k.dtype, "keys")
    if k.dim() != 3:
        raise ValueError("keys must be a tensor [tokens, heads, dim]")
    _call("kv8_write", cache, k, v, page_table, cu, starts)


def read(cache, page_table, cu, starts=None, tokens=None, out_dtype=torch.bfloat16, out=None):
    """Keys and values [tokens, heads, dim] of fp32 or bf16, read from the cache.

    tokens: how many rows to return; at least cu's last entry to have them all.
    Positions without a page give zeros.  out: the two tensors to write instead,
    whose rows that belong to no sequence are left as they are (new tensors'
    are unspecified)."""
    if out is None:
        if tokens is None:
            raise ValueError("read needs tokens, the number of rows, or out")
        _i4._code(_i4._FLOATS, out_dtype, "output")
        held, vheld = cache[0].shape, cache[2].shape
        if len(held) != 4 or len(vheld) != 4:
            _refuse_cache(cache)
        device = cache[0].device
        out = (torch.empty(tokens, held[2], held[3], dtype=out_dtype, device=device),
               torch.empty(tokens, vheld[2], vheld[3], dtype=out_dtype, device=device))
    else:
        if out[0].dim() != 3 or (tokens is not None and out[0].shape[0] != tokens):
            raise ValueError("out must be two tensors [tokens, heads, dim]")
        _i4._code(_i4._FLOATS, out[0].dtype, "output")
    _call("kv8_read", cache, *out, page_table, cu, starts)
    return out
