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
    if t.is_contiguous():
        return page
    inner = 1
    for size, stride in zip(t.shape[:0:-1], t.stride()[:0:-1]):
        if size > 1 and stride != inner:
            raise ValueError(f"{what}: only the first dimension may be strided")
        inner *= size
    return t.stride(0) if t.shape[0] > 1 else page


def _call(fn, cache, rows, page_table, cu, starts):
    """Checks a cache, rows of keys and values [tokens, heads, dim] and the tables, and calls fn."""
    kc, ks, vc, vs = cache
    qt = _i4._BYTES.get(kc.dtype)
    if qt is None or kc.dim() != 4 or vc.dim() != 4 or vc.dtype != kc.dtype or kc.shape[:3] != vc.shape[:3]:
        raise ValueError("a cache's codes are two int8 or float8_e4m3fn tensors [pages, page_size, heads, dim] that agree "
                         f"but for dim; got {kc.dtype} {tuple(kc.shape)}, {vc.dtype} {tuple(vc.shape)}")
    dt = rows[0].dtype
    tokens = rows[0].shape[0]
    pages, size, heads, _ = kc.shape
    tensors = []
    for c, s, t, what in ((kc, ks, rows[0], "keys"), (vc, vs, rows[1], "values")):
        dim = c.shape[3]
        if s.dtype != torch.float32 or s.shape != c.shape[:3]:
            raise ValueError(f"a cache's scales are float32 tensors of shape {tuple(c.shape[:3])}; got {s.dtype} "
                             f"{tuple(s.shape)}")
        if t.shape != (tokens, heads, dim) or t.dtype != dt:
            raise ValueError(f"{what} must be a {dt} tensor of shape {(tokens, heads, dim)}; got {t.dtype} "
                             f"{tuple(t.shape)}")
        token, head, one = t.stride()
        if one != 1 and dim > 1:
            raise ValueError(f"{what}'s heads must be contiguous")
        tensors.append(Tensor(c.data_ptr(), s.data_ptr(), _page_stride(c, size * heads * dim, "codes"),
                              _page_stride(s, size * heads, "scales"), t.data_ptr(), token if tokens > 1 else 0,
                              head if heads > 1 else 0, dim))
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 tensor [sequences, pages of a sequence]")
    seqs, width = page_table.shape
    for t, n, what in ((cu, seqs + 1, "cu"), (starts, seqs, "starts")):
        if t is not None and (t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous()):
            raise ValueError(f"{what} must be a contiguous int32 tensor of shape {(n,)}")
    stream = _i4._stream(rows[0], rows[1], kc, ks, vc, vs)
    _i4._stream(page_table, cu, starts)
    places = Places(page_table.data_ptr(), cu.data_ptr(), _i4._ptr(starts), seqs, width, tokens, heads, pages, size)
    _i4._done(fn, getattr(lib(), fn)(tensors[0], tensors[1], places, _i4._FLOATS[dt], qt, stream))


def write(k, v, cache, page_table, cu, starts=None):
    """Quantizes keys and values [tokens, heads, dim] (fp32 or bf16) into the cache.

    starts: int32 [sequences], the positions of the sequences' first rows (None:
    0).  Rows that belong to no sequence, and positions without a page (past the
    table, or a page number that is no page of the cache, as -1), are not
    written."""
    _i4._code(_i4._FLOATS, k.dtype, "keys")
    if k.dim() != 3:
        raise ValueError("keys must be a tensor [tokens, heads, dim]")
    _call("kv8_write", cache, (k, v), page_table, cu, starts)


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
        kc, _, vc, _ = cache
        if kc.dim() != 4 or vc.dim() != 4:
            raise ValueError("a cache's codes are two tensors [pages, page_size, heads, dim]")
        out = (torch.empty(tokens, kc.shape[2], kc.shape[3], dtype=out_dtype, device=kc.device),
               torch.empty(tokens, vc.shape[2], vc.shape[3], dtype=out_dtype, device=vc.device))
    else:
        if out[0].dim() != 3 or (tokens is not None and out[0].shape[0] != tokens):
            raise ValueError("out must be two tensors [tokens, heads, dim]")
        _i4._code(_i4._FLOATS, out[0].dtype, "output")
    _call("kv8_read", cache, out, page_table, cu, starts)
    return out
