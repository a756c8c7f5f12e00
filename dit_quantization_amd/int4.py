"""Python binding of include/int4.h: group-scaled 4-bit integer weights and
8-bit activations (argument marshalling only, as in dit_quantization_amd.nvfp4;
the entry points live in the same libnvfp4.so and there is no fallback path).

A weight is the triple (codes uint8 [N, K/2], scales bfloat16 [N, G], zeros
uint8 [N, G] or None for a symmetric one) with G = ceil(K / group_size); its
value is scale * (code - zero), zero = 8 where zeros is None.  Tensors live on
the current device and calls run on torch's current stream.

    codes, scales, zeros = int4.quantize(w)                       # w [N, K]
    xq, xs, res = int4.rmsnorm_quant8(x, gain, residual=res)      # x [M, K]
    y = int4.gemv_w4a8(xq, xs, codes, scales, zeros)              # bf16 [M, N], M <= 16
    y = int4.gemv_w4a16(x, codes, scales, zeros)                  # bf16 activations
"""
import ctypes
import math

import torch

from . import nvfp4 as _nv

F32, BF16, I8, E4M3 = 0, 1, 2, 3
GROUP_SIZES = (32, 64, 128)

_P, _I, _I64, _D = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_double
SIGNATURES = {
    "int4_quantize": (_I, [_P, _I, _I64, _I64, _I, _P, _P, _P, _P]),
    "int4_dequant": (_I, [_P, _P, _P, _I64, _I64, _I, _P, _I, _P]),
    "int4_gemv_w4a16": (_I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _P, _I, _P]),
    "int4_gemv_w4a8": (_I, [_P, _I, _P, _I, _P, _P, _P, _I, _I64, _I64, _I64, _P, _I, _P]),
    "int4_rmsnorm_quant8": (_I, [_P, _I, _I64, _P, _I, _I64, _P, _I, _D, _I64, _I64, _I, _I, _P, _P, _P, _P]),
}
_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_BYTES = {torch.int8: I8, torch.float8_e4m3fn: E4M3}

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


# A decode call costs the host about as much as the GPU, so what every call
# does is kept short: torch's own calls for the current device and stream, and
# checks by attribute without helper objects.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _ptr(t):
    return None if t is None else t.data_ptr()


def _code(table, dtype, what):
    code = table.get(dtype)
    if code is None:
        raise ValueError(f"unsupported {what} dtype {dtype}; expected one of {', '.join(str(d) for d in table)}")
    return code


def _stream(a, b=None, c=None, d=None, e=None, f=None):
    """The current stream of the current device, on which all the tensors have to be.

    (A stream that is being captured is refused by the library, before it
    launches anything.)"""
    dev = a.get_device()
    if (dev < 0 or dev != _current_device() or (b is not None and b.get_device() != dev)
            or (c is not None and c.get_device() != dev) or (d is not None and d.get_device() != dev)
            or (e is not None and e.get_device() != dev) or (f is not None and f.get_device() != dev)):
        where = ", ".join(str(t.device) for t in (a, b, c, d, e, f) if t is not None)
        raise ValueError(f"tensors must be on the current GPU; got them on {where}")
    return _raw_stream(dev)


def _done(fn, status):
    if status:
        _nv._check(fn, status)


def _contiguous(t):
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")


def _matrix(t, what):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    return shape


def _given(out, shape, dtype, what="out"):
    if out.shape != shape or out.dtype != dtype or not out.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return out


def _groups(cols, group_size):
    if group_size not in GROUP_SIZES:
        raise ValueError(f"group_size={group_size}: expected one of {GROUP_SIZES}")
    return -(-cols // group_size)


def _check_weight(codes, scales, zeros, group_size):
    """(N, K, G) of a packed weight, whose shapes and types have to agree."""
    N, half = _matrix(codes, "codes")
    want = (N, _groups(2 * half, group_size))
    if (codes.dtype != torch.uint8 or scales.dtype != torch.bfloat16 or scales.shape != want
            or (zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != want))):
        got = ", ".join(f"{t.dtype} {tuple(t.shape)}" for t in (codes, scales, zeros) if t is not None)
        raise ValueError("a packed weight is uint8 codes [N, K/2], bfloat16 scales [N, G] and uint8 zeros [N, G] or "
                         f"None, G = {want[1]} for groups of {group_size}; got {got}")
    if not (codes.is_contiguous() and scales.is_contiguous() and (zeros is None or zeros.is_contiguous())):
        raise ValueError("tensors must be contiguous")
    return N, 2 * half, want[1]


def quantize(w, group_size=128, symmetric=False, out=None):
    """Group-scaled 4-bit quantization of a [N, K] fp32/bf16 GPU tensor.

    Returns (codes uint8 [N, K/2], scales bfloat16 [N, G], zeros uint8 [N, G],
    or None where symmetric).  K must be a multiple of 32; the last group of a
    row may be short.  out: the three tensors to write instead."""
    N, K = _matrix(w, "w")
    dt = _code(_FLOATS, w.dtype, "weight")
    G = _groups(K, group_size)
    _contiguous(w)
    if out is None:
        stream = _stream(w)
        codes = torch.empty(N, K // 2, dtype=torch.uint8, device=w.device)
        scales = torch.empty(N, G, dtype=torch.bfloat16, device=w.device)
        zeros = None if symmetric else torch.empty(N, G, dtype=torch.uint8, device=w.device)
    else:
        codes, scales, zeros = out
        if (zeros is None) != bool(symmetric):
            raise ValueError("out's zeros must be None exactly where the quantization is symmetric")
        _given(codes, (N, K // 2), torch.uint8, "out's codes")
        _given(scales, (N, G), torch.bfloat16, "out's scales")
        if zeros is not None:
            _given(zeros, (N, G), torch.uint8, "out's zeros")
        stream = _stream(w, codes, scales, zeros)
    _done("int4_quantize", lib().int4_quantize(w.data_ptr(), dt, N, K, group_size, codes.data_ptr(), scales.data_ptr(),
                                               _ptr(zeros), stream))
    return codes, scales, zeros


def dequant(codes, scales, zeros=None, group_size=128, out_dtype=torch.float32, out=None):
    """scale * (code - zero) as a [N, K] fp32 (exact) or bf16 tensor."""
    N, K, _ = _check_weight(codes, scales, zeros, group_size)
    if out is None:
        dt = _code(_FLOATS, out_dtype, "output")
        stream = _stream(codes, scales, zeros)
        out = torch.empty(N, K, dtype=out_dtype, device=codes.device)
    else:
        dt = _code(_FLOATS, out.dtype, "output")
        _given(out, (N, K), out.dtype)
        stream = _stream(codes, scales, zeros, out)
    _done("int4_dequant", lib().int4_dequant(codes.data_ptr(), scales.data_ptr(), _ptr(zeros), N, K, group_size,
                                             out.data_ptr(), dt, stream))
    return out


def _product(x, codes, scales, zeros, group_size, out_dtype, out, x_scales=None):
    """Shape checks and output of a decode product: (M, N, K, out, its dtype code, stream)."""
    N, K, G = _check_weight(codes, scales, zeros, group_size)
    M, Kx = _matrix(x, "x")
    if Kx != K:
        raise ValueError(f"x has {Kx} columns, the weight {K}")
    if x_scales is not None:
        if x_scales.dtype != torch.float32 or (x_scales.shape != (M, 1) and x_scales.shape != (M, G)):
            raise ValueError(f"x_scales must be a float32 tensor of shape {(M, 1)} or {(M, G)}; got {x_scales.dtype} "
                             f"{tuple(x_scales.shape)}")
        _contiguous(x_scales)
    _contiguous(x)
    if out is None:
        dt = _code(_FLOATS, out_dtype, "output")
        stream = _stream(x, codes, scales, zeros, x_scales)
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    else:
        dt = _code(_FLOATS, out.dtype, "output")
        _given(out, (M, N), out.dtype)
        stream = _stream(x, codes, scales, zeros, x_scales, out)
    return M, N, K, out, dt, stream


def gemv_w4a16(x, codes, scales, zeros=None, group_size=128, out_dtype=torch.bfloat16, out=None):
    """y = x W^T for bf16 x [M, K] (M <= 16) and a packed weight [N, K]."""
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    M, N, K, out, dt, stream = _product(x, codes, scales, zeros, group_size, out_dtype, out)
    _done("int4_gemv_w4a16", lib().int4_gemv_w4a16(x.data_ptr(), codes.data_ptr(), scales.data_ptr(), _ptr(zeros),
                                                   group_size, M, N, K, out.data_ptr(), dt, stream))
    return out


def gemv_w4a8(x, x_scales, codes, scales, zeros=None, group_size=128, out_dtype=torch.bfloat16, out=None):
    """y = (x_scales x) W^T for int8 or float8_e4m3fn x [M, K] (M <= 16).

    x_scales: fp32 [M, 1] (one scale a row), or [M, G] (one for each of the
    weight's groups), as rmsnorm_quant8 returns them.  Where G is 1 both mean
    the same."""
    xt = _code(_BYTES, x.dtype, "activation")
    M, N, K, out, dt, stream = _product(x, codes, scales, zeros, group_size, out_dtype, out, x_scales)
    _done("int4_gemv_w4a8", lib().int4_gemv_w4a8(x.data_ptr(), xt, x_scales.data_ptr(),
                                                 0 if x_scales.shape[1] == 1 else group_size, codes.data_ptr(),
                                                 scales.data_ptr(), _ptr(zeros), group_size, M, N, K,
                                                 out.data_ptr(), dt, stream))
    return out


def _row_stride(t, cols, what):
    if t.is_contiguous():
        return cols
    if t.stride(1) != 1 and cols > 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else cols


def rmsnorm_quant8(x, weight=None, residual=None, eps=1e-6, group_size=0, out_dtype=torch.int8, out=None):
    """RMS norm of x [M, K] (+ residual), as 8-bit codes with scales.

    Returns (codes int8 or float8_e4m3fn [M, K], scales fp32 [M, 1], or
    [M, ceil(K / group_size)] with group_size 32, 64 or 128, and the sum
    x + residual in the residual's type, or None without a residual).  x is
    fp32 or bf16, the residual of x's type or fp32, the weight [K] fp32 or
    bf16 (None: ones).  x and the residual may have any row stride of whole
    16-byte units (slices of wider tensors).
    out: the three tensors to write instead; the third may be the residual or
    x itself where type and layout agree (the sum in place)."""
    M, K = shape = _matrix(x, "x")
    xdt = x.dtype
    xt, qt = _code(_FLOATS, xdt, "x"), _code(_BYTES, out_dtype if out is None else out[0].dtype, "output")
    if not 0 <= eps < math.inf:
        raise ValueError(f"eps={eps}: expected a finite value >= 0")
    group_size = group_size or 0
    G = _groups(K, group_size) if group_size else 1
    xs, rt, rs, wt = _row_stride(x, K, "x"), F32, 0, F32
    if residual is not None:
        rdt = residual.dtype
        if residual.shape != shape or (rdt != xdt and rdt != torch.float32):
            raise ValueError(f"residual must have x's shape {(M, K)} and its type or float32")
        rt, rs = _FLOATS[rdt], _row_stride(residual, K, "residual")
    if weight is not None:
        wt = _code(_FLOATS, weight.dtype, "weight")
        if weight.shape != (K,) or not weight.is_contiguous():
            raise ValueError(f"weight must be a contiguous tensor of shape {(K,)}")
    if out is None:
        stream = _stream(x, weight, residual)
        codes = torch.empty(M, K, dtype=out_dtype, device=x.device)
        scales = torch.empty(M, G, dtype=torch.float32, device=x.device)
        h = None if residual is None else torch.empty(M, K, dtype=rdt, device=x.device)
    else:
        codes, scales, h = out
        if (h is None) != (residual is None):
            raise ValueError("out's sum must be None exactly where there is no residual")
        _given(codes, (M, K), codes.dtype, "out's codes")
        _given(scales, (M, G), torch.float32, "out's scales")
        if h is not None:
            _given(h, (M, K), residual.dtype, "out's sum")
        stream = _stream(x, weight, residual, codes, scales, h)
    _done("int4_rmsnorm_quant8",
          lib().int4_rmsnorm_quant8(x.data_ptr(), xt, xs, _ptr(residual), rt, rs, _ptr(weight), wt, eps, M, K,
                                    group_size, qt, codes.data_ptr(), scales.data_ptr(), _ptr(h), stream))
    return codes, scales, h
