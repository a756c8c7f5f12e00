"""Python binding of include/fp8.h: FP8 weights scaled by 128 x 128 blocks and
8-bit activations scaled by groups of columns (argument marshalling only, as in
dit_quantization_amd.int4; the entry points live in the same libnvfp4.so and
there is no fallback path).

A weight is the pair (codes float8_e4m3fn [N, K], scales float32 [ceil(N / 128),
ceil(K / 128)]); activations are the pair (codes [M, K], scales float32 [M,
ceil(K / group)]), as quantize_act and int4.rmsnorm_quant8 return them; a value
is scale * code.  Tensors live on the current device and calls run on torch's
current stream.

    codes, scales = fp8.quantize(w)                                  # w [N, K]
    xq, xs, _ = int4.rmsnorm_quant8(x, gain, group_size=128, out_dtype=torch.float8_e4m3fn)
    h = fp8.gemm(xq, xs, codes, scales)                              # bf16 [M, N], any M
    aq, as_ = fp8.quantize_act(h[:, F:], gate=h[:, :F])              # SiLU(gate) x, E4M3 in groups of 128
"""
import ctypes

import torch

from . import int4 as _i4
from . import nvfp4 as _nv

BLOCK = 128

_P, _I, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
SIGNATURES = {
    "fp8_quantize": (_I, [_P, _I, _I64, _I64, _I64, _P, _P, _P]),
    "fp8_quantize_act": (_I, [_P, _I64, _P, _I64, _I, _I64, _I64, _I, _I, _P, _P, _P]),
    "fp8_gemm": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _I, _P]),
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


def quantize(w, out=None):
    """E4M3 codes and block scales of a [N, K] fp32/bf16 GPU tensor.

    Returns (codes float8_e4m3fn [N, K], scales float32 [ceil(N / 128),
    ceil(K / 128)]).  K must be a multiple of 16; w may have any row stride of
    whole 16-byte units.  out: the two tensors to write instead."""
    N, K = _i4._matrix(w, "w")
    dt = _i4._code(_i4._FLOATS, w.dtype, "weight")
    stride = _i4._row_stride(w, K, "w")
    shape = (-(-N // BLOCK), -(-K // BLOCK))
    if out is None:
        stream = _i4._stream(w)
        codes = torch.empty(N, K, dtype=torch.float8_e4m3fn, device=w.device)
        scales = torch.empty(shape, dtype=torch.float32, device=w.device)
    else:
        codes, scales = out
        _i4._given(codes, (N, K), torch.float8_e4m3fn, "out's codes")
        _i4._given(scales, shape, torch.float32, "out's scales")
        stream = _i4._stream(w, codes, scales)
    _i4._done("fp8_quantize", lib().fp8_quantize(w.data_ptr(), dt, stride, N, K, codes.data_ptr(), scales.data_ptr(),
                                                 stream))
    return codes, scales


def quantize_act(x, gate=None, group_size=128, out_dtype=torch.float8_e4m3fn, out=None):
    """8-bit codes and group scales of x [M, K], or of SiLU(gate) * x.

    Returns (codes int8 or float8_e4m3fn [M, K], scales float32 [M, ceil(K /
    group_size)]), group_size 32, 64 or 128.  x is fp32 or bf16, gate None or of
    x's shape and type; both may have any row stride of whole 16-byte units
    (the halves of one wider tensor).  fp8.gemm takes E4M3 in groups of 128,
    int4.gemv_w4a8 either type in its weight's groups.  out: the two tensors to
    write instead."""
    M, K = shape = _i4._matrix(x, "x")
    dt = _i4._code(_i4._FLOATS, x.dtype, "x")
    qt = _i4._code(_i4._BYTES, out_dtype if out is None else out[0].dtype, "output")
    G = _i4._groups(K, group_size)
    stride, gate_stride = _i4._row_stride(x, K, "x"), 0
    if gate is not None:
        if gate.shape != shape or gate.dtype != x.dtype:
            raise ValueError(f"gate must have x's shape {(M, K)} and its type")
        gate_stride = _i4._row_stride(gate, K, "gate")
    if out is None:
        stream = _i4._stream(x, gate)
        codes = torch.empty(M, K, dtype=out_dtype, device=x.device)
        scales = torch.empty(M, G, dtype=torch.float32, device=x.device)
    else:
        codes, scales = out
        _i4._given(codes, (M, K), codes.dtype, "out's codes")
        _i4._given(scales, (M, G), torch.float32, "out's scales")
        stream = _i4._stream(x, gate, codes, scales)
    _i4._done("fp8_quantize_act",
              lib().fp8_quantize_act(x.data_ptr(), stride, _i4._ptr(gate), gate_stride, dt, M, K, group_size, qt,
                                     codes.data_ptr(), scales.data_ptr(), stream))
    return codes, scales


def gemm(x, x_scales, codes, scales, out_dtype=torch.bfloat16, out=None):
    """y = (x_scales x) (scales codes)^T, [M, N] of bf16 or fp32.

    x float8_e4m3fn [M, K] with x_scales float32 [M, ceil(K / 128)]; codes and
    scales as quantize returns them for a [N, K] weight.  Any M.  Sums are
    fp32's, but the FP8 matrix instruction, which takes the bf16 products of many
    rows, cuts each 8 columns' products off 13 bits below their largest
    (include/fp8.h has the bound); out_dtype=torch.float32 never does."""
    M, K = _i4._matrix(x, "x")
    N, Kw = _i4._matrix(codes, "codes")
    if K != Kw:
        raise ValueError(f"x has {K} columns, the weight {Kw}")
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    G = -(-K // BLOCK)
    if (x.dtype != e4m3 or codes.dtype != e4m3 or x_scales.dtype != f32 or scales.dtype != f32
            or x_scales.shape != (M, G) or scales.shape != (-(-N // BLOCK), G)):
        got = ", ".join(f"{t.dtype} {tuple(t.shape)}" for t in (x, x_scales, codes, scales))
        raise ValueError(f"a product takes float8_e4m3fn x [M, K] and codes [N, K] with float32 scales {(M, G)} and "
                         f"{(-(-N // BLOCK), G)}; got {got}")
    if not (x.is_contiguous() and x_scales.is_contiguous() and codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("tensors must be contiguous")
    if out is None:
        dt = _i4._code(_i4._FLOATS, out_dtype, "output")
        stream = _i4._stream(x, x_scales, codes, scales)
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    else:
        dt = _i4._code(_i4._FLOATS, out.dtype, "output")
        _i4._given(out, (M, N), out.dtype)
        stream = _i4._stream(x, x_scales, codes, scales, out)
    _i4._done("fp8_gemm", lib().fp8_gemm(x.data_ptr(), x_scales.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, N,
                                         K, out.data_ptr(), dt, stream))
    return out
