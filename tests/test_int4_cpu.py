"""Checks of the group-scaled 4-bit weight path that need no GPU: the header's
symbols, the argument checks of the C ABI and of the binding, and pins of the
tests' plain reference."""
import os
import re

import numpy as np
import pytest
import torch

from dit_quantization_amd import int4
from dit_quantization_amd import nvfp4 as nv
from tests import int4_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000            # fake, aligned, non-null address: validation never dereferences
BIG = 1 << 40


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "int4.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(int4_[a-z0-9_]+)\s*\(", src))
    assert names == set(int4.SIGNATURES)
    L = int4.lib()
    for n in names:
        assert hasattr(L, n), n


def test_quantize_validation():
    f = int4.lib().int4_quantize

    def call(x=A, dt=int4.F32, rows=4, cols=64, group=32, codes=A, scales=A, zeros=A):
        return f(x, dt, rows, cols, group, codes, scales, zeros, None)

    assert call(x=None) == call(codes=None) == call(scales=None) == nv.ERR_NULL
    assert call(dt=int4.I8) == nv.ERR_DTYPE
    assert call(rows=-1) == call(cols=-32) == call(cols=24) == call(rows=BIG, cols=BIG) == nv.ERR_SHAPE
    assert call(cols=48) == call(group=16) == call(group=0) == call(group=96) == nv.ERR_UNSUPPORTED
    assert call(cols=(1 << 24) + 32) == nv.ERR_UNSUPPORTED
    assert call(x=A + 8) == call(codes=A + 2) == call(scales=A + 1) == nv.ERR_ALIGN
    assert f(None, int4.BF16, 0, 64, 32, None, None, None, None) == nv.OK
    assert f(None, int4.BF16, 4, 0, 32, None, None, None, None) == nv.OK
    assert f(None, int4.BF16, 0, 48, 32, None, None, None, None) == nv.ERR_UNSUPPORTED


def test_dequant_validation():
    f = int4.lib().int4_dequant

    def call(codes=A, scales=A, zeros=A, rows=4, cols=64, group=64, out=A, dt=int4.F32):
        return f(codes, scales, zeros, rows, cols, group, out, dt, None)

    assert call(codes=None) == call(scales=None) == call(out=None) == nv.ERR_NULL
    assert call(dt=int4.E4M3) == nv.ERR_DTYPE
    assert call(rows=-1) == call(cols=40) == nv.ERR_SHAPE
    assert call(cols=48) == call(group=256) == nv.ERR_UNSUPPORTED
    assert call(codes=A + 1) == call(scales=A + 1) == call(out=A + 8) == nv.ERR_ALIGN
    assert f(None, None, None, 0, 64, 32, None, int4.F32, None) == nv.OK


def test_gemv_validation():
    L = int4.lib()

    def a16(x=A, codes=A, scales=A, zeros=A, group=128, M=1, N=64, K=64, y=A, dt=int4.BF16):
        return L.int4_gemv_w4a16(x, codes, scales, zeros, group, M, N, K, y, dt, None)

    def a8(x=A, xt=int4.I8, xs=A, xg=0, codes=A, scales=A, zeros=A, group=128, M=1, N=64, K=64, y=A, dt=int4.BF16):
        return L.int4_gemv_w4a8(x, xt, xs, xg, codes, scales, zeros, group, M, N, K, y, dt, None)

    for f in (a16, a8):
        assert f(x=None) == f(codes=None) == f(scales=None) == f(y=None) == nv.ERR_NULL
        assert f(dt=int4.I8) == nv.ERR_DTYPE
        assert f(M=-1) == f(N=-1) == f(K=40) == f(K=-32) == nv.ERR_SHAPE
        assert f(M=17) == f(K=48) == f(K=0) == f(group=48) == f(K=(1 << 24) + 32) == nv.ERR_UNSUPPORTED
        assert f(N=(1 << 28) + 1) == nv.ERR_UNSUPPORTED
        assert f(x=A + 8) == f(codes=A + 4) == f(scales=A + 1) == f(y=A + 2) == nv.ERR_ALIGN
        assert f(x=None, codes=None, scales=None, zeros=None, y=None, M=0) == nv.OK
        assert f(x=None, codes=None, scales=None, zeros=None, y=None, N=0) == nv.OK
        assert f(M=0, K=40) == nv.ERR_SHAPE
    assert a8(xs=None) == nv.ERR_NULL
    assert a8(xt=int4.BF16) == a8(xt=9) == nv.ERR_DTYPE
    assert a8(xg=64) == nv.ERR_UNSUPPORTED
    assert a8(xs=A + 2) == nv.ERR_ALIGN


def test_rmsnorm_validation():
    f = int4.lib().int4_rmsnorm_quant8

    def call(x=A, xt=int4.BF16, xs=64, r=A, rt=int4.BF16, rs=64, w=A, wt=int4.BF16, eps=1e-6, rows=4, cols=64, group=0,
             qt=int4.I8, q=A, s=A, h=A):
        return f(x, xt, xs, r, rt, rs, w, wt, eps, rows, cols, group, qt, q, s, h, None)

    assert call(x=None) == call(q=None) == call(s=None) == call(h=None) == nv.ERR_NULL
    assert call(xt=int4.I8) == call(rt=7) == call(wt=7) == call(qt=int4.BF16) == nv.ERR_DTYPE
    assert call(xt=int4.F32, rt=int4.BF16) == nv.ERR_DTYPE                # a residual narrower than x
    assert call(eps=-1e-6) == call(eps=float("nan")) == call(eps=float("inf")) == nv.ERR_FLAGS
    assert call(rows=-1) == call(cols=24) == call(cols=-16) == call(xs=48) == call(rs=48) == nv.ERR_SHAPE
    assert call(cols=65552, xs=65552, rs=65552) == call(group=16) == nv.ERR_UNSUPPORTED
    assert call(x=A + 8) == call(r=A + 8) == call(h=A + 8) == call(w=A + 8) == call(q=A + 4) == nv.ERR_ALIGN
    assert call(s=A + 2) == call(xs=68) == call(rs=68) == nv.ERR_ALIGN    # rows of 136 bytes
    assert call(rows=0, x=None, r=None, w=None, q=None, s=None, h=None) == nv.OK
    assert call(cols=0, xs=0, rs=0) == nv.ERR_SHAPE                       # a norm of nothing


def _weight(N=8, K=64, G=2):
    return (torch.zeros((N, K // 2), dtype=torch.uint8), torch.zeros((N, G), dtype=torch.bfloat16),
            torch.zeros((N, G), dtype=torch.uint8))


def test_binding_refuses_wrong_arguments():
    """Shapes, types, layouts and group sizes are refused before anything
    asks for a GPU."""
    c, s, z = _weight()
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    x8, xs = torch.zeros((2, 64), dtype=torch.int8), torch.ones((2, 1))
    bad = [
        lambda: int4.quantize(torch.zeros(64)),
        lambda: int4.quantize(torch.zeros((4, 64), dtype=torch.float16)),
        lambda: int4.quantize(torch.zeros((4, 64)), group_size=16),
        lambda: int4.quantize(torch.zeros((64, 4)).t()),
        lambda: int4.quantize(torch.zeros((8, 64)), 32, True, out=(c, s, z)),
        lambda: int4.quantize(torch.zeros((8, 64)), 32, False, out=(c, s, None)),
        lambda: int4.quantize(torch.zeros((8, 64)), 64, False, out=(c, s, z)),
        lambda: int4.dequant(c, s, z, 64),
        lambda: int4.dequant(c, s, z, 32, out_dtype=torch.float16),
        lambda: int4.dequant(c, s.float(), z, 32),
        lambda: int4.dequant(c, s, z[:, :1], 32),
        lambda: int4.dequant(c, s, z, 32, out=torch.zeros((8, 32))),
        lambda: int4.gemv_w4a16(x.float(), c, s, z, 32),
        lambda: int4.gemv_w4a16(x[:, :32], c, s, z, 32),
        lambda: int4.gemv_w4a16(x[0], c, s, z, 32),
        lambda: int4.gemv_w4a16(torch.zeros((64, 2), dtype=torch.bfloat16).t(), c, s, z, 32),
        lambda: int4.gemv_w4a16(x, c, s, z, 128),
        lambda: int4.gemv_w4a16(x, c, s, z, 32, out=torch.zeros((2, 9))),
        lambda: int4.gemv_w4a8(x, xs, c, s, z, 32),
        lambda: int4.gemv_w4a8(x8, xs.double(), c, s, z, 32),
        lambda: int4.gemv_w4a8(x8, torch.ones((2, 3)), c, s, z, 32),
        lambda: int4.gemv_w4a8(x8, torch.ones((2, 4))[:, ::2], c, s, z, 32),
        lambda: int4.rmsnorm_quant8(x[0]),
        lambda: int4.rmsnorm_quant8(x, out_dtype=torch.uint8),
        lambda: int4.rmsnorm_quant8(x, eps=-1.0),
        lambda: int4.rmsnorm_quant8(x, eps=float("nan")),
        lambda: int4.rmsnorm_quant8(x, group_size=48),
        lambda: int4.rmsnorm_quant8(x, torch.ones(32)),
        lambda: int4.rmsnorm_quant8(x, torch.ones(64, dtype=torch.float16)),
        lambda: int4.rmsnorm_quant8(x, residual=torch.zeros((1, 64))),
        lambda: int4.rmsnorm_quant8(x.float(), residual=x),
        lambda: int4.rmsnorm_quant8(torch.zeros((64, 2), dtype=torch.bfloat16).t()),
        lambda: int4.rmsnorm_quant8(x, out=(x8, xs, x)),
        lambda: int4.rmsnorm_quant8(x, residual=x, out=(x8, xs, None)),
        lambda: int4.rmsnorm_quant8(x, residual=x, out=(x8, xs, x.float())),
        lambda: int4.rmsnorm_quant8(x, group_size=32, out=(x8, xs, None)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")


def test_reference_pins():
    """The plain reference against values worked out by hand."""
    assert np.array_equal(ref.unpack(np.array([[0x40, 0x51, 0x62, 0x73]], np.uint8)), [[0, 1, 2, 3, 4, 5, 6, 7]])
    c = np.random.default_rng(0).integers(0, 16, (3, 96)).astype(np.uint8)
    assert np.array_equal(ref.unpack(ref.pack(c)), c)
    w = np.zeros((1, 32), np.float32)
    w[0, :4] = [7.0, -3.5, 0.5, 1.5]                         # s = 1: ties to even
    codes, s, z = ref.quantize(w, 32, True)
    assert s[0, 0] == 1 and z[0, 0] == 8 and list(codes[0, :5]) == [15, 4, 8, 10, 8]
    w[0, :4] = [10.0, -5.0, 2.5, -4.5]
    codes, s, z = ref.quantize(w, 32, False)
    assert s[0, 0] == 1 and z[0, 0] == 5 and list(codes[0, :5]) == [15, 0, 7, 1, 5]
    assert list(ref.to_e4m3(np.array([448.0, 500.0, 1.0625, 1.1875, 2.0 ** -10, 1.5 * 2.0 ** -9, -464.1]))) == \
        [448, 448, 1.0, 1.25, 0.0, 2 * 2.0 ** -9, -448]
    every = np.arange(256, dtype=np.uint8)
    v = ref.e4m3_bytes_to_f64(every[(every & 0x7F) != 0x7F])
    assert np.array_equal(ref.to_e4m3(v), v) and v.max() == 448
    assert np.array_equal(v, torch.from_numpy(every[(every & 0x7F) != 0x7F]).view(torch.float8_e4m3fn).double().numpy())
    q, s, h = ref.rmsnorm_quant8([[3.0, -4.0]], None, [[0.0, 0.0]], True, 0.0, 0, False)
    assert list(q[0]) == [95, -127] and abs(s[0, 0] - (4 / np.sqrt(12.5) / 127)) < 1e-9 and list(h[0]) == [3, -4]


class _Reached(Exception):
    """Raised in the place of the look at the device: every check of the binding has passed."""


def test_binding_refusals_come_from_its_own_checks(monkeypatch):
    """Each wrong call is refused for its own reason, before the device is
    looked at, and right ones get there."""
    def reached(*tensors):
        raise _Reached
    monkeypatch.setattr(int4, "_stream", reached)
    c, s, z = _weight()
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    x8, xs = torch.zeros((2, 64), dtype=torch.int8), torch.ones((2, 1))
    w, f8 = torch.zeros((8, 64)), torch.float8_e4m3fn
    half, wide = torch.zeros((8, 64), dtype=torch.float16), torch.zeros((2, 128), dtype=torch.bfloat16)
    turned = torch.zeros((64, 2), dtype=torch.bfloat16).t()
    gapped = torch.zeros((8, 4), dtype=torch.bfloat16)[:, ::2]
    good = [
        lambda: int4.quantize(w), lambda: int4.quantize(w.bfloat16(), 32, True),
        lambda: int4.quantize(w, 32, out=(c, s, z)), lambda: int4.quantize(w, 32, True, out=(c, s, None)),
        lambda: int4.dequant(c, s, z, 32), lambda: int4.dequant(c, s, None, 32, torch.bfloat16),
        lambda: int4.dequant(c, s, z, 32, out=w),
        lambda: int4.gemv_w4a16(x, c, s, z, 32), lambda: int4.gemv_w4a16(x, c, s, None, 32, torch.float32),
        lambda: int4.gemv_w4a16(x, c, s, z, 32, out=torch.zeros((2, 8))),
        lambda: int4.gemv_w4a8(x8, xs, c, s, z, 32), lambda: int4.gemv_w4a8(x8.to(f8), torch.ones((2, 2)), c, s, z, 32),
        lambda: int4.rmsnorm_quant8(x), lambda: int4.rmsnorm_quant8(x, torch.ones(64), x, 0.0, 32, f8),
        lambda: int4.rmsnorm_quant8(wide[:, :64], residual=wide[:, 64:].float()[:, :64]),
        lambda: int4.rmsnorm_quant8(x, residual=x, out=(x8, xs, x)),
    ]
    for i, f in enumerate(good):
        with pytest.raises(_Reached):
            f()
            pytest.fail(f"right call {i} did not reach the device")
    packed, flat, side = "a packed weight is", "must be a 2-D tensor", "must be contiguous"
    bad = [
        (flat, lambda: int4.quantize(torch.zeros(64))),
        ("unsupported weight dtype", lambda: int4.quantize(half)),
        ("group_size=16", lambda: int4.quantize(w, group_size=16)),
        (side, lambda: int4.quantize(torch.zeros((64, 8)).t())),
        ("zeros must be None exactly", lambda: int4.quantize(w, 32, True, out=(c, s, z))),
        ("zeros must be None exactly", lambda: int4.quantize(w, 32, False, out=(c, s, None))),
        ("out's codes", lambda: int4.quantize(w, 32, out=(c[:, :16], s, z))),
        ("out's codes", lambda: int4.quantize(w, 32, out=(c.to(torch.int8), s, z))),
        ("out's scales", lambda: int4.quantize(w, 64, out=(c, s, z))),
        ("out's scales", lambda: int4.quantize(w, 32, out=(c, gapped, z))),
        ("out's zeros", lambda: int4.quantize(w, 32, out=(c, s, z[:4]))),
        (flat, lambda: int4.dequant(c[0], s, z, 32)),
        (packed, lambda: int4.dequant(c, s, z, 64)),
        (packed, lambda: int4.dequant(c.to(torch.int8), s, z, 32)),
        (packed, lambda: int4.dequant(c, s.float(), z, 32)),
        (packed, lambda: int4.dequant(c, s[:4], z, 32)),
        (packed, lambda: int4.dequant(c, s, z[:, :1], 32)),
        (packed, lambda: int4.dequant(c, s, z.to(torch.int8), 32)),
        (side, lambda: int4.dequant(torch.zeros((32, 8), dtype=torch.uint8).t(), s, z, 32)),
        (side, lambda: int4.dequant(c, gapped, z, 32)),
        (side, lambda: int4.dequant(c, s, torch.zeros((2, 8), dtype=torch.uint8).t(), 32)),
        ("group_size=48", lambda: int4.dequant(c, s, z, 48)),
        ("unsupported output dtype", lambda: int4.dequant(c, s, z, 32, out_dtype=torch.float16)),
        ("unsupported output dtype", lambda: int4.dequant(c, s, z, 32, out=half)),
        ("out must be a contiguous", lambda: int4.dequant(c, s, z, 32, out=torch.zeros((8, 32)))),
        ("out must be a contiguous", lambda: int4.dequant(c, s, z, 32, out=torch.zeros((64, 8)).t())),
        ("2-D bfloat16", lambda: int4.gemv_w4a16(x.float(), c, s, z, 32)),
        ("x has 32 columns", lambda: int4.gemv_w4a16(x[:, :32], c, s, z, 32)),
        (flat, lambda: int4.gemv_w4a16(x[0], c, s, z, 32)),
        (side, lambda: int4.gemv_w4a16(turned, c, s, z, 32)),
        (packed, lambda: int4.gemv_w4a16(x, c, s, z, 128)),
        ("unsupported output dtype", lambda: int4.gemv_w4a16(x, c, s, z, 32, torch.float16)),
        ("out must be a contiguous", lambda: int4.gemv_w4a16(x, c, s, z, 32, out=torch.zeros((2, 9)))),
        ("out must be a contiguous", lambda: int4.gemv_w4a16(x, c, s, z, 32, out=torch.zeros((8, 2)).t())),
        ("unsupported activation dtype", lambda: int4.gemv_w4a8(x, xs, c, s, z, 32)),
        ("x_scales must be", lambda: int4.gemv_w4a8(x8, xs.double(), c, s, z, 32)),
        ("x_scales must be", lambda: int4.gemv_w4a8(x8, torch.ones((2, 3)), c, s, z, 32)),
        ("x_scales must be", lambda: int4.gemv_w4a8(x8, torch.ones(2), c, s, z, 32)),
        (side, lambda: int4.gemv_w4a8(x8, torch.ones((2, 4))[:, ::2], c, s, z, 32)),
        (flat, lambda: int4.rmsnorm_quant8(x[0])),
        ("unsupported x dtype", lambda: int4.rmsnorm_quant8(half)),
        ("unsupported output dtype", lambda: int4.rmsnorm_quant8(x, out_dtype=torch.uint8)),
        ("eps=-1.0", lambda: int4.rmsnorm_quant8(x, eps=-1.0)),
        ("eps=nan", lambda: int4.rmsnorm_quant8(x, eps=float("nan"))),
        ("eps=inf", lambda: int4.rmsnorm_quant8(x, eps=float("inf"))),
        ("group_size=48", lambda: int4.rmsnorm_quant8(x, group_size=48)),
        ("weight must be", lambda: int4.rmsnorm_quant8(x, torch.ones(32))),
        ("weight must be", lambda: int4.rmsnorm_quant8(x, torch.ones(128)[::2])),
        ("unsupported weight dtype", lambda: int4.rmsnorm_quant8(x, torch.ones(64, dtype=torch.float16))),
        ("residual must have", lambda: int4.rmsnorm_quant8(x, residual=torch.zeros((1, 64)))),
        ("residual must have", lambda: int4.rmsnorm_quant8(x.float(), residual=x)),
        ("x's rows must be contiguous", lambda: int4.rmsnorm_quant8(turned)),
        ("residual's rows must be contiguous", lambda: int4.rmsnorm_quant8(x, residual=turned)),
        ("sum must be None exactly", lambda: int4.rmsnorm_quant8(x, out=(x8, xs, x))),
        ("sum must be None exactly", lambda: int4.rmsnorm_quant8(x, residual=x, out=(x8, xs, None))),
        ("out's sum", lambda: int4.rmsnorm_quant8(x, residual=x, out=(x8, xs, x.float()))),
        ("out's sum", lambda: int4.rmsnorm_quant8(x, residual=x, out=(x8, xs, turned))),
        ("out's scales", lambda: int4.rmsnorm_quant8(x, group_size=32, out=(x8, xs, None))),
        ("out's codes", lambda: int4.rmsnorm_quant8(x, out=(x8[:, :32], xs, None))),
    ]
    for i, (why, f) in enumerate(bad):
        with pytest.raises(ValueError, match=why):
            f()
            pytest.fail(f"call {i} was accepted")
