"""Checks of the 8-bit layers and of the paged 8-bit cache that need no GPU:
the headers' symbols, the argument checks of the C ABI and of the bindings, and
pins of the tests' plain reference."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from dit_quantization_amd import fp8, int4, kvcache
from dit_quantization_amd import nvfp4 as nv
from tests import eight_bit_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000            # fake, aligned, non-null address: validation never dereferences
BIG = 1 << 40
E4 = torch.float8_e4m3fn


@pytest.mark.parametrize("module,header,prefix", [(fp8, "fp8.h", "fp8"), (kvcache, "kvcache.h", "kv8")])
def test_library_exports_every_declared_symbol(module, header, prefix):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(%s_[a-z0-9_]+)\s*\(" % prefix, src))
    assert names == set(module.SIGNATURES)
    for n in names:
        assert hasattr(module.lib(), n), n


# ---- the reference

def test_reference_e4m3_matches_torch():
    b = np.arange(127, dtype=np.uint8)
    assert np.array_equal(ref.E4M3, torch.from_numpy(b).view(E4).double().numpy())
    mids = (ref.E4M3[1:] + ref.E4M3[:-1]) / 2
    v = np.concatenate([ref.E4M3, mids, np.nextafter(mids.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.nextafter(mids.astype(np.float32), np.float32(500)).astype(np.float64),
                        np.random.default_rng(0).uniform(0, 448, 4000)])
    v = np.concatenate([v, -v]).astype(np.float32)
    assert np.array_equal(ref.nearest_e4m3(v.astype(np.float64)), torch.from_numpy(v).to(E4).double().numpy())
    assert ref.nearest_e4m3(np.array([464.0, 1e9])).tolist() == [448.0, 448.0]


def test_reference_scales_and_codes():
    q, s = ref.encode(np.array([0.0, 0.0]), True)
    assert q.tolist() == [0, 0] and s == 1
    q, s = ref.encode(np.array([127.0, -2.5, 1.5]), False)
    assert s == 1 and q.tolist() == [127, -2, 2]
    q, s = ref.quantize_blocks(np.pad(np.full((1, 1), 448.0), ((0, 128), (0, 16))))
    assert s.shape == (2, 1) and s[:, 0].tolist() == [1, 1] and q[0, 0] == 448
    q, s = ref.quantize_groups(np.array([[896.0] * 32 + [1.0] * 8]), 32, True)
    assert s.tolist() == [[2.0, np.float32(1 / 448)]]
    assert np.allclose(ref.silu_product(np.ones(3), np.array([0.0, 1.0, -1e9])), [0, 0.7310585786300049, 0])


def test_reference_slots():
    table = np.array([[5, 2], [-1, 7]])
    assert ref.slots(table, [1, 3, 6], [1, 0], 2, 6, 8).tolist() == [-2, 11, 4, -1, -1, -1, -2, -2]


# ---- the C ABI's checks

def test_quantize_validation():
    f = fp8.lib().fp8_quantize

    def call(x=A, dt=int4.F32, stride=64, rows=4, cols=64, codes=A, scales=A):
        return f(x, dt, stride, rows, cols, codes, scales, None)

    assert call(x=None) == call(codes=None) == call(scales=None) == nv.ERR_NULL
    assert call(dt=int4.I8) == nv.ERR_DTYPE
    assert call(rows=-1) == call(cols=-16) == call(cols=24) == call(stride=48) == nv.ERR_SHAPE
    assert call(rows=BIG, stride=BIG) == nv.ERR_SHAPE
    assert call(cols=(1 << 24) + 16, stride=BIG) == nv.ERR_UNSUPPORTED
    assert call(x=A + 8) == call(codes=A + 4) == call(scales=A + 2) == call(stride=66) == nv.ERR_ALIGN
    assert call(dt=int4.BF16, stride=68) == nv.ERR_ALIGN
    assert f(None, int4.BF16, 64, 0, 64, None, None, None) == nv.OK
    assert f(None, int4.BF16, 0, 4, 0, None, None, None) == nv.OK
    assert f(None, int4.BF16, 64, 0, 40, None, None, None) == nv.ERR_SHAPE


def test_quantize_act_validation():
    f = fp8.lib().fp8_quantize_act

    def call(x=A, xs=64, g=A, gs=64, dt=int4.BF16, rows=4, cols=64, group=128, qt=int4.E4M3, codes=A, scales=A):
        return f(x, xs, g, gs, dt, rows, cols, group, qt, codes, scales, None)

    assert call(x=None) == call(codes=None) == call(scales=None) == nv.ERR_NULL
    assert call(dt=int4.E4M3) == call(qt=int4.BF16) == nv.ERR_DTYPE
    assert call(rows=-1) == call(cols=24) == call(xs=48) == call(gs=48) == call(rows=BIG, xs=BIG) == nv.ERR_SHAPE
    assert call(rows=BIG, gs=BIG) == nv.ERR_SHAPE
    assert call(group=0) == call(group=16) == call(group=96) == call(group=256) == nv.ERR_UNSUPPORTED
    assert call(cols=(1 << 24) + 16, xs=BIG, gs=BIG) == nv.ERR_UNSUPPORTED
    assert call(x=A + 8) == call(g=A + 8) == call(codes=A + 4) == call(scales=A + 2) == nv.ERR_ALIGN
    assert call(xs=68) == call(gs=68) == nv.ERR_ALIGN
    assert call(rows=0, x=None, g=None, codes=None, scales=None) == nv.OK
    assert call(cols=0, x=None, g=None, codes=None, scales=None) == nv.OK


def test_gemm_validation():
    f = fp8.lib().fp8_gemm

    def call(x=A, xs=A, w=A, ws=A, M=4, N=64, K=64, y=A, dt=int4.BF16):
        return f(x, xs, w, ws, M, N, K, y, dt, None)

    assert call(x=None) == call(xs=None) == call(w=None) == call(ws=None) == call(y=None) == nv.ERR_NULL
    assert call(dt=int4.I8) == nv.ERR_DTYPE
    assert call(M=-1) == call(N=-1) == call(K=-16) == call(K=40) == nv.ERR_SHAPE
    assert call(K=0) == call(K=(1 << 22) + 16) == call(N=(1 << 26) + 1) == call(M=(1 << 31) + 1) == nv.ERR_UNSUPPORTED
    assert call(x=A + 8) == call(w=A + 8) == call(xs=A + 2) == call(ws=A + 2) == call(y=A + 2) == nv.ERR_ALIGN
    assert call(x=None, xs=None, w=None, ws=None, y=None, M=0) == nv.OK
    assert call(x=None, xs=None, w=None, ws=None, y=None, N=0) == nv.OK
    assert call(M=0, K=40) == nv.ERR_SHAPE


def _kv(fn="kv8_write", dt=int4.BF16, qt=int4.I8, **over):
    t = dict(codes=A, scales=A, code_stride=4 * 2 * 32, scale_stride=8, rows=A, token_stride=64, head_stride=32, dim=32)
    p = dict(page_table=A, cu=A, starts=A, seqs=2, table_width=3, tokens=5, heads=2, pages=9, page_size=4)
    for k, v in over.items():
        (t if k in t else p)[k] = v
    return getattr(kvcache.lib(), fn)(kvcache.Tensor(**t), kvcache.Tensor(**t), kvcache.Places(**p), dt, qt, None)


@pytest.mark.parametrize("fn", ["kv8_write", "kv8_read"])
def test_kv_validation(fn):
    def call(**over):
        return _kv(fn, **over)

    assert call(codes=None) == call(scales=None) == call(rows=None) == call(cu=None) == nv.ERR_NULL
    assert call(page_table=None) == nv.ERR_NULL
    assert call(dt=int4.I8) == call(qt=int4.F32) == nv.ERR_DTYPE
    for k in ("seqs", "table_width", "tokens", "heads", "pages", "dim", "token_stride", "head_stride"):
        assert call(**{k: -16}) == nv.ERR_SHAPE, k
    assert call(page_size=0) == call(dim=24) == call(dim=0) == nv.ERR_SHAPE
    assert call(code_stride=240) == call(scale_stride=7) == nv.ERR_SHAPE       # shorter than a page
    assert call(pages=(1 << 31) - 1, code_stride=1 << 60) == nv.ERR_SHAPE
    assert call(dim=1040, code_stride=BIG) == call(heads=65537, code_stride=BIG, scale_stride=BIG) == nv.ERR_UNSUPPORTED
    for k in ("seqs", "table_width", "tokens", "pages"):
        assert call(**{k: 1 << 31}) == nv.ERR_UNSUPPORTED, k
    assert call(page_size=1 << 31, code_stride=BIG, scale_stride=BIG) == nv.ERR_UNSUPPORTED
    assert call(tokens=(1 << 31) - 1, heads=65536, dim=1024, code_stride=BIG, scale_stride=BIG, head_stride=1024,
                token_stride=1 << 26) == nv.ERR_UNSUPPORTED
    assert call(codes=A + 8) == call(rows=A + 8) == call(scales=A + 2) == call(cu=A + 2) == nv.ERR_ALIGN
    assert call(starts=A + 1) == call(page_table=A + 1) == nv.ERR_ALIGN
    assert call(code_stride=264) == call(token_stride=68) == nv.ERR_ALIGN
    assert call(dt=int4.F32, token_stride=66) == nv.ERR_ALIGN
    assert call(tokens=0, codes=None, scales=None, rows=None, cu=None, page_table=None) == nv.OK
    assert call(heads=0, codes=None, scales=None, rows=None, cu=None, page_table=None) == nv.OK
    assert call(seqs=0, page_table=None) == nv.OK
    L = getattr(kvcache.lib(), fn)
    null = ctypes.POINTER(kvcache.Tensor)()
    t = kvcache.Tensor()
    assert L(null, t, kvcache.Places(), 0, 2, None) == L(t, null, kvcache.Places(), 0, 2, None) == nv.ERR_NULL


def test_read_refuses_rows_that_overlap():
    assert _kv("kv8_read", token_stride=0) == _kv("kv8_read", head_stride=0) == nv.ERR_SHAPE
    assert _kv("kv8_read", token_stride=32, head_stride=64) == nv.ERR_SHAPE    # 5 tokens span 160 elements
    assert _kv("kv8_read", token_stride=48) == _kv("kv8_read", head_stride=16) == nv.ERR_SHAPE


# ---- the bindings' checks

def test_binding_refuses_wrong_arguments():
    """Shapes, types and layouts are refused before anything asks for a GPU."""
    w, s = torch.zeros(130, 144).to(E4), torch.ones(2, 2)
    x, xs = torch.zeros(3, 144).to(E4), torch.ones(3, 2)
    f = torch.zeros(4, 64)
    bad = [
        lambda: fp8.quantize(torch.zeros(64)),
        lambda: fp8.quantize(f.half()),
        lambda: fp8.quantize(torch.zeros(64, 4).t()),
        lambda: fp8.quantize(f, out=(f.to(E4), torch.ones(1, 2))),
        lambda: fp8.quantize(f, out=(f.to(torch.int8), torch.ones(1, 1))),
        lambda: fp8.quantize_act(f[0]),
        lambda: fp8.quantize_act(f, group_size=0),
        lambda: fp8.quantize_act(f, group_size=16),
        lambda: fp8.quantize_act(f, out_dtype=torch.uint8),
        lambda: fp8.quantize_act(f.to(E4)),
        lambda: fp8.quantize_act(f, gate=f.bfloat16()),
        lambda: fp8.quantize_act(f, gate=f[:, :32]),
        lambda: fp8.quantize_act(f, gate=torch.zeros(64, 4).t()),
        lambda: fp8.quantize_act(f, out=(f.to(E4), torch.ones(4, 2))),
        lambda: fp8.gemm(x, xs, w[:, :128], s),
        lambda: fp8.gemm(x.float(), xs, w, s),
        lambda: fp8.gemm(x, xs.double(), w, s),
        lambda: fp8.gemm(x, xs[:, :1], w, s),
        lambda: fp8.gemm(x, xs, w, s[:1]),
        lambda: fp8.gemm(x, xs, w.view(torch.int8), s),
        lambda: fp8.gemm(x, xs.t().contiguous().t(), w, s),
        lambda: fp8.gemm(x[0], xs, w, s),
        lambda: fp8.gemm(x, xs, w, s, out_dtype=torch.float16),
        lambda: fp8.gemm(x, xs, w, s, out=torch.zeros(3, 131)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_kv_binding_refuses_wrong_arguments():
    cache = kvcache.new(6, 4, 2, 32, 16, torch.int8, "cpu")
    assert [tuple(t.shape) for t in cache] == [(6, 4, 2, 32), (6, 4, 2), (6, 4, 2, 16), (6, 4, 2)]
    k, v = torch.zeros(5, 2, 32), torch.zeros(5, 2, 16)
    table, cu, starts = torch.zeros(2, 3, dtype=torch.int32), torch.tensor([0, 2, 5], dtype=torch.int32), None
    bad = [
        lambda: kvcache.new(6, 4, 2, 32, dtype=torch.uint8, device="cpu"),
        lambda: kvcache.write(k.half(), v.half(), cache, table, cu),
        lambda: kvcache.write(k, v.bfloat16(), cache, table, cu),
        lambda: kvcache.write(k, k, cache, table, cu),
        lambda: kvcache.write(k[:4], v, cache, table, cu),
        lambda: kvcache.write(k[0], v[0], cache, table, cu),
        lambda: kvcache.write(torch.zeros(5, 32, 2).transpose(1, 2), v, cache, table, cu),
        lambda: kvcache.write(k, v, (cache[0], cache[1], cache[2].to(E4), cache[3]), table, cu),
        lambda: kvcache.write(k, v, (cache[0], cache[1].double(), cache[2], cache[3]), table, cu),
        lambda: kvcache.write(k, v, (cache[0], cache[1][:5], cache[2], cache[3]), table, cu),
        lambda: kvcache.write(k, v, (cache[0].view(torch.uint8), cache[1], cache[2].view(torch.uint8), cache[3]), table, cu),
        lambda: kvcache.write(k, v, (torch.zeros(6, 4, 32, 2, dtype=torch.int8).transpose(2, 3), *cache[1:]), table, cu),
        lambda: kvcache.write(k, v, cache, table.long(), cu),
        lambda: kvcache.write(k, v, cache, table[:, ::2], cu),
        lambda: kvcache.write(k, v, cache, table[0], cu),
        lambda: kvcache.write(k, v, cache, table, cu[:2]),
        lambda: kvcache.write(k, v, cache, table, cu.long()),
        lambda: kvcache.write(k, v, cache, table, cu, torch.zeros(3, dtype=torch.int32)),
        lambda: kvcache.read(cache, table, cu),
        lambda: kvcache.read(cache, table, cu, tokens=5, out_dtype=torch.float16),
        lambda: kvcache.read(cache, table, cu, out=(k, k)),
        lambda: kvcache.read(cache, table, cu, tokens=4, out=(k, v)),
        lambda: kvcache.read(cache, table, cu, out=(k, v.bfloat16())),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_bindings_refuse_cpu_tensors():
    f = torch.zeros(4, 64)
    cache = kvcache.new(6, 4, 2, 32, device="cpu")
    k = torch.zeros(5, 2, 32)
    table, cu = torch.zeros(2, 3, dtype=torch.int32), torch.tensor([0, 2, 5], dtype=torch.int32)
    for call in (lambda: fp8.quantize(f), lambda: fp8.quantize_act(f),
                 lambda: fp8.gemm(f.to(E4), torch.ones(4, 1), f.to(E4), torch.ones(1, 1)),
                 lambda: kvcache.write(k, k, cache, table, cu), lambda: kvcache.read(cache, table, cu, tokens=5)):
        with pytest.raises(ValueError, match="current GPU"):
            call()
