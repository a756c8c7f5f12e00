"""GPU parity of the group-scaled 4-bit weight path (include/int4.h) with the
plain fp64 forms of tests/int4_reference.py: codes, zero points, scales and
8-bit activations bit for bit, products within an any-order bound of their
fp32 sums."""
import ctypes

import numpy as np
import pytest
import torch

from dit_quantization_amd import int4
from dit_quantization_amd import nvfp4 as nv
from tests import int4_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FL = torch.bfloat16, torch.float32
HALF_BF16 = 2.0 ** -8                    # half a step, relative


def rng(seed):
    return np.random.default_rng(seed)


def tensor(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)


def f32(t):
    return t.float().cpu().numpy()


def e4m3_values(t):
    return ref.e4m3_bytes_to_f64(t.view(torch.uint8).cpu().numpy())


# ---- the weight quantizer and its inverse

def weights(rows, cols, seed, kind):
    g = rng(seed)
    w = (g.standard_t(5, (rows, cols)) * 0.02).astype(np.float32)
    if kind == "edges":
        w[0] = 0                                              # a row of zeros
        if rows > 1:
            w[1] = g.integers(-15, 16, cols) * np.float32(0.5)   # ties everywhere
        if rows > 2:
            w[2] = np.abs(w[2])                               # one sign: the zero point on a border
        if rows > 3:
            w[3] = -np.abs(w[3])
        if rows > 4:
            w[4] *= np.float32(1e-38)                         # scales below the normal range, some 0
        if rows > 5:
            w[5] *= np.float32(1e38)
            w[5, :2] = [3.0e38, -3.0e38]                      # a range beyond fp32
        if rows > 6:
            w[6] = np.where(g.random(cols) < 0.5, np.float32(-0.0), w[6])
        if rows > 7:
            w[7] = np.float32(1e-45) * g.integers(-40, 41, cols)   # whole denormals
    return w


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,cols,bf16,kind", [(1, 32, False, "edges"), (8, 32, False, "edges"), (8, 96, True, "edges"),
                                                 (9, 416, False, "edges"), (33, 1024, True, "edges"),
                                                 (257, 160, False, "plain"), (5, 14336, True, "plain"),
                                                 (130, 4128, False, "edges")])
def test_quantize_and_dequant(rows, cols, bf16, kind, group):
    print(f"[case] quantize {rows}x{cols} bf16={bf16} {kind} group={group}", flush=True)
    w = tensor(weights(rows, cols, rows + cols, kind), torch.bfloat16 if bf16 else torch.float32)
    wf = f32(w)
    for symmetric in (True, False):
        codes, scales, zeros = int4.quantize(w, group, symmetric)
        rc, rs, rz = ref.quantize(wf, group, symmetric)
        assert np.array_equal(f32(scales), rs)
        assert zeros is None if symmetric else np.array_equal(zeros.cpu().numpy(), rz)
        assert np.array_equal(ref.unpack(codes.cpu().numpy()), rc)
        d = ref.dequant(rc, rs, rz, group)
        with np.errstate(over="ignore"):
            assert np.array_equal(f32(int4.dequant(codes, scales, zeros, group)), d.astype(np.float32))
            assert np.array_equal(f32(int4.dequant(codes, scales, zeros, group, torch.bfloat16)),
                                  ref.bf16(d.astype(np.float32)))


def test_quantize_writes_only_its_outputs():
    """Buffers given to the call, with guards behind them."""
    w = tensor(weights(7, 96, 3, "plain"))
    whole = [torch.full((7 * 48 + 64,), 77, dtype=torch.uint8, device=DEV),
             torch.full((7 * 2 + 64,), 3.0, dtype=torch.bfloat16, device=DEV),
             torch.full((7 * 2 + 64,), 99, dtype=torch.uint8, device=DEV)]
    out = (whole[0][:7 * 48].view(7, 48), whole[1][:14].view(7, 2), whole[2][:14].view(7, 2))
    got = int4.quantize(w, 64, out=out)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out))
    want = ref.quantize(f32(w), 64, False)
    assert np.array_equal(ref.unpack(got[0].cpu().numpy()), want[0]) and np.array_equal(got[2].cpu().numpy(), want[2])
    for t, n, v in zip(whole, (7 * 48, 14, 14), (77, 3, 99)):
        assert bool((t[n:] == v).all())
    y = torch.full((7 * 96 + 64,), 5.0, device=DEV)
    int4.dequant(*got, group_size=64, out=y[:7 * 96].view(7, 96))
    assert bool((y[7 * 96:] == 5).all())
    assert np.array_equal(f32(y[:7 * 96]).reshape(7, 96), ref.dequant(*want, 64).astype(np.float32))


# ---- the decode products

def packed_weight(N, K, group, symmetric, seed):
    g = rng(seed)
    G = -(-K // group)
    codes = g.integers(0, 16, (N, K)).astype(np.uint8)
    scales = ref.bf16((0.02 * np.exp(g.standard_normal((N, G)))).astype(np.float32))
    zeros = np.full((N, G), 8, np.uint8) if symmetric else g.integers(0, 16, (N, G)).astype(np.uint8)
    dev = (torch.from_numpy(ref.pack(codes)).to(DEV), tensor(scales, torch.bfloat16),
           None if symmetric else torch.from_numpy(zeros).to(DEV))
    return (codes, scales, zeros), dev


def activations(kind, M, K, group, grouped, seed):
    """(device arguments, fp64 values) of x: 'bf16', 'int8' or 'e4m3'."""
    g = rng(seed)
    if kind == "bf16":
        x = tensor(g.standard_normal((M, K)), torch.bfloat16)
        return (x,), f32(x).astype(np.float64)
    G = -(-K // group) if grouped else 1
    sx = np.exp(g.standard_normal((M, G))).astype(np.float32)
    if kind == "int8":
        q = g.integers(-128, 128, (M, K)).astype(np.int8)
        x, v = torch.from_numpy(q).to(DEV), q.astype(np.float64)
    else:
        x = tensor(np.clip(g.standard_normal((M, K)) * 60, -448, 448)).to(torch.float8_e4m3fn)
        v = e4m3_values(x)
    return (x, torch.from_numpy(sx).to(DEV)), v * (ref.per_element(sx, K, group) if grouped else sx.astype(np.float64))


def call(kind, args, w, group, dtype):
    f = int4.gemv_w4a16 if kind == "bf16" else int4.gemv_w4a8
    return f(*args, *w, group_size=group, out_dtype=dtype)


def check_product(kind, M, N, K, group, symmetric, grouped, dtype, seed):
    print(f"[case] {kind} M={M} N={N} K={K} group={group} sym={symmetric} grouped={grouped} {dtype}", flush=True)
    hw, w = packed_weight(N, K, group, symmetric, seed)
    args, x = activations(kind, M, K, group, grouped, seed + 1)
    y = call(kind, args, w, group, dtype)
    assert y.shape == (M, N) and y.dtype == dtype
    ystar, a = ref.product(x, *hw, group)
    tau = ref.product_bound(a, K)
    if dtype == torch.bfloat16:
        tau = tau * (1 + HALF_BF16) + HALF_BF16 * np.abs(ystar)
    err = np.abs(f32(y) - ystar)
    assert np.all(err <= tau), f"{(err > tau).sum()} of {err.size} outputs off; worst {np.max(err / tau)} of the bound"
    if dtype == torch.float32 and ystar.size >= 64:
        # independent roundings: sqrt(160 + K / 32) of them at 2^-24 on sums of
        # code and zero parts, up to 8 times the size of their difference
        # (codes and zeros uniform: rms 8.8 each, rms difference 6.5)
        assert np.linalg.norm(err) <= 8 * np.sqrt(160 + K / 32) * 2.0 ** -24 * np.linalg.norm(ystar)
    return y


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M", [1, 4])
def test_products_of_small_values(kind, M):
    """Values and scales near the lower end of fp32's normal range lose nothing:
    powers of two times a call's inputs give the same result times them."""
    hw, w = packed_weight(48, 640, 64, False, 31)
    args, _ = activations(kind, M, 640, 64, False, 32)
    y = call(kind, args, w, 64, FL)
    tiny = 2.0 ** -96
    if kind == "bf16":
        small = call(kind, (args[0] * tiny,), w, 64, FL)
    else:
        small = call(kind, (args[0], args[1] * tiny), w, 64, FL)
    assert torch.equal(small, y * tiny)
    small = call(kind, args, (w[0], w[1] * tiny, w[2]), 64, FL)
    assert torch.equal(small, y * tiny)


# M, N, K: one row and one block; rows that end inside a group; odd N; each
# count of rows; lengths that no power of two divides; every kernel's range
SHAPES = [(1, 1, 32), (1, 7, 96), (1, 64, 256), (1, 129, 4128), (1, 65, 14336), (1, 5, 33824), (2, 33, 160), (3, 16, 32),
          (4, 100, 1024), (5, 17, 544), (7, 8193, 128), (8, 31, 4096), (11, 40, 14336), (16, 1, 64), (16, 200, 2080),
          (16, 8200, 256), (1, 9000, 128), (13, 1025, 992), (3, 5000, 192), (16, 4112, 1056), (6, 8190, 512),
          (1, 3000, 8224), (1, 4099, 160), (2, 48, 8704)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
def test_products(kind, shape):
    M, N, K = shape
    for i, group in enumerate((32, 64, 128)):
        for symmetric in (False, True):
            grouped = kind != "bf16" and symmetric == (i % 2 == 0)
            check_product(kind, M, N, K, group, symmetric, grouped, torch.float32 if symmetric else torch.bfloat16,
                          100 * M + N + K + group)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M", range(1, 17))
def test_products_at_every_row_count(kind, M):
    check_product(kind, M, 96, 640, 128, False, kind != "bf16", torch.float32, M)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(1, 14336, 4096), (4, 4096, 14336), (16, 14336, 4096)])
def test_products_at_layer_sizes(kind, M, N, K):
    check_product(kind, M, N, K, 128, False, False, torch.float32, M + K)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M", [1, 16])
def test_products_at_the_largest_k(kind, M):
    """K = 2^24, the limit of 32-bit row offsets: a weight that is zero but
    for codes spread over the whole row, so the sums are short."""
    K, N, group = 1 << 24, 3, 128
    print(f"[case] {kind} M={M} N={N} K={K}", flush=True)
    g = rng(5)
    at = np.unique(np.concatenate([[0, 1, K // 2, K - 1], g.integers(0, K, 60)]))
    codes = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device=DEV)
    byte, high = (at // 8) * 4 + at % 4, at % 8 >= 4
    host = np.full((N, K // 2), 0x88, np.uint8)
    for n in range(N):
        for b, h in zip(byte, high):
            v = int(g.integers(0, 16))
            host[n, b] = (host[n, b] & 0x0F) | (v << 4) if h else (host[n, b] & 0xF0) | v
    codes = torch.from_numpy(host).to(DEV)
    scales = torch.full((N, K // group), 0.5, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((M, K), device=DEV)
    idx = torch.from_numpy(at).to(DEV)
    x[:, idx] = torch.from_numpy(g.integers(-3, 4, (M, len(at))).astype(np.float32)).to(DEV)
    if kind == "bf16":
        y = int4.gemv_w4a16(x.bfloat16(), codes, scales, out_dtype=torch.float32)
    else:
        y = int4.gemv_w4a8(x.to(torch.int8 if kind == "int8" else torch.float8_e4m3fn),
                           torch.ones((M, 1), device=DEV), codes, scales, out_dtype=torch.float32)
    q = np.stack([np.where(high, host[n, byte] >> 4, host[n, byte] & 15) for n in range(N)]).astype(np.float64) - 8
    want = 0.5 * (f32(x[:, idx]).astype(np.float64) @ q.T)       # whole halves: exact in fp32
    assert np.array_equal(f32(y).astype(np.float64), want)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M", [1, 3, 8, 16])
def test_products_of_one_sign(kind, M):
    """Activations of one sign, whose code and zero parts are far larger than
    their difference, stay within the bound of the sums."""
    for N, K, group in ((48, 8704, 32), (4200, 1056, 64), (8200, 544, 128)):
        print(f"[case] one sign {kind} M={M} N={N} K={K} group={group}", flush=True)
        hw, w = packed_weight(N, K, group, False, 51)
        g = rng(52)
        x = np.abs(g.standard_normal((M, K))) + 1
        if kind == "bf16":
            args = (tensor(x, BF),)
            v = f32(args[0]).astype(np.float64)
        else:
            G, grouped = -(-K // group), group != 64
            q = tensor(x * 25).to(torch.int8) if kind == "int8" else tensor(x * 60).to(torch.float8_e4m3fn)
            sx = np.exp(g.standard_normal((M, G if grouped else 1))).astype(np.float32)
            args = (q, torch.from_numpy(sx).to(DEV))
            v = q.cpu().numpy().astype(np.float64) if kind == "int8" else e4m3_values(q)
            v = v * (ref.per_element(sx, K, group) if grouped else sx)
        ystar, a = ref.product(v, *hw, group)
        err = np.abs(f32(call(kind, args, w, group, FL)) - ystar)
        tau = ref.product_bound(a, K)
        assert np.all(err <= tau), f"worst {np.max(err / tau)} of the bound"


def test_products_write_only_their_outputs_and_repeat():
    """Odd sizes between guards, and the same bits on every call."""
    for kind in ("bf16", "int8", "e4m3"):
        for M, N, K in ((1, 37, 96), (3, 37, 416), (16, 131, 96)):
            print(f"[case] guards {kind} {M} {N} {K}", flush=True)
            _, w = packed_weight(N, K, 64, False, 7)
            args, _ = activations(kind, M, K, 64, True, 8)
            f = int4.gemv_w4a16 if kind == "bf16" else int4.gemv_w4a8
            for dt in (torch.float32, torch.bfloat16):
                buf = torch.full((M * N + 128,), 5.0, dtype=dt, device=DEV)
                f(*args, *w, group_size=64, out=buf[64:64 + M * N].view(M, N))
                assert bool((buf[:64] == 5).all()) and bool((buf[64 + M * N:] == 5).all())
                assert torch.equal(buf[64:64 + M * N].view(M, N), f(*args, *w, group_size=64, out_dtype=dt))


@pytest.mark.parametrize("M,N", [(1, 40), (1, 4200), (4, 40), (9, 4200), (16, 8300)])
def test_products_with_scales_anywhere(M, N):
    """Scales and zero points at any address their types allow give the same."""
    for kind in ("bf16", "int8"):
        _, (c, s, z) = packed_weight(N, 1024, 128, False, 41)
        args, _ = activations(kind, M, 1024, 128, True, 42)
        y = call(kind, args, (c, s, z), 128, FL)
        s2, z2 = torch.empty(s.numel() + 9, dtype=BF, device=DEV), torch.empty(z.numel() + 9, dtype=torch.uint8, device=DEV)
        for i in (1, 2, 3):
            a, b = s2[i:i + s.numel()].view_as(s), z2[i:i + z.numel()].view_as(z)
            a.copy_(s)
            b.copy_(z)
            assert torch.equal(call(kind, args, (c, a, b), 128, FL), y)


def test_rows_do_not_depend_on_each_other():
    """A row of zeros and a loud row beside others leave them as they are."""
    _, w = packed_weight(70, 512, 128, False, 9)
    (x, xs), _ = activations("int8", 6, 512, 128, True, 10)
    y = int4.gemv_w4a8(x, xs, *w, out_dtype=torch.float32)
    x2, xs2 = x.clone(), xs.clone()
    x2[0] = 0
    xs2[3] = 1e30
    y2 = int4.gemv_w4a8(x2, xs2, *w, out_dtype=torch.float32)
    assert bool((y2[0] == 0).all())
    for m in (1, 2, 4, 5):
        assert torch.equal(y[m], y2[m])


# ---- the norm

def norm_inputs(rows, cols, seed, x_bf16, res, w):
    g = rng(seed)
    x = g.standard_normal((rows, cols)) * np.where(g.random(cols) < 0.02, 20, 1)
    x = tensor(x, torch.bfloat16 if x_bf16 else torch.float32)
    r = None if res is None else tensor(2 * g.standard_normal((rows, cols)), res)
    wt = None if w is None else tensor(1 + 0.2 * g.standard_normal(cols), w)
    return x, r, wt


def check_norm(x, r, wt, eps, group, dtype, out=None):
    # inputs are read before the call: it may write onto them
    xf, rf, wf = f32(x), None if r is None else f32(r), None if wt is None else f32(wt)
    q, s, h = int4.rmsnorm_quant8(x, wt, residual=r, eps=eps, group_size=group, out_dtype=dtype, out=out)
    e4m3 = dtype == torch.float8_e4m3fn
    rq, rs, rh = ref.rmsnorm_quant8(xf, wf, rf, r is not None and r.dtype == torch.bfloat16, eps, group, e4m3)
    assert q.dtype == dtype and s.dtype == torch.float32
    assert np.array_equal(f32(s), rs), f"scales: {np.abs(f32(s) / rs - 1).max()}"
    v = e4m3_values(q) if e4m3 else q.cpu().numpy().astype(np.float64)
    assert np.array_equal(v, rq), f"{(v != rq).sum()} of {v.size} codes differ"
    assert h is None if r is None else np.array_equal(f32(h), rh)
    return q, s, h


COLS = [16, 48, 64, 128, 144, 272, 1040, 2048, 2064, 4096, 8208, 14336, 16400, 65536]
@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
@pytest.mark.parametrize("cols", COLS)
def test_norm(cols, dtype):
    """Every type of input and every granularity at rows that leave blocks part empty."""
    for i, (x_bf16, res, w) in enumerate([(True, BF, BF), (True, FL, FL), (False, FL, BF), (False, None, None),
                                          (True, None, FL)]):
        for group in (0, 32, 64, 128):
            rows = (1, 3, 5, 2, 7)[i] if cols > 4096 else (1, 35, 6, 70, 129)[i]
            print(f"[case] norm {rows}x{cols} x_bf16={x_bf16} res={res} w={w} group={group} {dtype}", flush=True)
            x, r, wt = norm_inputs(rows, cols, cols + group + i, x_bf16, res, w)
            check_norm(x, r, wt, 1e-6, group, dtype)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
@pytest.mark.parametrize("rows,cols,group", [(2000, 4096, 128), (20011, 128, 0), (600, 14336, 0), (5000, 64, 32)])
def test_norm_many_rows(rows, cols, group, dtype):
    print(f"[case] norm {rows}x{cols} group={group} {dtype}", flush=True)
    x, r, wt = norm_inputs(rows, cols, rows, True, BF if group else None, BF)
    check_norm(x, r, wt, 1e-5, group, dtype)


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_edges(eps, dtype):
    """Rows and groups of zeros, sums that cancel, values near both ends of
    fp32, ties and scales below the normal range."""
    g = rng(11)
    x = g.standard_normal((12, 256)).astype(np.float32)
    x[0] = 0
    x[1, :128] = 0
    x[2] = np.float32(1e-30) * x[2]
    x[3] = np.float32(3e37) * x[3]
    x[4] = np.float32(1e-44)
    x[5] = 1.0
    x[6] = g.integers(-127, 128, 256)
    x[7, 1:] = 0
    x[8] = np.where(g.random(256) < 0.5, np.float32(-0.0), x[8])
    r = np.zeros_like(x)
    r[9] = -x[9]                                     # the sum is zero
    w = np.ones(256, np.float32)
    w[64:96] = 0
    w[96:128] = 1e-44
    w[200] = -3.0
    for group in (0, 32, 64, 128):
        check_norm(tensor(x), tensor(r), tensor(w), eps, group, dtype)
        check_norm(tensor(x), None, None, eps, group, dtype)
        check_norm(tensor(x[[0, 1, 5, 6, 7, 8]], BF), tensor(r[:6], BF), tensor(w, BF), eps, group, dtype)


def test_norm_strides_in_place_and_guards():
    """Slices of wider tensors, the sum written onto the residual or x, and
    nothing written past the outputs."""
    wide, res = tensor(rng(1).standard_normal((9, 3 * 128)), BF), tensor(rng(2).standard_normal((9, 2, 128)), BF)
    wt = tensor(rng(3).standard_normal(128), BF)
    check_norm(wide[:, 128:256], res[:, 1], wt, 1e-6, 0, torch.int8)
    check_norm(wide[:, 256:], res[:, 0], wt, 1e-6, 64, torch.float8_e4m3fn)
    check_norm(wide[4:5, 8:136], res[3:4, 1], wt, 1e-6, 32, torch.int8)
    for onto in ("residual", "x"):
        for rows, cols in ((5, 128), (3, 4096)):
            x, r, wt = norm_inputs(rows, cols, 4, True, BF, BF)
            q = torch.full((rows * cols + 64,), 9, dtype=torch.int8, device=DEV)
            s = torch.full((rows + 16,), 7.0, device=DEV)
            out = (q[:rows * cols].view(rows, cols), s[:rows].view(rows, 1), r if onto == "residual" else x)
            got = check_norm(x, r, wt, 1e-6, 0, torch.int8, out=out)
            assert got[2].data_ptr() == (r if onto == "residual" else x).data_ptr()
            assert bool((q[rows * cols:] == 9).all()) and bool((s[rows:] == 7).all())
    with pytest.raises(ValueError):                  # rows of 20 bytes
        int4.rmsnorm_quant8(torch.zeros((4, 40), dtype=BF, device=DEV)[:, :16].as_strided((3, 16), (18, 1)))
    with pytest.raises(ValueError):                  # rows that overlap
        int4.rmsnorm_quant8(torch.zeros((1, 16), dtype=BF, device=DEV).expand(4, 16))


@pytest.mark.parametrize("cols", [256, 4096, 16400, 40016])
def test_norm_sums_in_bf16(cols):
    """Sums that end half way between bf16 values, below its normal range and
    next to its largest value, written onto the residual."""
    g = rng(cols)
    x = g.standard_normal((4, cols)).astype(np.float32)
    r = g.standard_normal((4, cols)).astype(np.float32)
    x[0] = g.integers(128, 256, cols)                # + 1/2: half way
    r[0] = g.choice([-0.5, 0.5], cols)
    x[1], r[1] = x[1] * 2.0 ** -130, r[1] * 2.0 ** -131
    x[2], r[2] = 2.0 ** 127, (2.0 ** 126 - 2.0 ** 119) * g.choice([1, -1], cols)
    w = tensor(np.ones(cols), BF)
    for group, dtype in ((0, torch.int8), (128, torch.float8_e4m3fn)):
        rt = tensor(r, BF)
        out = (torch.empty((4, cols), dtype=dtype, device=DEV),
               torch.empty((4, -(-cols // group) if group else 1), dtype=torch.float32, device=DEV), rt)
        got = check_norm(tensor(x, BF), rt, w, 0.0, group, dtype, out=out)
        assert got[2] is rt


def test_norm_of_more_rows_than_one_launch_takes():
    """2^24 + 5 rows of 16 columns: the rows of either launch as if alone."""
    rows = (1 << 24) + 5
    print(f"[case] norm {rows}x16", flush=True)
    x = torch.randn((rows, 16), device=DEV, dtype=BF, generator=torch.Generator(DEV).manual_seed(1))
    r, wt = x.flip(0).contiguous(), torch.linspace(0.5, 1.5, 16, device=DEV)
    whole = int4.rmsnorm_quant8(x, wt, residual=r)
    for part in (slice(0, 1000), slice((1 << 24) - 500, rows)):
        alone = int4.rmsnorm_quant8(x[part], wt, residual=r[part])
        assert all(torch.equal(a[part], b) for a, b in zip(whole, alone))


# ---- together, and as a caller may use them


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 elements, and codes of more than 2^31 bytes:
    the last rows as if alone."""
    rows, cols = (1 << 19) + 3, 8192 + 32
    print(f"[case] {rows}x{cols}", flush=True)
    x = torch.randn((rows, cols), device=DEV, dtype=BF, generator=torch.Generator(DEV).manual_seed(2))
    last = slice(rows - 70, rows)
    w = int4.quantize(x, 128)
    part = int4.quantize(x[last], 128)
    assert all(torch.equal(a[last], b) for a, b in zip(w, part))
    assert torch.equal(int4.dequant(*w, out_dtype=BF)[last], int4.dequant(*part, out_dtype=BF))
    q, s, _ = int4.rmsnorm_quant8(x, group_size=128)
    q1, s1, _ = int4.rmsnorm_quant8(x[last], group_size=128)
    assert torch.equal(q[last], q1) and torch.equal(s[last], s1)
    del x
    for M in (1, 3):
        v = q[:M].contiguous(), s[:M].contiguous()
        y, y1 = int4.gemv_w4a8(*v, *w, out_dtype=FL), int4.gemv_w4a8(*v, *part, out_dtype=FL)
        # other shapes of the call may add in another order
        a = torch.from_numpy(ref.product(q[:M].cpu().numpy() * ref.per_element(f32(s[:M]), cols, 128),
                                         ref.unpack(part[0].cpu().numpy()), f32(part[1]), part[2].cpu().numpy(), 128)[1])
        assert np.all(np.abs(f32(y[:, last]) - f32(y1)) <= 2 * ref.product_bound(a.numpy(), cols))

def test_decode_mlp():
    """Norm, gate and up products on its codes, activation, down product in 16
    bits: one MLP of a decoder on a batch of four tokens, each step against
    the plain form of the same inputs."""
    M, H, F, group = 4, 512, 1376, 128
    g = rng(21)
    mats = [tensor(g.standard_t(5, s) * 0.05, BF) for s in ((F, H), (F, H), (H, F))]
    packed = [int4.quantize(m, group, symmetric=i == 2) for i, m in enumerate(mats)]
    plain = [ref.quantize(f32(m), group, i == 2) for i, m in enumerate(mats)]
    x, r, wt = norm_inputs(M, H, 22, True, BF, BF)
    for dtype, xg in ((torch.int8, 0), (torch.float8_e4m3fn, group)):
        q, s, h = check_norm(x, r, wt, 1e-6, xg, dtype)
        v = e4m3_values(q) if xg else q.cpu().numpy().astype(np.float64)
        v = v * (ref.per_element(f32(s), H, group) if xg else f32(s).astype(np.float64))
        parts = []
        for p, hp in zip(packed[:2], plain[:2]):
            y = int4.gemv_w4a8(q, s, *p, group_size=group, out_dtype=torch.float32)
            ystar, a = ref.product(v, *hp, group)
            assert np.all(np.abs(f32(y) - ystar) <= ref.product_bound(a, H))
            parts.append(y)
        act = (torch.nn.functional.silu(parts[0]) * parts[1]).to(BF)
        y = int4.gemv_w4a16(act, *packed[2], group_size=group, out_dtype=torch.float32)
        ystar, a = ref.product(f32(act), *plain[2], group)
        assert np.all(np.abs(f32(y) - ystar) <= ref.product_bound(a, F))
        # the whole layer against the unquantized one: 4-bit weights, 8-bit inputs
        y0 = f32(act).astype(np.float64) @ f32(mats[2]).astype(np.float64).T
        assert np.linalg.norm(f32(y) - y0) < 0.2 * np.linalg.norm(y0)


def test_streams_and_concurrent_calls():
    """Calls follow torch's current stream; calls on two streams at once give
    what each gives alone."""
    cases = []
    for seed, kind, M in ((1, "bf16", 1), (2, "int8", 5), (3, "e4m3", 16), (4, "int8", 1)):
        _, w = packed_weight(1024, 2048, 128, False, seed)
        args, _ = activations(kind, M, 2048, 128, True, seed)
        cases.append((kind, args, w))
    x, r, wt = norm_inputs(300, 2048, 5, True, BF, BF)
    alone = [call(k, a, w, 128, FL) for k, a, w in cases] + list(int4.rmsnorm_quant8(x, wt, residual=r))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got.append([call(k, a, w, 128, FL) for k, a, w in cases] + list(int4.rmsnorm_quant8(x, wt, residual=r)))
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, alone))


def test_empty_calls():
    """No rows, or no outputs: empty results, no launch."""
    _, w = packed_weight(8, 64, 32, False, 1)
    none = torch.zeros((0, 64), dtype=BF, device=DEV)
    assert int4.gemv_w4a16(none, *w, group_size=32).shape == (0, 8)
    assert int4.gemv_w4a8(none.to(torch.int8), torch.zeros((0, 1), device=DEV), *w, group_size=32).shape == (0, 8)
    c, s, z = int4.quantize(none, 32)
    assert c.shape == (0, 32) and s.shape == (0, 2) and z.shape == (0, 2)
    assert int4.dequant(c, s, z, 32).shape == (0, 64)
    assert int4.gemv_w4a16(torch.ones((3, 64), dtype=BF, device=DEV), c, s, z, 32).shape == (3, 0)
    q, s, h = int4.rmsnorm_quant8(none, residual=none)
    assert q.shape == (0, 64) and s.shape == (0, 1) and h.shape == (0, 64)


def test_refusals():
    """Other devices, too many rows and capturing streams are refused before
    anything runs."""
    _, w = packed_weight(8, 64, 32, False, 1)
    x = torch.zeros((17, 64), dtype=BF, device=DEV)
    with pytest.raises(nv.NVFP4Error):
        int4.gemv_w4a16(x, *w, group_size=32)
    with pytest.raises(ValueError):
        int4.gemv_w4a16(x[:1].cpu(), *w, group_size=32)
    with pytest.raises(ValueError):
        int4.rmsnorm_quant8(x, torch.ones(64))
    with pytest.raises(ValueError):
        int4.quantize(torch.zeros((4, 64)))
    with pytest.raises(nv.NVFP4Error):
        int4.quantize(torch.zeros((4, 48), device=DEV), 32)
    marker = torch.zeros(1, device=DEV)
    y = torch.full((1, 8), 7.0, device=DEV)
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    with torch.cuda.graph(g, stream=side):
        marker.add_(1.0)                             # one node, so the graph is not empty; it is never replayed
        with pytest.raises(nv.NVFP4Error, match="not capture-safe"):
            int4.gemv_w4a16(x[:1], *w, group_size=32, out=y)
        with pytest.raises(nv.NVFP4Error, match="not capture-safe"):
            int4.rmsnorm_quant8(x)
        st = int4.lib().int4_gemv_w4a16(p(x), p(w[0]), p(w[1]), p(w[2]), 32, 1, 8, 64, p(y), int4.F32,
                                        ctypes.c_void_p(side.cuda_stream))
    torch.cuda.synchronize()
    assert st == nv.ERR_CAPTURE and bool((y == 7).all())


# ---- far values, exact sums, long loops

def check_norm_nearest(x, r, wt, eps, group, dtype):
    """check_norm for inputs whose quotients may lie closer to half way than
    fp64 tells: with eps = 1e-6 and h far below it 1 / sqrt(eps) is 1000 to
    within 2^-55, and y / scale can be a half to within 2^-55 too (110.5 +
    2.5e-15 is one of these), where the order of two fp64 products decides.
    A code then is a nearest one to within the error of either side.  That is
    below 2^-45 of the quotient: at most 74 additions of squares (64 a thread
    and 10 exchanges; numpy's pairwise sums fewer), of which the root halves the
    effect, and fewer than 30 further roundings, each 2^-53: 67 x 2^-53 < 2^-46.
    (A quotient further than that from half way has one nearest code, so all
    codes of ordinary quotients are equal.)"""
    xf, rf, wf = f32(x), None if r is None else f32(r), f32(wt)
    q, s, h = int4.rmsnorm_quant8(x, wt, residual=r, eps=eps, group_size=group, out_dtype=dtype)
    e4m3 = dtype == torch.float8_e4m3fn
    rq, rs, rh = ref.rmsnorm_quant8(xf, wf, rf, r is not None, eps, group, e4m3)
    assert np.array_equal(f32(s), rs), f"scales: {np.abs(f32(s) / rs - 1).max()}"
    assert h is None if r is None else np.array_equal(f32(h), rh)
    codes = e4m3_values(q) if e4m3 else q.cpu().numpy().astype(np.float64)
    d = (xf if r is None else rh).astype(np.float64)
    with np.errstate(divide="ignore"):
        inv = 1 / np.sqrt((d * d).sum(1) / d.shape[1] + eps)
    inv[~d.any(1)] = 0
    v = d * wf * inv[:, None] / ref.per_element(rs, d.shape[1], group or d.shape[1])
    off = np.abs(v - codes) > np.abs(v - rq) + 2 * 2.0 ** -45 * np.abs(v)
    assert not off.any(), f"{off.sum()} of {off.size} codes are not nearest"


NORM_EXTREMES = [16, 64, 256, 1040, 4096, 8208, 14336, 16400, 65536]


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn], ids=["int8", "e4m3"])
@pytest.mark.parametrize("cols", NORM_EXTREMES)
def test_norm_where_products_leave_fp32(cols, dtype):
    """bf16 values and weights whose products pass fp32's range at either end
    although the norm and its scale are ordinary: whole rows, and single groups
    of a row beside ordinary ones."""
    g = rng(cols)
    sign = lambda: g.choice([1.0, -1.0], cols)  # noqa: E731
    x = g.standard_normal((7, cols))
    x[1] = 2.0 ** 127 * sign()                                # h w passes the largest value
    x[2] = 2.0 ** 126 * g.uniform(0.5, 1.9, cols) * sign()
    x[3] = 2.0 ** -70 * g.uniform(0.5, 2, cols) * sign()      # with a small weight: below the normal range
    x[4] = 2.0 ** -120 * g.uniform(0.5, 2, cols) * sign()     # ... and below the smallest value
    x[5] = 0
    x[6, : cols // 2] *= 2.0 ** -100                          # some groups only
    x[6, cols // 2] = 2.0 ** 127
    r = np.zeros((7, cols))
    r[2], r[3] = -x[2] / 2, x[3]
    weights = [np.full(cols, 2.0), np.exp2(g.uniform(1, 60, cols)) * sign(), np.exp2(g.uniform(-75, -65, cols)),
               np.where(np.arange(cols) % 128 < 64, 2.0 ** -80, 2.0 ** 40)]
    for i, w in enumerate(weights):
        for eps in (0.0, 1e-6):
            for group in (0, 32, 64, 128):
                print(f"[case] norm extremes {cols} weight {i} eps={eps} group={group} {dtype}", flush=True)
                check_norm_nearest(tensor(x, BF), tensor(r, BF) if i % 2 else None, tensor(w, BF), eps, group, dtype)


def exact_product(kind, M, N, K, group, grouped, seed):
    """Inputs whose differences code - zero are few and small while codes, zero
    points and activations are not, and scales of 8 significant bits: each
    group's sums of x code and of x are whole numbers below 2^24, and the sums
    of s sx x (code - zero) are multiples of 2^-7 below 2^17 in any order, so
    the product is exact wherever a group's difference is taken before its
    scale.  (device arguments, weight, the product)"""
    g = rng(seed)
    G = -(-K // group)
    zeros = g.integers(1, 15, (N, G)).astype(np.uint8)
    d = np.where(g.random((N, K)) < min(0.1, 400 / K), g.choice([-1, 1], (N, K)), 0)
    codes = (np.repeat(zeros, group, 1)[:, :K] + d).astype(np.uint8)
    scales = g.integers(129, 256, (N, G)) / 128
    x = (8 * g.integers(8, 16, (M, K)) if kind == "e4m3" else g.integers(64, 128, (M, K))).astype(np.float64)
    w = (torch.from_numpy(ref.pack(codes)).to(DEV), tensor(scales, BF), torch.from_numpy(zeros).to(DEV))
    v = x
    if kind == "bf16":
        args = (tensor(x, BF),)
    else:
        sx = g.integers(1, 3, (M, G if grouped else 1)).astype(np.float64)
        args = (tensor(x).to(torch.int8 if kind == "int8" else torch.float8_e4m3fn), tensor(sx))
        v = x * (ref.per_element(sx, K, group) if grouped else sx)
    sd = ref.per_element(scales, K, group) * d
    for m in range(M):                                       # sums of any runs of 32: all partial sums stay below 2^17
        parts = np.abs((v[m] * sd[:64]).reshape(-1, K // 32, 32).sum(2)).sum(1)
        assert parts.max() < 2.0 ** 17
    return args, w, v @ sd.T


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M", [1, 3, 8, 16])
def test_products_take_the_zero_point_off_inside_the_group(kind, M):
    """The sums of x (code - zero) of a group are formed before they meet its
    scale: exact here, however large the parts they are the difference of."""
    for N, K, group, grouped in ((48, 4096, 128, True), (37, 8704, 32, False), (37, 4128, 64, True),
                                 (4200, 1056, 64, False), (4200, 8704, 128, True), (8200, 544, 32, True),
                                 (8200, 4608, 128, False)):
        print(f"[case] exact {kind} M={M} N={N} K={K} group={group} grouped={grouped}", flush=True)
        args, w, want = exact_product(kind, M, N, K, group, grouped, M + N + K)
        y = f32(call(kind, args, w, group, FL)).astype(np.float64)
        assert np.array_equal(y, want), f"{(y != want).sum()} of {y.size} differ, worst {np.abs(y - want).max()}"


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M,N,K,group", [(1, 48, 8704, 32), (1, 5000, 4096, 128), (3, 40, 14336, 64),
                                         (16, 4200, 1056, 64), (8, 8200, 4608, 128)])
def test_products_stay_within_the_stated_bound(kind, M, N, K, group):
    """The bound of include/int4.h, of which INT8 has only the part of the sums
    over groups, for activations of both signs and of one."""
    (codes, scales, zeros), w = packed_weight(N, K, group, False, 81)
    for grouped in (False, True):
        for one_sign in (False, True):
            print(f"[case] bound {kind} M={M} N={N} K={K} group={group} {grouped} {one_sign}", flush=True)
            args, v = activations(kind, M, K, group, grouped, 82)
            if one_sign:
                x = args[0].float().abs().clamp(max=127 if kind == "int8" else 3e38)
                args = (x.to(args[0].dtype),) + args[1:]
                v = f32(x).astype(np.float64)
                if kind != "bf16":
                    sx = f32(args[1]).astype(np.float64)
                    v = v * (ref.per_element(sx, K, group) if grouped else sx)
            y = f32(call(kind, args, w, group, FL)).astype(np.float64)
            s, d = ref.per_element(scales, K, group), codes.astype(np.float64) - ref.per_element(zeros, K, group)
            ystar, a = ref.product(v, codes, scales, zeros, group)
            runs = np.stack([np.abs(((s * d) * v[m]).reshape(N, K // 32, 32).sum(2)).sum(1) for m in range(M)])
            tau = 2.0 ** -24 * ((0 if kind == "int8" else 129) * a + (K / 32 + 26) * runs)
            assert np.all(np.abs(y - ystar) <= tau), f"worst {np.max(np.abs(y - ystar) / tau)} of the bound"


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("M", [1, 5])
def test_products_with_scales_far_apart(kind, M):
    """Group scales whose product with the weight's leaves fp32's range though
    the result does not: each sum is scaled by one and then by the other."""
    N, K, group = 40, 4096, 128
    g = rng(61)
    G = K // group
    codes = g.integers(0, 16, (N, K)).astype(np.uint8)
    zeros = g.integers(0, 16, (N, G)).astype(np.uint8)
    codes[0] = np.repeat(zeros[0], group)                    # a row of zeros
    q = g.integers(1, 127, (M, K)) if kind == "int8" else 8 * g.integers(8, 16, (M, K))
    x = tensor(q).to(torch.int8 if kind == "int8" else torch.float8_e4m3fn)
    s0 = ref.bf16(g.uniform(1, 2, (N, G)).astype(np.float32))
    x0 = g.uniform(1, 2, (M, G)).astype(np.float32)
    packed, z = torch.from_numpy(ref.pack(codes)).to(DEV), torch.from_numpy(zeros).to(DEV)
    s, sx = (s0 * np.float32(2.0 ** -72)), (x0 * np.float32(2.0 ** -73))
    y = f32(int4.gemv_w4a8(x, tensor(sx), packed, tensor(s, BF), z, out_dtype=FL)).astype(np.float64)
    ystar, a = ref.product(q * ref.per_element(sx, K, group), codes, s, zeros, group)
    # each of the sum's operations may also round at 2^-149, fp32's last step
    assert np.all(np.abs(y - ystar) <= ref.product_bound(a, K) + (160 + K / 32) * 2.0 ** -149)
    assert np.abs(ystar[:, 1:]).max() > 2.0 ** -126 and not y[:, 0].any()
    s, sx = (s0 * np.float32(2.0 ** 10)), (x0 * np.float32(2.0 ** 120))
    y = f32(int4.gemv_w4a8(x, tensor(sx), packed, tensor(s, BF), z, out_dtype=FL))
    assert not y[:, 0].any()                                 # not 0 times infinity


@pytest.mark.parametrize("M,N", [(1, 48), (1, 4200), (4, 48), (16, 8200)])
def test_products_of_bf16_below_the_normal_range(M, N):
    """Activations that are whole multiples of bf16's smallest value count."""
    K, group = 640, 64
    (codes, _, zeros), w = packed_weight(N, K, group, False, 71)
    v = rng(72).integers(-3, 4, (M, K)).astype(np.float64)
    x = tensor(v * 2.0 ** -133, BF)
    s = torch.full_like(w[1], 1024.0)
    y = f32(int4.gemv_w4a16(x, w[0], s, w[2], group, FL)).astype(np.float64)
    want = v @ (codes.astype(np.float64) - ref.per_element(zeros, K, group)).T * 2.0 ** -123
    assert np.array_equal(y, want)


def product_on_gpu(v, w, group):
    """ref.product in fp64 torch, for large weights."""
    codes, scales, zeros = w
    c = codes.reshape(codes.shape[0], -1, 1, 4)
    c = torch.cat([c & 15, c >> 4], 2).reshape(codes.shape[0], -1).double()
    K = c.shape[1]
    spread = lambda t: t.double().repeat_interleave(group, 1)[:, :K]  # noqa: E731
    s = spread(scales)
    z = 8.0 if zeros is None else spread(zeros)
    y = v @ (s * (c - z)).T.contiguous()
    return y.cpu().numpy(), (v.abs() @ (s * (c + z)).T.contiguous()).cpu().numpy()


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("M,N,K,group,symmetric,grouped", [
    (5, 5000, 8704, 128, False, True), (16, 5000, 8224, 64, True, False), (1, 6000, 9216, 32, False, True),
    (16, 8200, 8704, 32, True, True), (1, 8300, 12288, 128, False, False), (8, 8250, 12320, 64, False, True),
    (3, 8200, 8224, 128, True, False), (16, 14336, 4096, 128, False, True)])
def test_products_in_several_passes(kind, M, N, K, group, symmetric, grouped):
    """Waves that go over their part of K more than once, with two and four row
    tiles, K a multiple of 512 and not; and a full batch on a layer's weight."""
    print(f"[case] passes {kind} M={M} N={N} K={K} group={group} sym={symmetric} grouped={grouped}", flush=True)
    _, w = packed_weight(N, K, group, symmetric, M + N + K)
    args, v = activations(kind, M, K, group, grouped, M + K)
    ystar, a = product_on_gpu(torch.from_numpy(v).to(DEV), w, group)
    err = np.abs(f32(call(kind, args, w, group, FL)) - ystar)
    tau = ref.product_bound(a, K)
    assert np.all(err <= tau), f"{(err > tau).sum()} of {err.size} outputs off; worst {np.max(err / tau)} of the bound"


def test_every_entry_point_refuses_a_capturing_stream():
    """Nothing is launched and no output changes."""
    _, (c, s, z) = packed_weight(8, 64, 32, False, 1)
    x, x8 = torch.ones((1, 64), dtype=BF, device=DEV), torch.ones((1, 64), dtype=torch.int8, device=DEV)
    xs, w = torch.ones((1, 1), device=DEV), torch.ones((8, 64), device=DEV)
    y, d = torch.full((1, 8), 7.0, device=DEV), torch.full((8, 64), 7.0, device=DEV)
    q, qs, h = torch.full_like(x8, 7), torch.full_like(xs, 7.0), torch.full_like(x, 7.0)
    c2, s2, z2 = torch.full_like(c, 7), torch.full_like(s, 7.0), torch.full_like(z, 7)
    marker = torch.zeros(1, device=DEV)
    torch.cuda.synchronize()
    L, side, graph = int4.lib(), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    st = ctypes.c_void_p(side.cuda_stream)
    with torch.cuda.graph(graph, stream=side):
        marker.add_(1.0)                             # one node, so the graph is not empty; it is never replayed
        got = [L.int4_quantize(p(w), int4.F32, 8, 64, 32, p(c2), p(s2), p(z2), st),
               L.int4_dequant(p(c), p(s), p(z), 8, 64, 32, p(d), int4.F32, st),
               L.int4_gemv_w4a16(p(x), p(c), p(s), p(z), 32, 1, 8, 64, p(y), int4.F32, st),
               L.int4_gemv_w4a8(p(x8), int4.I8, p(xs), 0, p(c), p(s), p(z), 32, 1, 8, 64, p(y), int4.F32, st),
               L.int4_rmsnorm_quant8(p(x), int4.BF16, 64, p(x), int4.BF16, 64, None, 0, 1e-6, 1, 64, 0, int4.I8, p(q),
                                     p(qs), p(h), st)]
    torch.cuda.synchronize()
    assert got == [nv.ERR_CAPTURE] * 5
    assert all(bool((t.float() == 7).all()) for t in (y, d, q, qs, h, c2, s2, z2))
