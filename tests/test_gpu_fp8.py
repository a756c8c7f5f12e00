"""GPU parity of the 8-bit layers (include/fp8.h) with the plain fp64 forms of
tests/eight_bit_reference.py: codes and scales bit for bit, products exact on
small whole numbers and within a derived bound otherwise."""
import numpy as np
import pytest
import torch

from dit_quantization_amd import fp8, int4
from dit_quantization_amd import nvfp4 as nv
from tests import eight_bit_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FL, E4, I8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8
HALF_BF16 = 2.0 ** -8                    # half a step, relative
U32 = 2.0 ** -24


def rng(seed):
    return np.random.default_rng(seed)


def tensor(a, dtype=FL):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)


def host(t):
    return t.float().cpu().numpy() if t.dtype == BF else t.cpu().numpy()


def values(codes):
    return codes.cpu().numpy().astype(np.float64) if codes.dtype == I8 else ref.e4m3_values(codes.view(torch.uint8).cpu().numpy())


# ---- the weight quantizer

def weights(rows, cols, seed, kind):
    g = rng(seed)
    w = (g.standard_t(5, (rows, cols)) * 0.02).astype(np.float32)
    if kind == "edges":
        block = np.arange(rows)[:, None] // 128 + np.arange(cols) // 128
        w = np.where(block % 5 == 1, np.float32(0), w)                                       # blocks of zeros
        w = np.where(block % 5 == 2, g.integers(-28, 29, w.shape).astype(np.float32) / 64, w)    # ties, with the next line
        w[(block % 5 == 2) & (np.arange(rows)[:, None] % 7 == 0)] = 0.4375                   # s = 2^-10
        w = np.where(block % 5 == 3, w * np.float32(1e-38), w)                               # scales below the normal range
        w = np.where(block % 5 == 4, np.where(g.random(w.shape) < 0.5, np.float32(-0.0), w * np.float32(1e37)), w)
    if kind == "ties":
        # maxima of 7 2^j give scales that are powers of two; multiples of half a step everywhere
        w = (g.integers(-448 * 32, 448 * 32 + 1, w.shape) / 32).astype(np.float32)
        w[::128, ::128] = 448.0
    if kind == "denormal":
        w = (np.float32(1e-45) * g.integers(-4000, 4001, w.shape)).astype(np.float32)
    return w


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (127, 144), (128, 128), (129, 400), (260, 1040), (5, 14336)])
@pytest.mark.parametrize("kind", ["plain", "edges", "ties", "denormal"])
@pytest.mark.parametrize("bf16", [False, True])
def test_quantize(rows, cols, kind, bf16):
    print(f"[case] quantize {rows}x{cols} {kind} bf16={bf16}", flush=True)
    w = tensor(weights(rows, cols, rows + cols, kind), BF if bf16 else FL)
    codes, scales = fp8.quantize(w)
    rc, rs = ref.quantize_blocks(host(w))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(values(codes), rc)


def test_quantize_strided_rows_and_only_its_outputs():
    wide = tensor(weights(131, 208 + 64, 5, "plain"), BF)
    w = wide[:, 32:32 + 208]
    whole = torch.full((131 * 208 + 64,), 77, dtype=torch.uint8, device=DEV)
    sw = torch.full((4 + 16,), 3.0, device=DEV)
    out = (whole[:131 * 208].view(131, 208).view(E4), sw[:4].view(2, 2))
    assert fp8.quantize(w, out=out)[0] is out[0]
    rc, rs = ref.quantize_blocks(host(w))
    assert np.array_equal(values(out[0]), rc) and np.array_equal(out[1].cpu().numpy(), rs)
    assert bool((whole[131 * 208:] == 77).all()) and bool((sw[4:] == 3.0).all())


def test_quantize_offsets_past_32_bits():
    """2^19 + 1 rows of 4112 bf16 columns (4.3 GB): the first and the last rows of blocks."""
    rows, cols = (1 << 19) + 1, 4112
    w = torch.empty(rows, cols, dtype=BF, device=DEV)
    w.view(torch.int16).fill_(0x3C00)
    g = rng(9)
    first, last = tensor(g.standard_normal((128, cols)), BF), tensor(g.standard_normal((129, cols)), BF)
    w[:128], w[-129:] = first, last
    codes, scales = fp8.quantize(w)
    for part, at, s_at in ((first, slice(0, 128), slice(0, 1)), (last, slice(rows - 129, rows), slice(-2, None))):
        rc, rs = ref.quantize_blocks(host(part))
        assert np.array_equal(values(codes[at]), rc) and np.array_equal(scales[s_at].cpu().numpy(), rs)


# ---- the activation quantizer

def acts(rows, cols, seed, kind):
    g = rng(seed)
    x = g.standard_normal((rows, cols)).astype(np.float32)
    gate = (g.standard_normal((rows, cols)) * 3).astype(np.float32)
    x[:, g.random(cols) < 0.02] *= 20
    if kind == "edges":
        x[0, :] = 0
        gate.flat[::7] = [0.0]
        gate.flat[3::11] = -0.0
        gate.flat[5::13] = 100.0
        gate.flat[6::13] = -100.0
        gate.flat[8::17] = -1e4
        gate.flat[9::17] = 1e4
        if rows > 1:
            gate[1] = -95.0           # products below fp32's normal range
        if rows > 2:
            gate[2] = -1e30           # and below fp64's: zeros
        if rows > 3:
            x[3] *= np.float32(1e-42)
        if rows > 4:
            x[4] *= np.float32(1e36)
            gate[4] = np.clip(gate[4], -9, 9)
        if rows > 5:
            x[5] = (g.integers(-254, 255, cols) / 2).astype(np.float32)    # ties, INT8 without a gate
            x[5, ::32] = 127.0
    return x, gate


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (7, 80), (9, 144), (64, 128), (33, 1040), (3, 14336)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("silu", [False, True])
def test_quantize_act(rows, cols, group, bf16, silu):
    print(f"[case] act {rows}x{cols} group={group} bf16={bf16} silu={silu}", flush=True)
    for kind in ("plain", "edges"):
        x, gate = (tensor(t, BF if bf16 else FL) for t in acts(rows, cols, rows + cols, kind))
        gate = gate if silu else None
        y = ref.silu_product(host(x), None if gate is None else host(gate))
        for dtype in (E4, I8):
            codes, scales = fp8.quantize_act(x, gate, group, dtype)
            rc, rs = ref.quantize_groups(y, group, dtype == E4)
            assert np.array_equal(scales.cpu().numpy(), rs), kind
            assert np.array_equal(values(codes), rc), kind


@pytest.mark.parametrize("seed", range(4))
def test_quantize_act_many(seed):
    """A million gated products: every border between codes is met closely."""
    for bf16 in (True, False):
        x, gate = (tensor(t, BF if bf16 else FL) for t in acts(256, 4096, seed, "plain"))
        y = ref.silu_product(host(x), host(gate))
        for dtype, group in ((E4, 128), (I8, 64)):
            codes, scales = fp8.quantize_act(x, gate, group, dtype)
            rc, rs = ref.quantize_groups(y, group, dtype == E4)
            assert np.array_equal(scales.cpu().numpy(), rs) and np.array_equal(values(codes), rc)


@pytest.mark.parametrize("rows", [65536, 640])
def test_quantize_act_every_gate(rows):
    """All finite bf16 gates (a group each), or every hundredth: the scale has 24 bits of SiLU(gate) in every
    group."""
    bits = torch.arange(0, 65536, 65536 // rows, dtype=torch.int32, device=DEV)[:rows]
    g = (bits << 16).view(FL)
    g = torch.where(torch.isfinite(g), g, 0.0)
    gate = g.to(BF)[:, None].expand(rows, 128).contiguous()
    x = torch.ones(rows, 128, dtype=BF, device=DEV)
    x[:, 1::2] = 0.8125
    y = ref.silu_product(host(x), host(gate))
    rc, rs = ref.quantize_groups(y, 32, True)
    c, s = fp8.quantize_act(x, gate, group_size=32)
    # Bit for bit but for scales that fp64 cannot decide (include/fp8.h: within 2^-44 of a border).  There are such:
    # SiLU(g) = g/2 + g^2/4 - g^4/48 ..., and for g = 1.5 2^-24, say, (g/2 + g^2/4) / 448 = 2^-34 12/7 (1 + 0.75 2^-24)
    # lies half way between two fp32 numbers (12/7 2^23 = .. + 6/7, and 12/7 2^23 0.75 2^-24 = 9/14, together 3/2), with
    # the true value 2^-76 of itself below.
    got, exact = host(s), np.abs(y).reshape(rows, 4, 32).max(2) / 448
    off = got != rs
    half_way = (got.astype(np.float64) + rs.astype(np.float64)) / 2
    assert (np.abs(got.view(np.int32) - rs.view(np.int32))[off] == 1).all()
    assert (np.abs(exact - half_way)[off] <= 2.0 ** -44 * exact[off]).all() and off.sum() < 64
    # (the codes of these do not depend on which of the two scales it is)
    assert np.array_equal(values(c), rc)


def test_quantize_act_halves_of_a_product_and_only_its_outputs():
    F = 208
    h = tensor(rng(3).standard_normal((5, 2 * F)), BF)
    whole = torch.full((5 * F + 64,), 77, dtype=torch.uint8, device=DEV)
    sw = torch.full((10 + 16,), 3.0, device=DEV)
    out = (whole[:5 * F].view(5, F).view(E4), sw[:10].view(5, 2))
    fp8.quantize_act(h[:, F:], gate=h[:, :F], out=out)
    rc, rs = ref.quantize_groups(ref.silu_product(host(h)[:, F:], host(h)[:, :F]), 128, True)
    assert np.array_equal(values(out[0]), rc) and np.array_equal(out[1].cpu().numpy(), rs)
    assert bool((whole[5 * F:] == 77).all()) and bool((sw[10:] == 3.0).all())


# ---- the product

def operand(rows, cols, seed, kind):
    """E4M3 codes in a larger buffer of NaN codes (0x7F) before and behind them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    whole = torch.full((rows * cols + 4096,), 0x7F, dtype=torch.uint8, device=DEV)
    t = whole[1024:1024 + rows * cols].view(rows, cols).view(E4)
    if kind == "whole":
        v = torch.randint(-2, 3, (rows, cols), generator=g, device=DEV).float()
    else:
        v = torch.randn(rows, cols, generator=g, device=DEV) * 100
        if kind == "loud":
            v *= torch.where(torch.rand(cols, generator=g, device=DEV) < 0.02, 1.0, 0.02)
    t.copy_(v.clamp(-448, 448).to(E4))
    return t


def scales(*shape, seed, power=False):
    """Scales (powers of two, so that a product of whole numbers stays exact), and NaN behind them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = int(np.prod(shape))
    whole = torch.full((n + 64,), float("nan"), device=DEV)
    s = whole[:n].view(*shape)
    e = torch.randint(-2, 3, shape, generator=g, device=DEV).float()
    s.copy_(torch.exp2(e) if power else torch.exp2(e) * (1 + torch.rand(shape, generator=g, device=DEV)) * 1e-3)
    return s


def product(x, xs, w, ws):
    """(y, sum |p|, fp64) of the scaled operands on the GPU, and the largest product of each 8 columns, added up."""
    K, N = x.shape[1], w.shape[0]
    k = torch.arange(K, device=DEV) // 128
    X = x.double() * xs.double()[:, k]
    W = w.double() * ws.double()[torch.arange(N, device=DEV) // 128][:, k]
    y, a = X @ W.t().contiguous(), X.abs() @ W.abs().t().contiguous()
    return y, a


def check_product(y, x, xs, w, ws):
    """fp32 sums in any order, bf16's rounding, and for bf16 outputs the FP8
    matrix instruction: it aligns the products of 8 neighbouring columns to the
    largest and cuts them off 13 bits below that one's exponent, so that each of
    the 7 others loses less than 2^-13 of it: 7 2^-13 of the largest of 8,
    which is at most their sum."""
    ystar, a = product(x, xs, w, ws)
    K = x.shape[1]
    # additions in a block, of blocks, the scales' two products
    tau = (K + 4) * U32 * a
    if y.dtype == BF:
        tau = tau + 7 * 2.0 ** -13 * a
        tau = tau * (1 + HALF_BF16) + HALF_BF16 * ystar.abs()
    err = (y.double() - ystar).abs()
    bad = err > tau
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outputs, worst {float((err / tau).max())} of the bound"
    # the errors of different columns do not pile up: on the whole well inside the bound
    return float((err / a.clamp(min=1e-300)).max())


SIZES = [(1, 1, 16), (1, 16, 128), (1, 300, 144), (2, 1024, 4096), (5, 129, 1040), (15, 17, 272), (16, 128, 4112),
         (17, 257, 128), (33, 64, 656), (64, 200, 1040), (65, 384, 272), (100, 1000, 528), (128, 130, 2064), (130, 257, 400),
         (255, 129, 144), (257, 513, 384), (333, 700, 1040), (512, 512, 512), (777, 1100, 256), (1030, 2056, 144)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, FL])
def test_gemm_whole_numbers(M, N, K, dtype):
    """Codes of -2..2 and scales that are powers of two: every partial sum is a
    multiple of 2^-4 below 2^18, so fp32 has the result exactly."""
    print(f"[case] gemm whole {M}x{N}x{K} {dtype}", flush=True)
    x, w = operand(M, K, 1, "whole"), operand(N, K, 2, "whole")
    G = -(-K // 128)
    xs, ws = scales(M, G, seed=3, power=True), scales(-(-N // 128), G, seed=4, power=True)
    whole = torch.full((M * N + 64,), 5.0, dtype=dtype, device=DEV)
    out = whole[:M * N].view(M, N)
    assert fp8.gemm(x, xs, w, ws, out=out) is out
    ystar, _ = product(x, xs, w, ws)
    assert torch.equal(out, ystar.to(dtype))
    assert bool((whole[M * N:] == 5.0).all())


@pytest.mark.parametrize("M,N,K", SIZES + [(16, 4096, 14336), (48, 2048, 14336), (300, 1024, 14336), (1500, 4096, 1024)])
@pytest.mark.parametrize("kind", ["plain", "loud"])
def test_gemm_random(M, N, K, kind):
    print(f"[case] gemm {kind} {M}x{N}x{K}", flush=True)
    x, w = operand(M, K, 5, kind), operand(N, K, 6, kind)
    G = -(-K // 128)
    xs, ws = scales(M, G, seed=7), scales(-(-N // 128), G, seed=8)
    for dtype in (BF, FL):
        y = fp8.gemm(x, xs, w, ws, out_dtype=dtype)
        check_product(y, x, xs, w, ws)
        assert torch.equal(y, fp8.gemm(x, xs, w, ws, out_dtype=dtype)), "two calls differ"


@pytest.mark.parametrize("M", [1, 16, 40, 130, 520])
@pytest.mark.parametrize("dtype", [BF, FL])
def test_gemm_one_hot(M, dtype):
    """A single product an output: code times code and two scales, rounded."""
    N, K = 600, 656
    x, w = torch.zeros(M, K, device=DEV), operand(N, K, 11, "plain")
    at = torch.randint(0, K, (M,), generator=torch.Generator(device=DEV).manual_seed(12), device=DEV)
    x[torch.arange(M, device=DEV), at] = 448.0
    x = x.to(E4)
    xs, ws = scales(M, 6, seed=13), scales(5, 6, seed=14)
    y = fp8.gemm(x, xs, w, ws, out_dtype=dtype).double()
    ystar, _ = product(x, xs, w, ws)
    tol = 3 * U32 + (HALF_BF16 if dtype == BF else 0) * (1 + 3 * U32)
    assert bool(((y - ystar).abs() <= tol * ystar.abs()).all())


@pytest.mark.parametrize("M", [3, 40, 300])
def test_gemm_scales_at_the_ends_of_fp32(M):
    """Scales whose product leaves fp32's normal range although the result does not."""
    N, K = 300, 400
    x, w = operand(M, K, 15, "plain"), operand(N, K, 16, "plain")
    for a, b in ((1e-30, 1e-12), (1e-12, 1e-30), (1e38, 1e-30), (1e-30, 1e38), (2.0 ** -120, 2.0 ** -10), (1e-42, 1e38)):
        xs = torch.full((M, 4), a, device=DEV)
        ws = torch.full((3, 4), b, device=DEV)
        for dtype in (BF, FL):
            check_product(fp8.gemm(x, xs, w, ws, out_dtype=dtype), x, xs, w, ws)


# A size for each of the launcher's kernels (16, 32, 64, 128 and 256 rows of x a
# workgroup, with N that allows 16-byte stores and that does not), several tiles a
# workgroup, and two launches.
TILES = [(7, 9001), (9, 8904), (33, 4144), (131, 2137), (390, 1411), (40, 8400), (270, 6005), (700, 2056), (201, 8301),
         (513, 5016), (390, 9349), (1100, 6008), (1156, 6805), (900, 8752), (3300, 9001), (3300, 9000), (2000, 16600)]


@pytest.mark.parametrize("M,N", TILES)
def test_gemm_tiles(M, N):
    """1 to 6, 8 and 9 blocks of columns, the last one short or not: every remainder of a kernel's stages."""
    for K in (16, 144, 272, 384, 528, 656, 1024, 1040):
        print(f"[case] gemm tiles {M}x{N}x{K}", flush=True)
        x, w = operand(M, K, 31, "plain"), operand(N, K, 32, "plain")
        G = -(-K // 128)
        xs, ws = scales(M, G, seed=33), scales(-(-N // 128), G, seed=34)
        for dtype in (BF, FL):
            whole = torch.full((M * N + 64,), 5.0, dtype=dtype, device=DEV)
            y = fp8.gemm(x, xs, w, ws, out=whole[:M * N].view(M, N))
            check_product(y, x, xs, w, ws)
            assert bool((whole[M * N:] == 5.0).all())


@pytest.mark.parametrize("M,N", TILES)
def test_gemm_tiles_with_scales_at_the_ends_of_fp32(M, N):
    """In one of four blocks, and another one's every third row, the product of
    the scales is 2^-127, below fp32's normal numbers, elsewhere 2^-126."""
    K = 400
    x, w = operand(M, K, 35, "plain"), operand(N, K, 36, "plain")
    xs, ws = torch.full((M, 4), 2.0 ** -60, device=DEV), torch.full((-(-N // 128), 4), 2.0 ** -66, device=DEV)
    xs[:, 1], ws[:, 1] = 2.0 ** -120, 2.0 ** -7
    xs[:, 2], ws[:, 2] = 2.0 ** 13, 2.0 ** -139
    xs[::3, 2] = 2.0 ** 12
    k = torch.arange(K, device=DEV) // 128
    X = x.double() * (xs.double() * 2.0 ** 60)[:, k]
    W = w.double() * (ws.double() * 2.0 ** 66)[torch.arange(N, device=DEV) // 128][:, k]
    ystar, a = X @ W.t().contiguous(), X.abs() @ W.abs().t().contiguous()
    for dtype in (BF, FL):
        y = fp8.gemm(x, xs, w, ws, out_dtype=dtype).double() * 2.0 ** 126
        # as check_product, and half a step of fp32's smallest numbers, 2^-150, for the blocks' sums (four) and
        # their additions, of bf16's, 2^-134, for the result
        tau = (K + 4) * U32 * a + 8 * 2.0 ** (126 - 150)
        if dtype == BF:
            tau = tau + 7 * 2.0 ** -13 * a
            tau = tau * (1 + HALF_BF16) + HALF_BF16 * ystar.abs() + 2.0 ** (126 - 134)
        bad = (y - ystar).abs() > tau
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outputs"


@pytest.mark.parametrize("M,N", [(5, 264), (300, 264), (700, 2056), (513, 5016), (3300, 9000)])
def test_gemm_output_aligned_to_4_bytes(M, N):
    K = 400
    x, w = operand(M, K, 37, "whole"), operand(N, K, 38, "whole")
    xs, ws = scales(M, 4, seed=39, power=True), scales(-(-N // 128), 4, seed=40, power=True)
    want = fp8.gemm(x, xs, w, ws, out_dtype=FL)
    for dtype, at in ((BF, 2), (FL, 1), (FL, 2)):
        whole = torch.full((M * N + 64,), 5.0, dtype=dtype, device=DEV)
        fp8.gemm(x, xs, w, ws, out=whole[at:at + M * N].view(M, N))
        assert torch.equal(whole[at:at + M * N].view(M, N), want.to(dtype))
        assert bool((whole[:at] == 5.0).all()) and bool((whole[at + M * N:] == 5.0).all())


def test_gemm_many_at_once():
    """Large products on four streams at a time, which share nothing."""
    sizes = [(1300, 6000, 784), (900, 8752, 528), (3300, 9000, 400), (2000, 16600, 1040)]
    ops = []
    for i, (M, N, K) in enumerate(sizes):
        G = -(-K // 128)
        ops.append((operand(M, K, 50 + i, "plain"), scales(M, G, seed=60 + i), operand(N, K, 70 + i, "plain"),
                    scales(-(-N // 128), G, seed=80 + i)))
    want = [fp8.gemm(*o) for o in ops]
    streams = [torch.cuda.Stream() for _ in ops]
    got = [[] for _ in ops]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, g in zip(streams, ops, got):
            with torch.cuda.stream(s):
                g.append(fp8.gemm(*o))
    torch.cuda.synchronize()
    for y, g in zip(want, got):
        assert all(torch.equal(y, a) for a in g)


def test_gemm_longest_rows():
    """K = 2^22, the most the call takes: sums of 2^22 products in every tile kernel."""
    K = 1 << 22
    for M, N in ((1, 16), (20, 16), (130, 130)):
        print(f"[case] gemm {M}x{N}x{K}", flush=True)
        x, w = torch.zeros(M, K, device=DEV, dtype=torch.uint8).view(E4), operand(N, K, 17, "whole")
        hot = torch.randint(0, K, (M, 500), generator=torch.Generator(device=DEV).manual_seed(18), device=DEV)
        hot[:, 0], hot[:, 1] = 0, K - 1
        x.view(torch.uint8).scatter_(1, hot, 0x38)          # 1.0
        G = K // 128
        xs, ws = torch.ones(M, G, device=DEV), torch.ones(-(-N // 128), G, device=DEV)
        want = torch.stack([w[:, h.unique()].float().sum(1) for h in hot])
        assert torch.equal(fp8.gemm(x, xs, w, ws, out_dtype=FL), want)
        assert torch.equal(fp8.gemm(x, xs, w, ws), want.to(BF))


def test_gemm_offsets_past_32_bits():
    """x of 4.4 GB and y of 5.3 GB: the first and the last rows."""
    for M, N, K in (((1 << 20) + 37, 48, 4112), ((1 << 17) + 5, 20000, 16)):
        print(f"[case] gemm {M}x{N}x{K}", flush=True)
        x, w = torch.zeros(M, K, dtype=torch.uint8, device=DEV).view(E4), operand(N, K, 19, "whole")
        G = -(-K // 128)
        rows = torch.cat([torch.arange(40), torch.arange(M - 40, M)]).to(DEV)
        part = operand(80, K, 20, "whole")
        x.view(torch.uint8)[rows] = part.view(torch.uint8)
        xs, ws = torch.ones(M, G, device=DEV), torch.ones(-(-N // 128), G, device=DEV)
        y = fp8.gemm(x, xs, w, ws)
        assert torch.equal(y[rows], (part.float() @ w.float().t().contiguous()).to(BF))
        assert bool((y[M // 2] == 0).all())
        del x, y


# ---- calls

def test_empty_calls():
    e = torch.empty(0, 64, device=DEV)
    assert [t.shape for t in fp8.quantize(e)] == [(0, 64), (0, 1)]
    assert [t.shape for t in fp8.quantize(torch.empty(5, 0, device=DEV))] == [(5, 0), (1, 0)]
    assert [t.shape for t in fp8.quantize_act(e, e)] == [(0, 64), (0, 1)]
    w, ws = fp8.quantize(torch.randn(20, 64, device=DEV))
    assert fp8.gemm(e.to(E4), torch.empty(0, 1, device=DEV), w, ws).shape == (0, 20)
    x, xs = fp8.quantize_act(torch.randn(3, 64, device=DEV))
    assert fp8.gemm(x, xs, w[:0], ws[:0]).shape == (3, 0)


def test_side_stream_and_two_calls_at_once():
    """Calls on two streams, interleaved, give what each gives alone."""
    G = 33
    sets = []
    for seed, M in ((21, 16), (22, 300)):
        x, w = operand(M, G * 128, seed, "plain"), operand(1000, G * 128, seed + 10, "plain")
        sets.append((x, scales(M, G, seed=seed), w, scales(8, G, seed=seed + 1)))
    alone = [fp8.gemm(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(fp8.gemm(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, alone[i]) for g in got[i])


def test_capture_is_refused():
    """Inside a capture that records one unrelated node and is never replayed."""
    w = torch.randn(64, 128, device=DEV)
    x = torch.randn(2, 128, device=DEV)
    (c, s), (xq, xs) = fp8.quantize(w), fp8.quantize_act(x)
    y = torch.full((2, 64), 5.0, dtype=BF, device=DEV)
    mark = torch.zeros(4, device=DEV)
    outs = ((c.clone(), s.clone()), (xq.clone(), xs.clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mark.add_(1.0)
        for call in (lambda: fp8.quantize(w, out=outs[0]), lambda: fp8.quantize_act(x, out=outs[1]),
                     lambda: fp8.gemm(xq, xs, c, s, out=y)):
            with pytest.raises(nv.NVFP4Error) as e:
                call()
            assert e.value.status == nv.ERR_CAPTURE
    torch.cuda.synchronize()
    assert bool((y == 5.0).all())
    assert torch.equal(fp8.gemm(xq, xs, c, s, out=y), fp8.gemm(xq, xs, c, s))


def test_activations_of_a_norm_and_of_the_4_bit_product():
    """What the quantizers give is what the products of both weights take."""
    x, gain = tensor(rng(30).standard_normal((6, 512))), tensor(1 + 0.1 * rng(31).standard_normal(512))
    w = torch.randn(320, 512, generator=torch.Generator(device=DEV).manual_seed(32), device=DEV) * 0.05
    c, s = fp8.quantize(w)
    xq, xs, _ = int4.rmsnorm_quant8(x, gain, group_size=128, out_dtype=E4)
    check_product(fp8.gemm(xq, xs, c, s), xq, xs, c, s)
    gate = int4.quantize(w, 64)
    for dtype in (I8, E4):
        aq, as_ = fp8.quantize_act(x, group_size=64, out_dtype=dtype)
        y = int4.gemv_w4a8(aq, as_, *gate, group_size=64, out_dtype=FL)
        k = torch.arange(512, device=DEV) // 64
        X = aq.double() * as_.double()[:, k]
        W = int4.dequant(*gate, group_size=64).double()
        # the bound of int4.h, code + zero at most 30 and |code - zero| at most 15
        size = X.abs() @ (30 * gate[1].double()[:, k]).t().contiguous()
        assert bool(((y.double() - X @ W.t().contiguous()).abs() <= (129 + 512 // 32 + 26) * U32 * size).all())
