"""The 8-bit layers (include/fp8.h) at the ends of what the calls take: the longest
rows in every kernel of many rows, outputs of millions of columns, calls of
several launches."""
import pytest
import torch

from dit_quantization_amd import fp8
from tests.test_gpu_fp8 import BF, DEV, E4, FL, I8, operand

pytestmark = pytest.mark.gpu
ONE = 0x38  # 1.0 in E4M3


def sparse(rows, K, hot, seed, rest):
    """Codes [rows, K]: whole numbers of -2..2 in the columns `hot`, the byte `rest` elsewhere, and NaN codes behind."""
    whole = torch.full((rows * K + 4096,), rest, dtype=torch.uint8, device=DEV)
    whole[rows * K:] = 0x7F
    t = whole[:rows * K].view(rows, K)
    v = torch.randint(-2, 3, (rows, hot.numel()), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).float()
    t[:, hot] = v.to(E4).view(torch.uint8)
    return t.view(E4), v


# bf16: tiles of 32 x 64, 64 x 64, 64 x 128, 128 x 128, 128 x 256, 256 x 256, with short last panels of both operands, and
# two launches. To fp32 the second to fourth are 64 x 64, 64 x 128 and 128 x 128.
LONGEST = [(40, 4200), (390, 1411), (700, 2056), (900, 3500), (1000, 5000), (2900, 4100), (2300, 4100)]


# 32768 blocks of columns and, in the last K, 32767
@pytest.mark.parametrize("K", [1 << 22, (1 << 22) - 16, (1 << 22) - 240])
@pytest.mark.parametrize("M,N", LONGEST)
def test_longest_rows(M, N, K):
    """K = 2^22 (panels of 256 rows are 2^30 bytes) and a little less: columns at both ends of the rows, at the ends of
    the last blocks, and some between; ones in the weight elsewhere, so that a wrong column of x or of the weight counts."""
    print(f"[case] gemm {M}x{N}x{K}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    hot = torch.cat([torch.arange(40, device=DEV), torch.arange(K - 300, K, device=DEV),
                     torch.randint(40, K - 300, (300,), generator=g, device=DEV)]).unique()
    x, xv = sparse(M, K, hot, 2, 0)
    w, wv = sparse(N, K, hot, 3, ONE)
    G = -(-K // 128)
    xs, ws = torch.ones(M, G, device=DEV), torch.ones(-(-N // 128), G, device=DEV)
    xs[1::2] = 0.5
    ws[1::2] = 2.0
    want = (xv @ wv.t().contiguous()) * xs[:, :1] * ws[torch.arange(N, device=DEV) // 128, 0]
    assert torch.equal(fp8.gemm(x, xs, w, ws, out_dtype=FL), want)
    assert torch.equal(fp8.gemm(x, xs, w, ws), want.to(BF))


@pytest.mark.parametrize("M,N,K", [(300, (1 << 21) + 264, 272), (257, (1 << 21) + 5, 400), (5, (1 << 22) + 130, 272)])
def test_millions_of_columns(M, N, K):
    """Rows of y that 256 of them pass 2^30 bytes."""
    print(f"[case] gemm {M}x{N}x{K}", flush=True)
    x, w = operand(M, K, 11, "whole"), operand(N, K, 12, "whole")
    G = -(-K // 128)
    xs, ws = torch.ones(M, G, device=DEV), torch.ones(-(-N // 128), G, device=DEV)
    for dtype in (BF, FL):
        y = fp8.gemm(x, xs, w, ws, out_dtype=dtype)
        for n in (*range(0, N, 1 << 19), N - 5000):
            part = w[n:n + 5000].float().t().contiguous()
            assert torch.equal(y[:, n:n + 5000], (x.float() @ part).to(dtype))
        del y


def near(boundary, rows):
    return torch.cat([torch.arange(300), torch.arange(boundary - 300, boundary + 300), torch.arange(rows - 300, rows)]).unique().to(DEV)


def test_product_of_several_launches():
    """2^29 + 777 rows of 16 columns: more tiles than a launch has."""
    M, N, K = (1 << 29) + 777, 16, 16
    x, w = torch.zeros(M, K, dtype=torch.uint8, device=DEV).view(E4), operand(N, K, 21, "whole")
    xs, ws = torch.ones(M, 1, device=DEV), torch.ones(1, 1, device=DEV)
    for boundary in (1 << 27, 1 << 28, 1 << 29):
        rows = near(boundary, M)
        part = operand(rows.numel(), K, 22, "whole")
        x.view(torch.uint8)[rows] = part.view(torch.uint8)
    y = fp8.gemm(x, xs, w, ws)
    for boundary in (1 << 27, 1 << 28, 1 << 29):
        rows = near(boundary, M)
        assert torch.equal(y[rows], (x[rows].float() @ w.float().t().contiguous()).to(BF))
    assert not bool(y[1000:2000].any())


def test_quantizers_of_several_launches():
    """Weights of 2^29 + 300 rows and activations of 2^30 + 300, of 16 columns."""
    g = torch.Generator(device=DEV).manual_seed(31)
    N, K = (1 << 29) + 300, 16
    w = torch.zeros(N, K, dtype=BF, device=DEV)
    rows = near(1 << 29, N)
    w[rows] = torch.randn(rows.numel(), K, generator=g, device=DEV).to(BF)
    c, s = fp8.quantize(w)
    for a in (0, (1 << 29) - 384, 1 << 29):
        cw, sw = fp8.quantize(w[a:a + 384])
        n = sw.shape[0]
        assert torch.equal(c[a:a + 384].view(torch.uint8), cw.view(torch.uint8)) and torch.equal(s[a // 128:a // 128 + n], sw)
    assert bool((s[100:200] == 1).all()) and not bool(c[12800:25600].view(torch.uint8).any())
    del w, c
    M = (1 << 30) + 300
    x = torch.zeros(M, K, dtype=BF, device=DEV)
    rows = near(1 << 30, M)
    x[rows] = torch.randn(rows.numel(), K, generator=g, device=DEV).to(BF)
    for dtype in (E4, I8):
        c, s = fp8.quantize_act(x, group_size=32, out_dtype=dtype)
        for a in (0, (1 << 30) - 300, 1 << 30):
            cx, sx = fp8.quantize_act(x[a:a + 300].contiguous(), group_size=32, out_dtype=dtype)
            assert torch.equal(c[a:a + 300].view(torch.uint8), cx.view(torch.uint8)) and torch.equal(s[a:a + 300], sx)
        del c
