"""The error bounds that include/fp8.h gives for the product: what the FP8
matrix instruction cuts off is bounded by the largest term of each 8 columns,
and fp32 outputs hold fp32 sums at every size."""
import pytest
import torch

from dit_quantization_amd import fp8
from tests.test_gpu_fp8 import BF, DEV, FL, HALF_BF16, U32, operand, scales

pytestmark = pytest.mark.gpu


def terms(x, xs, w, ws):
    """Scaled operands in fp64."""
    k = torch.arange(x.shape[1], device=DEV) // 128
    return x.double() * xs.double()[:, k], w.double() * ws.double()[torch.arange(w.shape[0], device=DEV) // 128][:, k]


def largest_of_8(X, W):
    """The largest term's magnitude of each 8 columns, added up, for each output."""
    total = torch.zeros(X.shape[0], W.shape[0], dtype=torch.float64, device=DEV)
    X, W = X.abs().t().contiguous(), W.abs().t().contiguous()
    for j in range(0, X.shape[0], 8):
        most = torch.zeros_like(total)
        for i in range(j, min(j + 8, X.shape[0])):
            torch.maximum(most, X[i, :, None] * W[i], out=most)
        total += most
    return total


# rows kernels, and each kernel of many rows (16-byte stores or not, a short last block or not)
SIZES = [(16, 300, 1040), (65, 384, 1040), (300, 1024, 14336), (131, 2137, 1040), (390, 1411, 4112), (40, 8400, 656),
         (700, 2056, 4112), (513, 5016, 1040), (900, 8752, 528), (2000, 16600, 656)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", ["plain", "loud"])
def test_product_bound(M, N, K, kind):
    """tau as the header has it: (K + 4) 2^-24 of all terms' magnitudes for fp32's
    sums and the scales, for bf16 outputs of many rows 7 2^-13 of the largest term
    of each 8 columns, and bf16's half step of the result."""
    print(f"[case] gemm bound {kind} {M}x{N}x{K}", flush=True)
    x, w = operand(M, K, 101, kind), operand(N, K, 102, kind)
    G = -(-K // 128)
    xs, ws = scales(M, G, seed=103), scales(-(-N // 128), G, seed=104)
    X, W = terms(x, xs, w, ws)
    ystar, a = X @ W.t().contiguous(), X.abs() @ W.abs().t().contiguous()
    sums = (K + 4) * U32 * a
    err = (fp8.gemm(x, xs, w, ws, out_dtype=FL).double() - ystar).abs()
    assert bool((err <= sums).all()), f"fp32: worst {float((err / sums).max())} of the bound"
    many = M > 16 and -(-M // 32) * -(-N // 16) > 512
    tau = sums + (7 * 2.0 ** -13 * largest_of_8(X, W) if many else 0)
    tau = tau * (1 + HALF_BF16) + HALF_BF16 * ystar.abs()
    err = (fp8.gemm(x, xs, w, ws).double() - ystar).abs()
    assert bool((err <= tau).all()), f"bf16: worst {float((err / tau).max())} of the bound"
