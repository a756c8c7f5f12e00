"""The choice of an FP8 product's kernels (csrc/fp8_plan.hpp), compiled for the
host: every plan is of kernels that can run it, estimated as what runs, and the
GPU tests' sizes reach every kernel."""
import ctypes
import os
import random
import subprocess

import pytest

from tests import test_gpu_fp8 as base
from tests import test_gpu_fp8_bounds as bounds
from tests import test_gpu_fp8_sizes as ends

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "fp8_plan.hpp"
using namespace nvfp4;
extern "C" void plan(long long M, long long N, long long K, int bf16, long long* out) {
  const Fp8Plan p = fp8_plan(M, N, K, bf16 != 0);
  out[0] = p.first, out[1] = p.second, out[2] = p.M, out[3] = p.N;
}
extern "C" double step(int kernel, int bf16, long long M, long long N) {
  for (const Fp8Tiles& t : kFp8Tiles16) if (bf16 && t.kernel == kernel) return t.step(M, N);
  for (const Fp8Tiles& t : kFp8Tiles32) if (!bf16 && t.kernel == kernel) return t.step(M, N);
  return -1;
}
"""
NAMES = ["none", "rows1x1", "rows1x2", "rows2x1", "rows2x2of8", "rows2x2of4", "32x64", "64x64", "64x128", "128x128", "128x256", "256x256"]
TILES = {True: NAMES[6:], False: ["64x64", "64x128", "128x128"]}
MAX_N = 1 << 21


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("fp8_plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dit_quantization_amd", "csrc"), "plan.cpp", "-o", "libplan.so"], cwd=d, check=True)
    L = ctypes.CDLL(str(d / "libplan.so"))
    L.plan.restype, L.plan.argtypes = None, [ctypes.c_longlong] * 3 + [ctypes.c_int, ctypes.c_void_p]
    L.step.restype, L.step.argtypes = ctypes.c_double, [ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong]
    return L


def plan(lib, M, N, K, bf16):
    out = (ctypes.c_longlong * 4)()
    lib.plan(M, N, K, bf16, out)
    return NAMES[out[0]], NAMES[out[1]], out[2], out[3]


def test_plans(lib):
    g = random.Random(1)

    def log(lo, hi):
        return int(round(lo * (hi / lo) ** g.random()))

    sizes = [(log(1, 20000), log(1, 40000), 16 * log(1, 2000)) for _ in range(3000)]
    sizes += [(log(1, 20000), log(1, 40000), g.choice([16, 128, 240, 256, 272])) for _ in range(1000)]
    sizes += [(log(1, 3000), g.choice([MAX_N - 8, MAX_N, MAX_N + 1, MAX_N + 8, 1 << 26]), 16 * log(1, 2000)) for _ in range(500)]
    sizes += [(1 << 31, 16, 16), (1 << 31, 1 << 26, 1 << 22), (1 << 31, 4096, 4096)]
    for M, N, K in sizes:
        for bf16 in (True, False):
            first, second, m, n = plan(lib, M, N, K, bf16)
            case = (M, N, K, bf16, first, second, m, n)
            if M <= 16 or -(-M // 32) * -(-N // 16) <= (512 if bf16 else 1024):
                assert first.startswith("rows") and second == "none" and (m, n) == (M, N), case
                continue
            able = [k for k in TILES[bf16] if k != "256x256" or (K > 256 and N <= MAX_N)]
            assert first in able and second in able + ["none"], case

            def us(kernel, rows, cols):
                return lib.step(NAMES.index(kernel), bf16, rows, cols)

            if second == "none":
                assert (m, n) == (M, N), case
                assert us(first, M, N) == min(us(k, M, N) for k in able), case
                continue
            # the rest are whole columns from a multiple of 128 on, or whole rows, and the sum is less by 5 %
            assert (m == M and 0 < n < N and n % 128 == 0) or (n == N and 0 < m < M), case
            rest = (M, N - n) if m == M else (M - m, N)
            assert us(second, *rest) == min(us(k, *rest) for k in able), case
            total = us(first, m, n) + us(second, *rest) + 3.0 * 128 / K
            assert total < 0.95 * min(us(k, M, N) for k in able), case


def test_gpu_tests_reach_every_kernel(lib):
    for name, K, sizes, rows in (("longest rows", 1 << 22, ends.LONGEST, {True: set(), False: set()}),
                                 ("tiles", 1040, base.TILES, {True: {"rows1x2"}, False: {"rows1x2", "rows2x2of4"}}),
                                 ("neighbours", None, bounds.NEIGHBOURS, {True: set(NAMES[1:5]), False: set(NAMES[1:6])})):
        for bf16 in (True, False):
            got = set()
            for s in sizes:
                got |= set(plan(lib, s[0], s[1], K or s[2], bf16)[:2])
            want = set(TILES[bf16]) | rows[bf16]
            assert want <= got, (name, bf16, want - got)
