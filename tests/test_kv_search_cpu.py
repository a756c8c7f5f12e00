"""The search for a row's sequence (csrc/kv_search.hpp), compiled for the host: up
to the most sequences that include/kvcache.h allows, and never an entry outside
cu."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "kv_search.hpp"
using namespace nvfp4;
template <class Cu>
static long long search(const Cu& cu, long long seqs, long long t, int* first, long long* outside) {
  int held[kCuHeld + 1];
  *outside = 0;
  const auto read = [&](long long i, long long end) {
    if (i < 0 || i >= end) { ++*outside; return 0; }
    return cu(i);
  };
  for (int k = 0; k <= kCuHeld; ++k) held[k] = read(cu_entry(k, seqs), seqs + 1);
  return sequence_of(held, [&](int64_t i) { return read(i, seqs); }, seqs, t, *first);
}
extern "C" long long of_array(const int* cu, long long seqs, long long t, int* first, long long* outside) {
  return search([=](long long i) { return cu[i]; }, seqs, t, first, outside);
}
// cu[i] = i / per, without an array
extern "C" long long of_line(long long per, long long seqs, long long t, int* first, long long* outside) {
  return search([=](long long i) { return (int)(i / per); }, seqs, t, first, outside);
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv_search")
    (d / "search.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dit_quantization_amd", "csrc"), "search.cpp", "-o", "libsearch.so"], cwd=d, check=True)
    L = ctypes.CDLL(str(d / "libsearch.so"))
    L.of_array.restype = L.of_line.restype = ctypes.c_longlong
    L.of_array.argtypes = [ctypes.c_void_p] + [ctypes.c_longlong] * 2 + [ctypes.c_void_p] * 2
    L.of_line.argtypes = [ctypes.c_longlong] * 3 + [ctypes.c_void_p] * 2
    return L


def call(f, *args):
    first, outside = ctypes.c_int(-7), ctypes.c_longlong()
    b = f(*args, ctypes.byref(first), ctypes.byref(outside))
    assert outside.value == 0, "read outside cu"
    return b, first.value


@pytest.mark.parametrize("seqs", [1, 2, 3, 255, 256, 257, 258, 300, 511, 512, 513, 700, 1000, 2049, 5000])
def test_matches_a_plain_search(lib, seqs):
    """Sequences of 0 to 4 rows (empty ones at the entries held, and runs of them), rows before and behind."""
    for kind in range(4):
        g = np.random.default_rng(seqs + kind)
        n = g.integers(0, 5, seqs)
        if kind == 1:
            n[g.random(seqs) < 0.8] = 0
        if kind == 2:
            n[:: -(-seqs // 256)] = 0
        if kind == 3:
            n[:] = 0
            n[seqs // 2] = 9
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32) + (3 if kind % 2 else 0)
        for t in range(int(cu[-1]) + 4):
            b = int(np.searchsorted(cu, t, side="right")) - 1
            got, first = call(lib.of_array, cu.ctypes.data, seqs, t)
            if b < 0 or b >= seqs:
                assert got == -1
            else:
                assert got == b and first == cu[b] <= t < cu[b + 1]


@pytest.mark.parametrize("seqs", [1 << 20, (1 << 31) - 300, (1 << 31) - 256, (1 << 31) - 255, (1 << 31) - 2, (1 << 31) - 1])
def test_most_sequences(lib, seqs):
    for per in (1, 2, 1000):
        last = seqs // per  # cu[seqs]
        for t in {0, 1, last // 2, last - 3, last - 2, last - 1, *range(0, last, last // 37)} - {last}:
            if not 0 <= t < last:
                continue
            got, first = call(lib.of_line, per, seqs, t)
            assert got == (t + 1) * per - 1 and first == t
        assert call(lib.of_line, per, seqs, last)[0] == -1
