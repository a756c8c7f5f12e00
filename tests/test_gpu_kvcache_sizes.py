"""Parity of the paged 8-bit cache (include/kvcache.h) where test_gpu_kvcache.py
does not go: more than 256 sequences, the kernels of large calls for every width
of heads and both types, calls of more than one launch."""
import numpy as np
import pytest
import torch

from dit_quantization_amd import kvcache
from tests import eight_bit_reference as ref
from tests.test_gpu_kvcache import BF, DEV, E4, FL, I8, batch, fresh, i32, rows, values

pytestmark = pytest.mark.gpu


def check(lengths, starts, size, H, dims, dtype, code, seed, first=0, behind=0, kind="plain"):
    """Writes rows into a cache of random contents and reads them back, each against the plain form."""
    table, cu, starts, pages, T = batch(lengths, starts, size, 3, seed, first, behind)
    cache = fresh(pages, size, H, dims, code, seed)
    want = [(values(cache[2 * i]).reshape(-1, H, d).copy(), cache[2 * i + 1].cpu().numpy().reshape(-1, H).copy()) for i, d in enumerate(dims)]
    slots = ref.slots(table, cu, starts, size, pages, T)
    live = slots >= 0
    assert live.sum() == sum(lengths)
    new = [rows(T, H, d, seed + 1 + i, kind, dtype) for i, d in enumerate(dims)]
    at = (i32(table), i32(cu), i32(starts))
    kvcache.write(*new, cache, *at)
    out = tuple(torch.full((T, H, d), 7.0, dtype=dtype, device=DEV) for d in dims)
    kvcache.read(cache, *at, out=out)
    for i, d in enumerate(dims):
        q, s = ref.encode(new[i].float().cpu().numpy().astype(np.float64)[live], code == E4)
        want[i][0][slots[live]], want[i][1][slots[live]] = q, s
        assert np.array_equal(values(cache[2 * i]).reshape(-1, H, d), want[i][0])
        assert np.array_equal(cache[2 * i + 1].cpu().numpy().reshape(-1, H), want[i][1])
        back = torch.full((T, H, d), 7.0)
        back[torch.from_numpy(live)] = torch.from_numpy((q * s.astype(np.float64)[..., None]).astype(np.float32))
        assert torch.equal(out[i].cpu(), back.to(dtype))


@pytest.mark.parametrize("seqs", [255, 256, 257, 300, 513, 1000, 5000])
@pytest.mark.parametrize("code", [I8, E4])
def test_many_sequences(seqs, code):
    """Sequences of 0 to 6 rows, empty ones at every place of the table's coarse entries and in runs."""
    for kind in range(3):
        print(f"[case] {seqs} sequences {code} {kind}", flush=True)
        g = np.random.default_rng(seqs + kind)
        n, starts = g.integers(0, 7, seqs), g.integers(0, 40, seqs)
        if kind == 1:
            n[::-(-seqs // 256)] = 0
        if kind == 2:
            n[g.random(seqs) < 0.9] = 0
        check(n.tolist(), starts.tolist(), 16, 2, (32, 48), BF, code, 3, first=5 * kind, behind=kind)


# at least 2^20 vectors: 4, 8, 16, 32 and 64 lanes a row, keys and values of different widths, numbers of heads that
# leave a workgroup's last round short
@pytest.mark.parametrize("H,dims,T", [(7, (64, 48), 37500), (5, (80, 128), 26301), (3, (192, 256), 22001), (2, (512, 272), 16501),
                                      (1, (1024, 16), 16501), (5, (16, 80), 27001)])
@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("code", [I8, E4])
def test_large_calls(H, dims, T, dtype, code):
    print(f"[case] {T} rows of {H} x {dims} {dtype} {code}", flush=True)
    lanes = next(n for n in (4, 8, 16, 32, 64) if max(dims) <= 16 * n)
    assert T * H * lanes >= 1 << 20 and T * H * max(dims) // 16 >= (1 << 20 if max(dims) != 80 else 0)
    g = np.random.default_rng(T)
    cut = np.sort(g.integers(0, T - 4, 299))
    lengths = np.diff(np.concatenate([[0], cut, [T - 4]]))
    check(lengths.tolist(), g.integers(0, 60, 300).tolist(), 32, H, dims, dtype, code, 5, first=1, behind=3)


def test_write_of_two_launches():
    """4 million tokens with a workgroup each: those behind the first launch's 2^22."""
    T, H, D, size = (1 << 22) + 100, 129, 16, 16
    base = torch.randn(8 * T + 16 * H, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF)
    k = base.as_strided((T, H, D), (8, 16, 1))          # every token has values of its own
    v = k[:1].expand(T, H, D)
    near = slice((1 << 22) - 50, T)
    cache, want = kvcache.new(10, size, H, D), kvcache.new(10, size, H, D)
    table = i32(np.random.default_rng(2).permutation(10)[None])
    kvcache.write(k, v, cache, table, i32([0, T]), i32([-near.start]))
    kvcache.write(k[near], v[near], want, table, i32([0, 150]))
    for a, b in zip(cache, want):
        assert torch.equal(a, b) and bool(a.any())


def test_read_of_two_launches():
    T, H, dims, size = (1 << 22) + 100, 9, (1024, 16), 16
    near = slice((1 << 22) - 50, T)
    for code in (I8, E4):
        cache = fresh(10, size, H, dims, code, 3)
        table = i32(np.random.default_rng(4).permutation(10)[None])
        out = tuple(torch.empty(T, H, d, dtype=BF, device=DEV) for d in dims)
        for o in out:
            o[near.start - 100:] = 7.0
        kvcache.read(cache, table, i32([near.start, T]), out=out)
        want = kvcache.read(cache, table, i32([0, 150]), tokens=150)
        for o, w in zip(out, want):
            assert torch.equal(o[near], w) and bool((o[near.start - 100:near.start] == 7.0).all())
        del out
