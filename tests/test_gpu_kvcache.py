"""GPU parity of the paged 8-bit cache (include/kvcache.h) with the plain fp64
forms of tests/eight_bit_reference.py: codes, scales and values bit for bit,
places that no row has left as they were, and a decoder layer in 8 bits that
uses the cache with the 8-bit layers."""
import numpy as np
import pytest
import torch

from dit_quantization_amd import fp8, int4, kvcache
from dit_quantization_amd import nvfp4 as nv
from tests import eight_bit_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, FL, E4, I8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


def values(codes):
    return codes.cpu().numpy().astype(np.float64) if codes.dtype == I8 else ref.e4m3_values(codes.view(torch.uint8).cpu().numpy())


def fresh(pages, size, heads, dims, dtype, seed=0):
    """A cache of random contents (no NaN codes)."""
    g = np.random.default_rng(seed)
    out = []
    for d in dims:
        b = g.integers(0, 127, (pages, size, heads, d)).astype(np.uint8) | (g.integers(0, 2, (pages, size, heads, d)) << 7).astype(np.uint8)
        out += [torch.from_numpy(b).to(DEV).view(dtype),
                torch.from_numpy(g.uniform(0.5, 2, (pages, size, heads)).astype(np.float32)).to(DEV)]
    return tuple(out)


def rows(T, H, D, seed, kind, dtype):
    g = np.random.default_rng(seed)
    x = g.standard_normal((T, H, D)).astype(np.float32)
    x[..., g.random(D) < 0.03] *= 20
    if kind == "edges":
        for t in range(T):
            if t % 6 == 1:
                x[t] = 0
            if t % 6 == 2:
                x[t] *= np.float32(1e-40)
            if t % 6 == 3:
                x[t] *= np.float32(1e36)       # at most 20 * 5 * 1e36
            if t % 6 == 4:
                x[t] = g.integers(-254, 255, (H, D)) / 2        # ties of INT8
                x[t, :, 0] = 127.0
            if t % 6 == 5:
                x[t] = g.integers(-448 * 4, 448 * 4 + 1, (H, D)) / 32     # and, scaled by 1, of E4M3
                x[t, :, D - 1] = -448.0
    return torch.from_numpy(x).to(DEV).to(dtype)


def batch(lengths, starts, size, spare, seed, first=0, behind=0):
    """(page table, cu, starts, pages, tokens) of sequences on shuffled pages."""
    g = np.random.default_rng(seed)
    need = [-(-(s + n) // size) for s, n in zip(starts, lengths)]
    pages = sum(need) + spare
    order = g.permutation(pages)
    table = np.full((len(lengths), max(max(need, default=0), 1)), -1, dtype=np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = first + np.concatenate([[0], np.cumsum(lengths)])
    return table, cu, np.asarray(starts), pages, int(cu[-1]) + behind


BATCHES = {
    "one": ([1], [0], 16),
    "decode": ([1] * 70, [(7 * i) % 33 for i in range(70)], 16),
    "uneven": ([5, 1, 0, 17, 33, 0, 2], [0, 15, 3, 31, 1, 0, 16], 16),
    "pages_of_one": ([3, 4], [2, 0], 1),
    "odd_pages": ([20, 3, 9], [6, 0, 13], 7),
    "empty_ends": ([0, 0, 6, 0, 0], [0, 1, 2, 3, 4], 32),
}


def check_write(name, H, dims, dtype, code, kind, first=0, behind=0, use_starts=True):
    lengths, starts, size = BATCHES[name]
    if not use_starts:
        starts = [0] * len(lengths)
    table, cu, starts, pages, T = batch(lengths, starts, size, 3, 1, first, behind)
    cache = fresh(pages, size, H, dims, code)
    before = [t.clone() for t in cache]
    new = [rows(T, H, d, 2 + i, kind, dtype) for i, d in enumerate(dims)]
    kvcache.write(new[0], new[1], cache, i32(table), i32(cu), i32(starts) if use_starts else None)
    slots = ref.slots(table, cu, starts, size, pages, T)
    live = slots >= 0
    assert live.sum() == sum(lengths)
    for i in range(2):
        q, s = ref.encode(new[i].float().cpu().numpy().astype(np.float64)[live], code == E4)
        want_q, want_s = values(before[2 * i]).reshape(-1, H, dims[i]), before[2 * i + 1].cpu().numpy().reshape(-1, H)
        want_q[slots[live]], want_s[slots[live]] = q, s
        assert np.array_equal(values(cache[2 * i]).reshape(want_q.shape), want_q)
        assert np.array_equal(cache[2 * i + 1].cpu().numpy().reshape(want_s.shape), want_s)


def check_read(name, H, dims, dtype, code, first=0, behind=0, use_starts=True):
    lengths, starts, size = BATCHES[name]
    if not use_starts:
        starts = [0] * len(lengths)
    table, cu, starts, pages, T = batch(lengths, starts, size, 3, 3, first, behind)
    cache = fresh(pages, size, H, dims, code, 5)
    out = tuple(torch.full((T, H, d), 7.0, dtype=dtype, device=DEV) for d in dims)
    got = kvcache.read(cache, i32(table), i32(cu), i32(starts) if use_starts else None, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    slots = ref.slots(table, cu, starts, size, pages, T)
    live = slots >= 0
    for i in range(2):
        q, s = values(cache[2 * i]).reshape(-1, H, dims[i]), cache[2 * i + 1].cpu().numpy().reshape(-1, H)
        want = torch.full((T, H, dims[i]), 7.0)
        want[torch.from_numpy(live)] = torch.from_numpy((q[slots[live]] * s[slots[live]].astype(np.float64)[..., None]).astype(np.float32))
        assert torch.equal(out[i].cpu(), want.to(dtype))


@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("dtype", [BF, FL])
@pytest.mark.parametrize("code", [I8, E4])
def test_write_and_read(name, dtype, code):
    print(f"[case] {name} {dtype} {code}", flush=True)
    check_write(name, 2, (64, 64), dtype, code, "edges")
    check_read(name, 2, (64, 64), dtype, code)
    check_write(name, 3, (32, 16), dtype, code, "plain", first=2, behind=3)
    check_read(name, 3, (32, 16), dtype, code, first=2, behind=3)
    check_write(name, 1, (48, 48), dtype, code, "edges", use_starts=False)
    check_read(name, 1, (48, 48), dtype, code, use_starts=False)


@pytest.mark.parametrize("H,dims", [(1, (16, 16)), (8, (128, 128)), (5, (80, 80)), (4, (96, 64)), (2, (192, 128)), (32, (128, 128)),
                                    (3, (256, 256)), (1, (576, 512)), (2, (272, 528)), (1, (1024, 16)), (7, (112, 240))])
@pytest.mark.parametrize("code", [I8, E4])
def test_head_layouts(H, dims, code):
    print(f"[case] heads {H} {dims} {code}", flush=True)
    for dtype in (BF, FL):
        check_write("uneven", H, dims, dtype, code, "edges", behind=1)
        check_read("uneven", H, dims, dtype, code, behind=1)


@pytest.mark.parametrize("code", [I8, E4])
def test_strides(code):
    """Rows that are slices of a fused projection, heads before tokens, and a
    cache whose keys and values share pages of one allocation."""
    H, D, size = 4, 64, 16
    table, cu, starts, pages, T = batch([5, 30, 1], [3, 0, 40], size, 2, 7)
    fused = rows(T, 3 * H, D, 8, "plain", BF)
    k, v = fused[:, H:2 * H], fused[:, 2 * H:]
    both = torch.zeros(pages, 2, size, H, D, dtype=torch.uint8, device=DEV).view(code)
    both_s = torch.zeros(pages, 2, size, H, device=DEV)
    cache = (both[:, 0], both_s[:, 0], both[:, 1], both_s[:, 1])
    plain = kvcache.new(pages, size, H, D, dtype=code)
    args = (i32(table), i32(cu), i32(starts))
    kvcache.write(k, v, cache, *args)
    kvcache.write(k.contiguous(), v.transpose(0, 1).contiguous().transpose(0, 1), plain, *args)
    for a, b in zip(cache, plain):
        assert torch.equal(a.contiguous().view(torch.uint8), b.view(torch.uint8))
    want = kvcache.read(plain, *args, tokens=T)
    out = torch.full((T, 2 * H, D), 9.0, dtype=BF, device=DEV)
    heads_first = torch.empty(H, T, D, dtype=BF, device=DEV).transpose(0, 1)
    kvcache.read(cache, *args, out=(out[:, H:], heads_first))
    assert torch.equal(out[:, H:], want[0]) and torch.equal(heads_first, want[1])
    assert bool((out[:, :H] == 9.0).all())
    # one token's keys for all of them
    kvcache.write(k[:1].expand(T, H, D), v, plain, *args)
    assert bool((kvcache.read(plain, *args, tokens=T)[0] == kvcache.read(plain, *args, tokens=1)[0]).all())


def test_round_trip_is_within_half_a_step():
    """A value comes back within half a step of its code: INT8 half a scale,
    E4M3 2^-4 of the value (2^-10 of a scale below its normal range), then bf16's half step."""
    table, cu, starts, pages, T = batch([50, 77], [0, 9], 16, 1, 9)
    k, v = rows(T, 4, 128, 10, "plain", FL), rows(T, 4, 128, 11, "plain", FL)
    for code in (I8, E4):
        cache = kvcache.new(pages, 16, 4, 128, dtype=code)
        kvcache.write(k, v, cache, i32(table), i32(cu), i32(starts))
        for dtype in (FL, BF):
            for new, got in zip((k, v), kvcache.read(cache, i32(table), i32(cu), i32(starts), tokens=T, out_dtype=dtype)):
                s = new.double().abs().amax(2, keepdim=True) / (127 if code == I8 else 448)
                step = s / 2 if code == I8 else torch.maximum(new.double().abs() * 2.0 ** -4, s * 2.0 ** -10)
                tol = step * (1 + 2.0 ** -22) + new.double().abs() * 2.0 ** -22
                if dtype == BF:
                    tol = tol + 2.0 ** -8 * (new.double().abs() + tol)
                assert bool(((got.double() - new.double()).abs() <= tol).all())


def test_places_outside_the_cache():
    """Page numbers that are no page, positions before 0 and past the table:
    nothing is written for them, and they read as zeros."""
    H, D, size, pages = 2, 32, 4, 6
    table = np.array([[5, -1, 2], [6, 0, 1 << 30], [-(1 << 31), 3, (1 << 31) - 1]])
    cu, starts = np.array([0, 14, 26, 40]), np.array([-3, 2, 0])
    T = 42
    for code in (I8, E4):
        cache = fresh(pages, size, H, (D, D), code, 3)
        before = [t.clone() for t in cache]
        k, v = rows(T, H, D, 1, "plain", BF), rows(T, H, D, 2, "plain", BF)
        kvcache.write(k, v, cache, i32(table), i32(cu), i32(starts))
        slots = ref.slots(table, cu, starts, size, pages, T)
        live = slots >= 0
        assert 0 < live.sum() < 20 and (slots == -1).sum() > 20
        for i, new in enumerate((k, v)):
            q, s = ref.encode(new.float().cpu().numpy().astype(np.float64)[live], code == E4)
            want_q, want_s = values(before[2 * i]).reshape(-1, H, D), before[2 * i + 1].cpu().numpy().reshape(-1, H)
            want_q[slots[live]], want_s[slots[live]] = q, s
            assert np.array_equal(values(cache[2 * i]).reshape(want_q.shape), want_q)
            assert np.array_equal(cache[2 * i + 1].cpu().numpy().reshape(want_s.shape), want_s)
        out = tuple(torch.full((T, H, D), 7.0, device=DEV) for _ in range(2))
        kvcache.read(cache, i32(table), i32(cu), i32(starts), out=out)
        for o in out:
            assert bool((o[torch.from_numpy(slots == -1).to(DEV)] == 0).all())
            assert bool((o[torch.from_numpy(slots == -2).to(DEV)] == 7.0).all())
            assert not bool((o[torch.from_numpy(live).to(DEV)] == 0).all(2).any())


def test_two_rows_of_one_place_leave_the_others():
    """Two sequences that share a page: the places they both write are unspecified, all others hold what they should."""
    H, D, size, pages = 2, 32, 4, 3
    table, cu = np.array([[2, 0], [2, 1]]), np.array([0, 8, 16])
    cache = kvcache.new(pages, size, H, D)
    k = rows(16, H, D, 1, "plain", BF)
    kvcache.write(k, k, cache, i32(table), i32(cu))
    got = kvcache.read(cache, i32(table), i32(cu), tokens=16, out_dtype=FL)[0]
    alone = kvcache.new(4, size, H, D)
    kvcache.write(k, k, alone, i32([[0, 1], [2, 3]]), i32(cu))
    want = kvcache.read(alone, i32([[0, 1], [2, 3]]), i32(cu), tokens=16, out_dtype=FL)[0]
    for part in (slice(4, 8), slice(12, 16)):
        assert torch.equal(got[part], want[part])


def test_offsets_past_32_bits():
    """A cache of 5.4 GB of codes a tensor; its last pages."""
    H, D, size, pages = 8, 128, 64, 82000
    codes = torch.zeros(pages, size, H, D, dtype=torch.uint8, device=DEV).view(I8)
    s = torch.zeros(pages, size, H, device=DEV)
    cache = (codes, s, codes.clone(), s.clone())
    table, cu, starts = np.array([[pages - 1, 0, pages - 2]]), np.array([0, 150]), np.array([20])
    k, v = rows(150, H, D, 1, "plain", BF), rows(150, H, D, 2, "plain", BF)
    kvcache.write(k, v, cache, i32(table), i32(cu), i32(starts))
    q, sc = ref.encode(k.float().cpu().numpy().astype(np.float64), False)
    assert np.array_equal(values(cache[0][pages - 1]).reshape(size, H, D)[20:], q[:44])
    assert np.array_equal(cache[1][pages - 1, 20:].cpu().numpy(), sc[:44])
    got = kvcache.read(cache, i32(table), i32(cu), i32(starts), tokens=150, out_dtype=FL)
    small = kvcache.new(3, size, H, D)
    kvcache.write(k, v, small, i32([[0, 1, 2]]), i32(cu), i32(starts))
    want = kvcache.read(small, i32([[0, 1, 2]]), i32(cu), i32(starts), tokens=150, out_dtype=FL)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_many_rows():
    """More rows than one pass of the grid takes, and rows of 2.4 GB."""
    H, D, size, T = 16, 128, 128, 300000
    pages = -(-T // size)
    for code in (I8, E4):
        cache = kvcache.new(pages, size, H, D, dtype=code)
        table = torch.randperm(pages, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.int32)[None]
        k = torch.randn(1000, H, D, device=DEV).to(BF).repeat(300, 1, 1)
        kvcache.write(k, k, cache, table, i32([0, T]))
        got = kvcache.read(cache, table, i32([0, T]), tokens=T)
        assert torch.equal(got[0], got[1])
        assert torch.equal(got[0].view(300, 1000, H, D), got[0][:1000].expand(300, 1000, H, D))
        q, s = ref.encode(k[:50].float().cpu().numpy().astype(np.float64), code == E4)
        want = torch.from_numpy((q * s.astype(np.float64)[..., None]).astype(np.float32)).to(BF)
        assert torch.equal(got[0][:50].cpu(), want)


def test_empty_calls():
    cache = kvcache.new(4, 4, 2, 32)
    e = torch.empty(0, 2, 32, device=DEV)
    kvcache.write(e, e, cache, i32(np.zeros((1, 1))), i32([0, 0]))
    assert kvcache.read(cache, i32(np.zeros((1, 1))), i32([0, 0]), tokens=0)[0].shape == (0, 2, 32)
    k = torch.ones(3, 2, 32, device=DEV)
    none = torch.zeros(0, 1, dtype=torch.int32, device=DEV)
    kvcache.write(k, k, cache, none, i32([0]))                  # no sequences
    kvcache.write(k, k, cache, torch.zeros(1, 0, dtype=torch.int32, device=DEV), i32([0, 3]))    # no pages in the table
    kvcache.write(k, k, kvcache.new(0, 4, 2, 32), i32(np.zeros((1, 1))), i32([0, 3]))            # no pages in the cache
    assert not bool(cache[0].any()) and not bool(cache[1].any())
    out = tuple(torch.full((3, 2, 32), 7.0, device=DEV) for _ in range(2))
    kvcache.read(cache, none, i32([0]), out=out)
    assert bool((out[0] == 7.0).all())
    kvcache.read(kvcache.new(0, 4, 2, 32), i32(np.zeros((1, 1))), i32([0, 2]), out=out)
    assert bool((out[0][:2] == 0).all()) and bool((out[0][2] == 7.0).all())


def test_capture_is_refused():
    cache = fresh(4, 4, 2, (32, 32), I8)
    before = [t.clone() for t in cache]
    k = torch.ones(3, 2, 32, device=DEV)
    table, cu = i32([[0, 1]]), i32([0, 3])
    out = (torch.full_like(k, 5.0), torch.full_like(k, 5.0))
    mark = torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mark.add_(1.0)
        for call in (lambda: kvcache.write(k, k, cache, table, cu), lambda: kvcache.read(cache, table, cu, out=out)):
            with pytest.raises(nv.NVFP4Error) as e:
                call()
            assert e.value.status == nv.ERR_CAPTURE
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(cache, before)) and bool((out[0] == 5.0).all())


def test_side_stream():
    table, cu, starts, pages, T = batch([40, 9], [0, 5], 16, 1, 9)
    k = rows(T, 4, 64, 10, "plain", BF)
    args = (i32(table), i32(cu), i32(starts))
    one, two = kvcache.new(pages, 16, 4, 64), kvcache.new(pages, 16, 4, 64)
    kvcache.write(k, k, one, *args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        kvcache.write(k, k, two, *args)
        got = kvcache.read(two, *args, tokens=T)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    assert torch.equal(got[0], kvcache.read(one, *args, tokens=T)[0])


# ---- a decoder layer in 8 bits

def attend(q, k, v, cu_q, cu_k):
    """Causal attention of packed sequences, queries at their sequences' ends (fp32, plain torch)."""
    out = torch.empty_like(q)
    rep = q.shape[1] // k.shape[1]
    for b in range(len(cu_q) - 1):
        Q = q[cu_q[b]:cu_q[b + 1]].float()
        K, V = (t[cu_k[b]:cu_k[b + 1]].float().repeat_interleave(rep, 1) for t in (k, v))
        n, m = Q.shape[0], K.shape[0]
        w = (Q[:, None] * K[None]).sum(3) / Q.shape[2] ** 0.5                     # [n, m, heads]
        ahead = torch.arange(m, device=DEV)[None] > torch.arange(m - n, m, device=DEV)[:, None]
        w = w.masked_fill(ahead[..., None], float("-inf")).softmax(1)
        out[cu_q[b]:cu_q[b + 1]] = (w[..., None] * V[None]).sum(1).to(out.dtype)
    return out


class Layer:
    """Norm, q/k/v, cache, attention, output projection, norm, gated MLP."""
    D, H, HK, E, F = 512, 8, 2, 64, 1040

    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def w(n, k):
            return torch.randn(n, k, generator=g, device=DEV) * k ** -0.5

        self.w = {"qkv": w((self.H + 2 * self.HK) * self.E, self.D), "o": w(self.D, self.H * self.E),
                  "gate_up": w(2 * self.F, self.D), "down": w(self.D, self.F)}
        self.q = {n: fp8.quantize(t) for n, t in self.w.items()}
        self.gain = torch.ones(2, self.D, device=DEV, dtype=BF)

    def step(self, h, cache, table, cu, starts, total):
        """h [T, D] bf16: the tokens at positions starts[b].. of their sequences, which then hold cu_all."""
        nq = self.H * self.E
        xq, xs, _ = int4.rmsnorm_quant8(h, self.gain[0], group_size=128, out_dtype=E4)
        qkv = fp8.gemm(xq, xs, *self.q["qkv"]).view(h.shape[0], -1, self.E)
        q, k, v = qkv[:, :self.H], qkv[:, self.H:self.H + self.HK], qkv[:, self.H + self.HK:]
        kvcache.write(k, v, cache, table, cu, starts)
        held = starts + cu[1:] - cu[:-1]
        cu_all = torch.cat([cu[:1], torch.cumsum(held, 0).to(torch.int32)])
        K, V = kvcache.read(cache, table, cu_all, tokens=total)
        a = attend(q, K, V, cu.tolist(), cu_all.tolist()).reshape(-1, nq)
        o = fp8.gemm(*fp8.quantize_act(a), *self.q["o"])
        xq, xs, h = int4.rmsnorm_quant8(o, self.gain[1], residual=h, group_size=128, out_dtype=E4)
        gu = fp8.gemm(xq, xs, *self.q["gate_up"])
        return h + fp8.gemm(*fp8.quantize_act(gu[:, self.F:], gate=gu[:, :self.F]), *self.q["down"])

    def plain(self, h, lengths):
        """The same layer of whole sequences in fp32, unquantized."""
        h = h.float()
        nq, nk = self.H * self.E, self.HK * self.E

        def norm(x):
            return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)

        qkv = norm(h) @ self.w["qkv"].t().contiguous()
        q, k, v = (t.reshape(h.shape[0], -1, self.E) for t in (qkv[:, :nq], qkv[:, nq:nq + nk], qkv[:, nq + nk:]))
        cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
        h = h + attend(q, k, v, cu, cu).reshape(-1, nq) @ self.w["o"].t().contiguous()
        gu = norm(h) @ self.w["gate_up"].t().contiguous()
        return h + (torch.nn.functional.silu(gu[:, :self.F]) * gu[:, self.F:]) @ self.w["down"].t().contiguous()


@pytest.mark.parametrize("code", [I8, E4])
def test_decoder_layer(code):
    """A prefill of three prompts, then two decode steps, against the whole
    sequences at once through the same calls and against the layer in fp32.

    E4M3 rounds a weight and an activation by at most 2^-4 each, so a product's
    error is at most about 2^-3 of sum |x||w|; errors of random sign add up to
    about (2^-4 / sqrt 3) sqrt 2 = 5 % of the product's own size, and the three
    products behind one another that a branch has to under 20 % of the branch."""
    layer, size, lengths, new = Layer(3), 16, [37, 5, 20], 2
    seqs = len(lengths)
    all_len = [n + new for n in lengths]
    h = torch.randn(sum(all_len), layer.D, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).to(BF)
    table, cu_all, _, pages, T = batch(all_len, [0] * seqs, size, 2, 5)
    table = i32(table)
    at = [np.arange(cu_all[b], cu_all[b + 1]) for b in range(seqs)]

    def run(cache, first, count):
        rows_ = torch.from_numpy(np.concatenate([at[b][first[b]:first[b] + count[b]] for b in range(seqs)])).to(DEV)
        cu = i32(np.concatenate([[0], np.cumsum(count)]))
        total = sum(first) + sum(count)
        return rows_, layer.step(h[rows_].contiguous(), cache, table, cu, i32(first), total)

    whole_cache = kvcache.new(pages, size, layer.HK, layer.E, dtype=code)
    _, whole = run(whole_cache, [0] * seqs, all_len)
    cache = kvcache.new(pages, size, layer.HK, layer.E, dtype=code)
    got = torch.empty_like(whole)
    rows_, y = run(cache, [0] * seqs, lengths)
    got[rows_] = y
    for i in range(new):
        rows_, y = run(cache, [n + i for n in lengths], [1] * seqs)
        got[rows_] = y
    want = layer.plain(h, all_len)
    # the branches' size: what the layer adds to its input
    size_of = (want - h.float()).square().mean().sqrt()
    assert float((whole.float() - want).square().mean().sqrt() / size_of) < 0.2
    assert float((got.float() - want).square().mean().sqrt() / size_of) < 0.2
    # steps and the whole batch differ by bf16's rounding of the products' outputs and codes that it moves
    assert float((got.float() - whole.float()).square().mean().sqrt() / size_of) < 0.05
