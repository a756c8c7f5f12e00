"""Plain fp64 numpy forms of the 8-bit layers and of the paged 8-bit cache
(definitions: include/fp8.h, include/kvcache.h), for the parity tests."""
import numpy as np


def _table():
    """Values of the E4M3 codes 0x00..0x7E, from their definition."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


E4M3 = _table()


def e4m3_values(b):
    """Values of E4M3 bytes (no NaN)."""
    b = np.asarray(b, dtype=np.uint8)
    return np.where(b & 128, -1.0, 1.0) * E4M3[b & 127]


def nearest_e4m3(v):
    """The E4M3 values nearest to v (fp64), ties to the even code, at most 448."""
    a = np.minimum(np.abs(v), 448.0)
    hi = np.minimum(np.searchsorted(E4M3, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(E4M3[hi] == a, hi, code)
    return np.copysign(E4M3[code], v)


def encode(v, e4m3):
    """(code values, scale fp32) of the values v (fp64, last axis) that share a scale."""
    top = np.abs(v).max(-1, initial=0.0)
    s = (top / (448.0 if e4m3 else 127.0)).astype(np.float32)
    s = np.where(s == 0, np.float32(1), s)
    q = v / s.astype(np.float64)[..., None]
    return (nearest_e4m3(q) if e4m3 else np.clip(np.rint(q), -127, 127)), s


def quantize_blocks(w):
    """(code values [N, K], scales [ceil(N/128), ceil(K/128)]) of a weight."""
    w = np.asarray(w, dtype=np.float64)
    N, K = w.shape
    codes, scales = np.zeros((N, K)), np.zeros((-(-N // 128), -(-K // 128)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = np.s_[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            q, s = encode(w[part].reshape(-1), True)
            codes[part], scales[i, j] = q.reshape(w[part].shape), s
    return codes, scales


def silu_product(x, gate):
    x = np.asarray(x, dtype=np.float64)
    if gate is None:
        return x
    g = np.asarray(gate, dtype=np.float64)
    with np.errstate(over="ignore"):
        return x * (g / (1 + np.exp(-g)))


def quantize_groups(y, group, e4m3):
    """(code values [M, K], scales [M, ceil(K / group)])."""
    M, K = y.shape
    codes, scales = np.zeros((M, K)), np.zeros((M, -(-K // group)), np.float32)
    for j in range(scales.shape[1]):
        part = np.s_[:, group * j:group * (j + 1)]
        codes[part], scales[:, j] = encode(y[part], e4m3)
    return codes, scales


def slots(page_table, cu, starts, page_size, pages, tokens):
    """For each row its slot in the cache (page * page_size + row), -1 where its
    position has no page, -2 where it belongs to no sequence."""
    out = np.full(tokens, -2, dtype=np.int64)
    for b in range(len(cu) - 1):
        for t in range(max(cu[b], 0), min(cu[b + 1], tokens)):
            at = int(t) - int(cu[b]) + (0 if starts is None else int(starts[b]))
            out[t] = -1
            if 0 <= at < page_table.shape[1] * page_size:
                page = int(page_table[b, at // page_size])
                if 0 <= page < pages:
                    out[t] = page * page_size + at % page_size
    return out
