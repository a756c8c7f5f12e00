"""Plain fp64 numpy forms of the group-scaled 4-bit weight path and of the
8-bit RMS norm (definitions: include/int4.h), for the parity tests."""
import numpy as np


def bf16(x):
    """fp32 values rounded to bf16 (nearest, ties to even), as fp32."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def slices(cols, group):
    step = group or max(cols, 1)
    return [slice(c, min(c + step, cols)) for c in range(0, cols, step)]


def quantize(w, group, symmetric):
    """(codes [N, K] 0..15, scales [N, G] fp32 holding bf16, zeros [N, G])."""
    w = np.asarray(w, dtype=np.float32).astype(np.float64)
    N, K = w.shape
    parts = slices(K, group)
    codes, scales, zeros = np.zeros((N, K), np.uint8), np.zeros((N, len(parts)), np.float32), np.zeros((N, len(parts)),
                                                                                                     np.uint8)
    for g, p in enumerate(parts):
        t = w[:, p]
        lo, hi = np.minimum(t.min(1), 0), np.maximum(t.max(1), 0)
        s = bf16(((np.maximum(hi, -lo) / 7) if symmetric else ((hi - lo) / 15)).astype(np.float32))
        d = s.astype(np.float64)
        live = d != 0
        safe = np.where(live, d, 1)
        z = np.full(N, 8.0) if symmetric else np.where(live, np.clip(np.rint(-lo / safe), 0, 15), 0)
        q = np.where(live[:, None], np.rint(t / safe[:, None]), 0)
        codes[:, p] = np.clip(q + z[:, None], 0, 15)
        scales[:, g], zeros[:, g] = s, z
    return codes, scales, zeros


def pack(codes):
    """[N, K] codes to bytes: byte 4 d + b = element 8 d + b | element 8 d + 4 + b << 4."""
    c = np.asarray(codes, dtype=np.uint8).reshape(codes.shape[0], -1, 2, 4)
    return np.ascontiguousarray((c[:, :, 0] | (c[:, :, 1] << 4)).reshape(codes.shape[0], -1))


def unpack(packed):
    b = np.asarray(packed, dtype=np.uint8).reshape(packed.shape[0], -1, 1, 4)
    return np.concatenate([b & 15, b >> 4], 2).reshape(packed.shape[0], -1)


def per_element(v, cols, group):
    """[N, G] values spread over the columns of their groups."""
    return np.repeat(np.asarray(v, dtype=np.float64), group, axis=1)[:, :cols]


def dequant(codes, scales, zeros, group):
    K = codes.shape[1]
    return per_element(scales, K, group) * (codes.astype(np.float64) - per_element(zeros, K, group))


def product(x, codes, scales, zeros, group):
    """(y, a): x W^T in fp64 and sum_k |x| s (code + zero), what the products'
    fp32 sums are made of (they add x code and take zero sum x off)."""
    K = codes.shape[1]
    s, z = per_element(scales, K, group), per_element(zeros, K, group)
    x = np.asarray(x, dtype=np.float64)
    return x @ (s * (codes.astype(np.float64) - z)).T, np.abs(x) @ (s * (codes + z)).T


def product_bound(a, K):
    """Any-order bound of the products' fp32 sums: a term meets at most 128
    additions inside its group, K / 32 between groups and 32 more for the scale
    factors, the lanes and the waves, each off by at most 2^-24 of a sum no
    larger than a."""
    return (160 + K / 32) * 2.0 ** -24 * a


def e4m3_bytes_to_f64(b):
    b = np.asarray(b, dtype=np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (np.maximum(e, 1) - 10.0), m * 2.0 ** -9)
    return np.where(b & 0x80, -v, v)


def to_e4m3(v):
    """fp64 to the nearest E4M3 value, ties to even, saturating at 448."""
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(v / step) * step, -448, 448)


def rmsnorm_quant8(x, weight, residual, res_bf16, eps, group, e4m3):
    """(codes as fp64 values, scales fp32, h fp32 or None) from fp32 inputs
    (holding bf16 values where the tensors are bf16)."""
    h = np.asarray(x, dtype=np.float32)
    if residual is not None:
        h = (h + np.asarray(residual, dtype=np.float32)).astype(np.float32)
        h = bf16(h) if res_bf16 else h
    d = h.astype(np.float64)
    R, C = d.shape
    t = d * (1.0 if weight is None else np.asarray(weight, dtype=np.float32).astype(np.float64))
    with np.errstate(divide="ignore", invalid="ignore"):
        inv = 1.0 / np.sqrt((d * d).sum(1) / max(C, 1) + eps)
    parts = slices(C, group)
    codes, scales = np.zeros((R, C)), np.ones((R, len(parts)), np.float32)
    for g, p in enumerate(parts):
        m = np.abs(t[:, p]).max(1)
        live = m > 0
        with np.errstate(invalid="ignore"):
            s = np.where(live, m * np.where(live, inv, 0) / (448.0 if e4m3 else 127.0), 0).astype(np.float32)
        s = np.where(s == 0, np.float32(1), s)
        v = t[:, p] * (np.where(live, inv, 0) / s.astype(np.float64))[:, None]
        codes[:, p] = to_e4m3(v) if e4m3 else np.clip(np.rint(v), -127, 127)
        scales[:, g] = s
    return codes, scales, None if residual is None else h
