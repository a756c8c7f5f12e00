"""Workloads of the group-scaled 4-bit weight path: RMS norm with an 8-bit
output, the weight quantizer and its inverse, and the decode products with
16-bit and 8-bit activations (dit_quantization_amd.int4).

`run` makes one call of an operator: in plain torch operations where `own` is
False, through the library where it is True.  `exact` evaluates the operator's
definition in 64 bits.

Format of a weight [N, K]: codes uint8 [N, K/2]; byte 4 d + b of a row holds
element 8 d + b in its low nibble and element 8 d + 4 + b in its high nibble;
one bf16 scale and, unless symmetric, one uint8 zero point for every group of
32, 64 or 128 elements of a row (the last group may be short); the weight is
scale * (code - zero), with zero = 8 throughout where it is symmetric.
The definitions fix every code and zero point, so these are compared as they
are stored; E4M3 codes are values of their type.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_TOP = {"int8": 127.0, "e4m3": 448.0}


def listed():
    return [
        # One token of an 8B model: the residual's addition and the norm before q/k/v, one scale for the row.
        {"name": "norm_decode_1x4096", "op": "norm", "rows": 1, "cols": 4096, "x": "bf16", "residual": "bf16", "out": "int8", "group": 0},
        # A prefill of 4096 tokens, scales for 128 columns each (block-scaled FP8 products).
        {"name": "norm_prefill_4096x4096", "op": "norm", "rows": 4096, "cols": 4096, "x": "bf16", "residual": "bf16", "out": "e4m3", "group": 128},
        # Query and key heads of an image token stream: many short rows, no residual.
        {"name": "norm_heads_110593x128", "op": "norm", "rows": 110593, "cols": 128, "x": "bf16", "residual": "", "out": "int8", "group": 0},
        # A ragged batch on a 32-bit residual stream at the MLP's width.
        {"name": "norm_f32_517x14336", "op": "norm", "rows": 517, "cols": 14336, "x": "bf16", "residual": "f32", "out": "e4m3", "group": 0},
        # Converting a checkpoint: the gate weight from 32 bits, with zero points.
        {"name": "quantize_14336x4096_g128", "op": "quantize", "N": 14336, "K": 4096, "x": "f32", "group": 128, "symmetric": False},
        # A key projection from bf16, symmetric, the finest groups.
        {"name": "quantize_1024x4096_g32", "op": "quantize", "N": 1024, "K": 4096, "x": "bf16", "group": 32, "symmetric": True},
        # Unpacking the down weight to bf16 for a long prompt's library product.
        {"name": "dequant_4096x14336_g128", "op": "dequant", "N": 4096, "K": 14336, "group": 128, "symmetric": False, "out": "bf16"},
        # A key projection whose rows end inside a group, to 32 bits.
        {"name": "dequant_1000x4128_g64", "op": "dequant", "N": 1000, "K": 4128, "group": 64, "symmetric": True, "out": "f32"},
        # Decoding one token through the gate weight, 16-bit activations.
        {"name": "w4a16_m1_14336x4096", "op": "w4a16", "M": 1, "N": 14336, "K": 4096, "group": 128, "symmetric": False, "out": "bf16"},
        # Five sequences through the down weight.
        {"name": "w4a16_m5_4096x14336", "op": "w4a16", "M": 5, "N": 4096, "K": 14336, "group": 64, "symmetric": True, "out": "bf16"},
        # One token through a key projection, INT8 activations with one scale: latency.
        {"name": "w4a8_m1_1024x4096", "op": "w4a8", "M": 1, "N": 1024, "K": 4096, "x": "int8", "x_group": False, "group": 128, "symmetric": True, "out": "bf16"},
        # A full decode batch through the gate weight, FP8 activations scaled by group.
        {"name": "w4a8_m16_14336x4096", "op": "w4a8", "M": 16, "N": 14336, "K": 4096, "x": "e4m3", "x_group": True, "group": 128, "symmetric": False, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "dequant", "w4a16", "w4a8", "w4a8"])
    if op == "norm":
        cols = 16 * _log(rng, 4, 1024)
        x = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "rows": _log(rng, 1, max(2, (4096 * 4096) // cols)), "cols": cols, "x": x, "residual": rng.choice(["", x, "f32"]),
                "out": rng.choice(["int8", "e4m3"]), "group": rng.choice([0, 0, 32, 64, 128])}
    K = 32 * _log(rng, 4, 448)
    N = _log(rng, 64, min(32768, (14336 * 4096) // K))
    case = {"op": op, "N": N, "K": K, "group": rng.choice([32, 64, 128, 128]), "symmetric": rng.random() < 0.5}
    if op == "quantize":
        return {**case, "x": rng.choice(["f32", "bf16"])}
    if op == "dequant":
        return {**case, "out": rng.choice(["f32", "bf16"])}
    case = {**case, "M": rng.choice([1, 1, 2, 3, 4, 6, 7, 8, 11, 13, 16]), "out": rng.choice(["bf16", "bf16", "f32"])}
    return case if op == "w4a16" else {**case, "x": rng.choice(["int8", "e4m3"]), "x_group": rng.random() < 0.5}


def _groups(t, group, fill=0.0):
    """[R, C] as [R, G, group], the last group filled up with `fill`."""
    pad = -t.shape[1] % group
    return torch.nn.functional.pad(t, (0, pad), value=fill).reshape(t.shape[0], -1, group)


def _pack(q):
    """Codes [N, K] (whole numbers 0..15) to bytes [N, K/2]."""
    q = q.to(torch.uint8).reshape(q.shape[0], -1, 2, 4)
    return (q[:, :, 0] | (q[:, :, 1] << 4)).reshape(q.shape[0], -1)


def _unpack(codes, dtype=torch.float32):
    c = codes.reshape(codes.shape[0], -1, 1, 4)
    return torch.cat([c & 15, c >> 4], 2).reshape(codes.shape[0], -1).to(dtype)


def _plain_quantize(w, group, symmetric):
    # Codes are whole numbers next to rounding borders: quotients in 64 bits (exact enough that no border is crossed: w has 24
    # significant bits and a scale 8), scales rounded to 32 bits and then to bf16, as the definition says.
    t = _groups(w.float(), group)
    if symmetric:
        s = (t.abs().amax(2).double() / 7).float().to(torch.bfloat16)
    else:
        lo, hi = t.amin(2).clamp(max=0), t.amax(2).clamp(min=0)
        s = ((hi.double() - lo.double()) / 15).float().to(torch.bfloat16)
    d = s.double()
    safe = torch.where(d == 0, torch.ones_like(d), d)
    z = torch.full_like(d, 8.0) if symmetric else torch.where(d == 0, torch.zeros_like(d), torch.round(-lo.double() / safe).clamp(0, 15))
    q = torch.where(d[..., None] == 0, torch.zeros((), dtype=torch.float64, device=w.device), torch.round(t.double() / safe[..., None]))
    q = (q + z[..., None]).clamp(0, 15).reshape(w.shape[0], -1)[:, :w.shape[1]]
    return _pack(q), s, None if symmetric else z.to(torch.uint8)


def _plain_dequant(codes, scales, zeros, group):
    t = _groups(_unpack(codes), group)
    z = 8.0 if zeros is None else zeros.float()[..., None]
    return ((t - z) * scales.float()[..., None]).reshape(codes.shape[0], -1)[:, :codes.shape[1] * 2]


def _to_e4m3(v):
    """64-bit values, rounded once to the nearest E4M3 value (ties to even, at most 448)."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _plain_norm(x, weight, residual, eps, group, out):
    h = x.float()
    if residual is not None:
        h = (h + residual.float()).to(residual.dtype)
    # next to rounding borders: in 64 bits
    d = h.double()
    y = d * weight.double() * torch.rsqrt((d * d).mean(1, keepdim=True) + eps)
    t = _groups(y, group or y.shape[1])
    s = (t.abs().amax(2) / _TOP[out]).float()
    s = torch.where(s == 0, torch.ones_like(s), s)
    v = t / s.double()[..., None]
    v = torch.round(v).clamp(-127, 127) if out == "int8" else _to_e4m3(v)
    q = v.reshape(y.shape[0], -1)[:, :y.shape[1]].to(_TYPES[out])
    return (q, s) if residual is None else (q, s, h)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    op = case["op"]
    if op == "norm":
        # hidden states with a few loud channels, as a trained model's
        loud = torch.rand(case["cols"], generator=g, device="cuda") < 0.01
        gain = torch.where(loud, 20.0, 1.0)
        x = (normal(case["rows"], case["cols"]) * gain).to(_TYPES[case["x"]])
        r = (normal(case["rows"], case["cols"]) * 2).to(_TYPES[case["residual"]]) if case["residual"] else None
        w = (1 + 0.2 * normal(case["cols"])).to(torch.bfloat16)
        return {**case, "xt": x, "rt": r, "wt": w, "eps": 1e-6}
    N, K, group = case["N"], case["K"], case["group"]
    # weights whose rows differ in spread (each row's over the root of a mean of five squares), as trained ones do
    w = normal(N, K) * 0.02
    w *= torch.rsqrt(sum(normal(N, 1).square() for _ in range(5)) / 5)
    if op == "quantize":
        return {**case, "wt": w.to(_TYPES[case["x"]])}
    c, s, z = _plain_quantize(w, group, case["symmetric"])
    st = {**case, "c": c, "s": s, "z": z}
    if op == "dequant":
        return st
    x = normal(case["M"], K)
    if op == "w4a16":
        return {**st, "xt": x.to(torch.bfloat16)}
    t = _groups(x, group if case["x_group"] else K)
    sx = t.abs().amax(2) / _TOP[case["x"]]
    q = t / sx[..., None]
    q = torch.round(q) if case["x"] == "int8" else q
    return {**st, "xq": q.reshape(case["M"], -1)[:, :K].contiguous().to(_TYPES[case["x"]]), "sx": sx}


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    op = st["op"]
    if op == "norm":
        return _plain_norm(st["xt"], st["wt"], st["rt"], st["eps"], st["group"], st["out"])
    if op == "quantize":
        c, s, z = _plain_quantize(st["wt"], st["group"], st["symmetric"])
        return (c, s) if z is None else (c, s, z)
    w = _plain_dequant(st["c"], st["s"], st["z"], st["group"])
    if op == "dequant":
        return w.to(_TYPES[st["out"]])
    if op == "w4a16":
        x = st["xt"].float()
    else:
        x = st["xq"].float()
        x = (_groups(x, st["group"]) * st["sx"][..., None]).reshape(x.shape[0], -1)[:, :x.shape[1]] if st["x_group"] else x * st["sx"]
    return (x @ w.t()).to(_TYPES[st["out"]])


def _run_own(st):
    from dit_quantization_amd import int4
    op, out = st["op"], st.get("out")
    if op == "norm":
        q, s, h = int4.rmsnorm_quant8(st["xt"], st["wt"], residual=st["rt"], eps=st["eps"], group_size=st["group"], out_dtype=_TYPES[out])
        return (q, s) if h is None else (q, s, h)
    if op == "quantize":
        c, s, z = int4.quantize(st["wt"], group_size=st["group"], symmetric=st["symmetric"])
        return (c, s) if z is None else (c, s, z)
    w = (st["c"], st["s"], st["z"])
    if op == "dequant":
        return int4.dequant(*w, group_size=st["group"], out_dtype=_TYPES[out])
    if op == "w4a16":
        return int4.gemv_w4a16(st["xt"], *w, group_size=st["group"], out_dtype=_TYPES[out])
    return int4.gemv_w4a8(st["xq"], st["sx"], *w, group_size=st["group"], out_dtype=_TYPES[out])


def work(case):
    size = {"f32": 4, "bf16": 2, "": 0}
    op = case["op"]
    if op == "norm":
        R, C = case["rows"], case["cols"]
        G = -(-C // case["group"]) if case["group"] else 1
        return {"bytes": R * C * (size[case["x"]] + 2 * size[case["residual"]] + 1) + 4 * R * G + 2 * C, "flops": 8 * R * C}
    N, K, G = case["N"], case["K"], -(-case["K"] // case["group"])
    packed = N * K // 2 + N * G * (2 if case["symmetric"] else 3)
    if op == "quantize":
        return {"bytes": N * K * size[case["x"]] + packed, "flops": 4 * N * K}
    if op == "dequant":
        return {"bytes": packed + N * K * size[case["out"]], "flops": 2 * N * K}
    M = case["M"]
    x = 2 * M * K if op == "w4a16" else M * K + 4 * M * (G if case["x_group"] else 1)
    return {"bytes": packed + x + M * N * size[case["out"]], "flops": 2 * M * N * K}


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "quantize":
        # codes and zero points are whole numbers; the scale before its roundings
        w, step = st["wt"].double(), st["group"]
        parts = w.split(step, 1)
        if st["symmetric"]:
            s = torch.stack([p.abs().max(1).values for p in parts], 1) / 7
            return None, s
        s = torch.stack([p.max(1).values.clamp(min=0) - p.min(1).values.clamp(max=0) for p in parts], 1) / 15
        return None, s, None
    if op == "norm":
        h = st["xt"].double() if st["rt"] is None else st["xt"].double() + st["rt"].double()
        # the norm is taken of the sum as it is stored
        d = h if st["rt"] is None else h.to(st["rt"].dtype).double()
        y = d / torch.sqrt(d.square().sum(1, keepdim=True) / d.shape[1] + st["eps"]) * st["wt"].double()
        parts = y.split(st["group"] or y.shape[1], 1)
        s = torch.stack([p.abs().max(1).values for p in parts], 1) / _TOP[st["out"]]
        if st["out"] == "int8":
            q = None
        else:
            unit = s.float().double().repeat_interleave(st["group"] or y.shape[1], 1)[:, :y.shape[1]]
            v = y / unit
            mag = v.abs().clamp(min=2.0 ** -6)
            step = torch.exp2(torch.floor(torch.log2(mag)) - 3)
            q = (v / step).round() * step
        return (q, s) if st["rt"] is None else (q, s, h)
    N, K = st["c"].shape[0], st["c"].shape[1] * 2
    k = torch.arange(K, device="cuda")
    byte = st["c"][:, (k // 8) * 4 + k % 4].int()
    code = torch.where((k % 8 >= 4)[None, :], byte // 16, byte % 16).double()
    at = k // st["group"]
    w = st["s"].double()[:, at] * (code - (8 if st["z"] is None else st["z"].double()[:, at]))
    if op == "dequant":
        return w
    if op == "w4a16":
        return st["xt"].double() @ w.T
    x = st["xq"].float().double() * (st["sx"].double()[:, at] if st["x_group"] else st["sx"].double())
    return x @ w.T
