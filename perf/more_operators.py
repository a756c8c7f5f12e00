"""Workloads of the 8-bit path of a decoder layer: weights in 128 x 128 blocks
and activations in groups quantized to 8 bits, the block-scaled FP8 product
(dit_quantization_amd.fp8), and the paged 8-bit key/value cache, quantized as
it is written and read back (dit_quantization_amd.kvcache).

`run` makes one call of an operator: in plain torch operations where `own` is
False, through the library where it is True.  `exact` evaluates the operator's
definition in 64 bits.

A scale is fp32(max|v| / top) of the values it serves (1 where that is 0), top
448 for E4M3 and 127 for INT8, and a code the value nearest to v / scale, ties
to even.  The definitions fix every code, so these are compared as they are
stored; E4M3 codes are values of their type.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_TOP = {"int8": 127.0, "e4m3": 448.0}
_SIZE = {"f32": 4, "bf16": 2}
_MOST = 4096 * 14336 * 4096   # products of the largest listed case
_CELLS = 65536 * 8 * 128      # elements of K (and of V) of the largest read


def listed():
    return [
        # Converting a checkpoint: the gate weight from 32 bits.
        {"name": "quantize_14336x4096_f32", "op": "quantize", "N": 14336, "K": 4096, "x": "f32"},
        # A fused projection from bf16 whose rows and columns end inside a block.
        {"name": "quantize_1100x4112_bf16", "op": "quantize", "N": 1100, "K": 4112, "x": "bf16"},
        # The MLP's middle of a prefill of 4096 tokens: SiLU, product, E4M3 in groups of 128 for the down product.
        {"name": "act_silu_4096x14336", "op": "act", "M": 4096, "K": 14336, "x": "bf16", "silu": True, "out": "e4m3", "group": 128},
        # Attention outputs of a decode batch to INT8 in groups of 64 (what the 4-bit products take): latency.
        {"name": "act_int8_13x4096", "op": "act", "M": 13, "K": 4096, "x": "bf16", "silu": False, "out": "int8", "group": 64},
        # One token through a key projection: latency.
        {"name": "gemm_m1_1024x4096", "op": "gemm", "M": 1, "N": 1024, "K": 4096, "out": "bf16"},
        # A decode batch through the down weight.
        {"name": "gemm_m16_4096x14336", "op": "gemm", "M": 16, "N": 4096, "K": 14336, "out": "bf16"},
        # A short prompt with odd sizes through a projection, to 32 bits.
        {"name": "gemm_m333_5000x4112_f32", "op": "gemm", "M": 333, "N": 5000, "K": 4112, "out": "f32"},
        # A prefill of 4096 tokens through the gate weight.
        {"name": "gemm_m4096_14336x4096", "op": "gemm", "M": 4096, "N": 14336, "K": 4096, "out": "bf16"},
        # One new token of each of 33 sequences appended to the cache: latency.
        {"name": "write_decode_33x8x128", "op": "write", "B": 33, "T": 33, "H": 8, "D": 128, "page": 16, "x": "bf16", "code": "e4m3", "most": 2048},
        # A packed prefill of five prompts of uneven lengths, INT8.
        {"name": "write_prefill_8191x8x128", "op": "write", "B": 5, "T": 8191, "H": 8, "D": 128, "page": 64, "x": "bf16", "code": "int8", "most": 1},
        # A prefix of one sequence for the next chunk of its prompt, heads of 80, to 32 bits.
        {"name": "read_prefix_777x4x80_f32", "op": "read", "B": 1, "T": 777, "H": 4, "D": 80, "page": 16, "code": "int8", "out": "f32", "most": 1},
        # Everything that 48 sequences hold, for a library's attention.
        {"name": "read_batch_65536x8x128", "op": "read", "B": 48, "T": 65536, "H": 8, "D": 128, "page": 64, "code": "e4m3", "out": "bf16", "most": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "act", "gemm", "gemm", "gemm", "write", "read"])
    if op in ("write", "read"):
        H, D = rng.choice([1, 2, 4, 5, 8, 8, 16, 32]), rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
        T = _log(rng, 1, max(2, (_CELLS if op == "read" else _CELLS // 8) // (H * D)))
        B = min(T, _log(rng, 1, 256))
        if op == "write" and rng.random() < 0.3:
            T = B
        case = {"op": op, "B": B, "T": T, "H": H, "D": D, "page": rng.choice([1, 7, 16, 16, 32, 64, 128]), "code": rng.choice(["e4m3", "int8"]),
                "most": rng.choice([1, 500, 2000]) if (T + B * 2000) * H * D <= _CELLS else 1}
        return {**case, "x": rng.choice(["bf16", "bf16", "f32"])} if op == "write" else {**case, "out": rng.choice(["bf16", "bf16", "f32"])}
    K = 16 * _log(rng, 8, 896)
    if op == "act":
        return {"op": op, "M": _log(rng, 1, max(2, 4096 * 14336 // K // 2)), "K": K, "x": rng.choice(["bf16", "bf16", "f32"]), "silu": rng.random() < 0.6,
                "out": rng.choice(["e4m3", "e4m3", "int8"]), "group": rng.choice([32, 64, 128, 128])}
    N = _log(rng, 64, min(32768, 14336 * 4096 // K))
    if op == "quantize":
        return {"op": op, "N": N, "K": K, "x": rng.choice(["f32", "bf16"])}
    return {"op": op, "M": _log(rng, 1, min(4096, _MOST // (N * K))), "N": N, "K": K, "out": rng.choice(["bf16", "bf16", "bf16", "f32"])}


# ---- plain forms

def _to_e4m3(v):
    """64-bit values, rounded once to the nearest E4M3 value (ties to even, at most 448)."""
    _, e = torch.frexp(v)
    # 2^(exponent - 3) by its bits: a power that is computed is not always exact, which would decide ties
    step = (((e - 1).clamp(min=-6).long() + 1020) << 52).view(torch.float64)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _codes(t, s, code):
    # next to rounding borders: in 64 bits
    v = t.double() / s.double()
    return torch.round(v).clamp(-127, 127) if code == "int8" else _to_e4m3(v)


def _scale(top_value, code):
    s = (top_value.double() / _TOP[code]).float()
    return torch.where(s == 0, torch.ones_like(s), s)


def _blocks(t, rows, cols):
    """[R, C] as [R', rows, C', cols], filled up with zeros."""
    t = torch.nn.functional.pad(t, (0, -t.shape[1] % cols, 0, -t.shape[0] % rows))
    return t.reshape(t.shape[0] // rows, rows, t.shape[1] // cols, cols)


def _quantized(t, rows, cols, code):
    b = _blocks(t, rows, cols)
    s = _scale(b.abs().amax((1, 3)), code)
    q = _codes(b, s[:, None, :, None], code)
    q = q.reshape(q.shape[0] * rows, -1)[:t.shape[0], :t.shape[1]]
    return q.to(_TYPES[code]), s


def _spread(q, s, rows, cols):
    """Codes times scales in 32 bits."""
    v = _blocks(q.float(), rows, cols) * s[:, None, :, None]
    return v.reshape(v.shape[0] * rows, -1)[:q.shape[0], :q.shape[1]]


def _slots(st):
    """Rows of the cache of all tokens, a token's sequence the last that starts at or before it."""
    t = torch.arange(st["T"], device=st["cu"].device, dtype=torch.int32)
    b = torch.searchsorted(st["cu"][1:].contiguous(), t, right=True)
    at = (st["starts"][b] + t - st["cu"][b]).long()
    return st["table"][b, at // st["page"]].long() * st["page"] + at % st["page"]


def _lengths(total, parts, g):
    """`parts` positive lengths of uneven sizes with the given total."""
    share = torch.rand(parts, generator=g, device="cuda") + 0.1
    n = 1 + torch.floor(share / share.sum() * (total - parts)).to(torch.int64)
    n[0] += total - n.sum()
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def loud(cols):
        # a few loud channels, as a trained model's activations have
        return torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)

    op = case["op"]
    if op in ("write", "read"):
        B, T, H, D, page = case["B"], case["T"], case["H"], case["D"], case["page"]
        n = _lengths(T, B, g)
        # positions of the first tokens: 0, or up to `most` tokens that the cache already holds
        starts = torch.floor(torch.rand(B, generator=g, device="cuda") * case["most"]).to(torch.int64)
        pages = (starts + n + page - 1) // page
        width, total = int(pages.max()), (T + B * case["most"]) // page + B  # the cache's size goes by the case alone
        # pages in the order in which a busy allocator hands them out; -1 behind a sequence's last
        order = torch.randperm(total, generator=g, device="cuda")
        first = torch.cumsum(pages, 0) - pages
        col = torch.arange(width, device="cuda")
        table = torch.where(col < pages[:, None], order[(first[:, None] + col).clamp(max=total - 1)], -1).to(torch.int32)
        cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        cu[1:] = torch.cumsum(n, 0)
        st = {**case, "table": table, "cu": cu, "starts": starts.to(torch.int32)}
        if op == "write":
            # slices of a fused projection's rows
            qkv = normal(T, 3, H, D)
            qkv[:, 1] *= loud(D)
            qkv = qkv.to(_TYPES[case["x"]])
            cache = [torch.zeros(total, page, H, D, device="cuda").to(_TYPES[case["code"]]) if i % 2 == 0 else
                     torch.zeros(total, page, H, device="cuda") for i in range(4)]
            return {**st, "k": qkv[:, 1], "v": qkv[:, 2], "cache": tuple(cache)}
        cache = []
        for _ in range(2):
            t = normal(total * page * H, D) * loud(D)
            s = _scale(t.abs().amax(1), case["code"])
            q = t / s[:, None]
            q = torch.round(q).clamp(-127, 127) if case["code"] == "int8" else q.clamp(-448, 448)
            cache += [q.to(_TYPES[case["code"]]).reshape(total, page, H, D), s.reshape(total, page, H)]
        return {**st, "cache": tuple(cache)}
    if op == "act":
        x = (normal(case["M"], case["K"]) * loud(case["K"])).to(_TYPES[case["x"]])
        gate = (normal(case["M"], case["K"]) * 2).to(_TYPES[case["x"]]) if case["silu"] else None
        return {**case, "xt": x, "gate": gate}
    N, K = case["N"], case["K"]
    # weights whose rows differ in spread (each row's over the root of a mean of five squares), as trained ones do
    w = normal(N, K) * 0.02
    w *= torch.rsqrt(sum(normal(N, 1).square() for _ in range(5)) / 5)
    if op == "quantize":
        return {**case, "wt": w.to(_TYPES[case["x"]])}
    q, s = _quantized(w, 128, 128, "e4m3")
    x, xs = _quantized(normal(case["M"], K) * loud(K), 1, 128, "e4m3")
    return {**case, "q": q, "s": s, "xq": x, "xs": xs}


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    op = st["op"]
    if op == "quantize":
        return _quantized(st["wt"].float(), 128, 128, "e4m3")
    if op == "act":
        y = st["xt"].double()
        if st["gate"] is not None:
            # products next to rounding borders: in 64 bits
            gate = st["gate"].double()
            y = gate / (1 + torch.exp(-gate)) * y
        return _quantized(y, 1, st["group"], st["out"])
    if op == "gemm":
        return (_spread(st["xq"], st["xs"], 1, 128) @ _spread(st["q"], st["s"], 128, 128).t()).to(_TYPES[st["out"]])
    slots = _slots(st)
    if op == "write":
        for new, codes, scales in ((st["k"], *st["cache"][:2]), (st["v"], *st["cache"][2:])):
            s = _scale(new.float().abs().amax(2), st["code"])
            # (bytes: an index assignment takes no 8-bit floating point)
            codes.view(torch.uint8).flatten(0, 1)[slots] = _codes(new, s[..., None], st["code"]).to(codes.dtype).view(torch.uint8)
            scales.flatten(0, 1)[slots] = s
        return st["cache"]
    return tuple((codes.view(torch.uint8).flatten(0, 1)[slots].view(codes.dtype).float() * scales.flatten(0, 1)[slots][..., None]).to(_TYPES[st["out"]])
                 for codes, scales in (st["cache"][:2], st["cache"][2:]))


def _run_own(st):
    from dit_quantization_amd import fp8, kvcache
    op = st["op"]
    if op == "quantize":
        return fp8.quantize(st["wt"])
    if op == "act":
        return fp8.quantize_act(st["xt"], st["gate"], group_size=st["group"], out_dtype=_TYPES[st["out"]])
    if op == "gemm":
        return fp8.gemm(st["xq"], st["xs"], st["q"], st["s"], out_dtype=_TYPES[st["out"]])
    if op == "write":
        kvcache.write(st["k"], st["v"], st["cache"], st["table"], st["cu"], st["starts"])
        return st["cache"]
    return kvcache.read(st["cache"], st["table"], st["cu"], st["starts"], tokens=st["T"], out_dtype=_TYPES[st["out"]])


def work(case):
    op = case["op"]
    if op in ("write", "read"):
        T, H, D = case["T"], case["H"], case["D"]
        wide = _SIZE[case["x"] if op == "write" else case["out"]]
        # both tensors; the sequences' places and a page number for each page that a token touches
        return {"bytes": 2 * T * H * (D * (wide + 1) + 4) + 8 * case["B"] + 4 * max(case["B"], T // case["page"]), "flops": 2 * T * H * D * (4 if op == "write" else 1)}
    K = case["K"]
    if op == "act":
        M, G = case["M"], -(-K // case["group"])
        return {"bytes": M * K * (_SIZE[case["x"]] * (2 if case["silu"] else 1) + 1) + 4 * M * G, "flops": M * K * (8 if case["silu"] else 4)}
    N = case["N"]
    blocks = -(-N // 128) * -(-K // 128)
    if op == "quantize":
        return {"bytes": N * K * (_SIZE[case["x"]] + 1) + 4 * blocks, "flops": 4 * N * K}
    M = case["M"]
    return {"bytes": (M + N) * K + 4 * blocks + 4 * M * -(-K // 128) + M * N * _SIZE[case["out"]], "flops": 2 * M * N * K}


# ---- the definitions in 64 bits

def _nearest_e4m3(v):
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return ((v / step).round() * step).clamp(-448, 448)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "quantize":
        w = st["wt"].double()
        s = torch.stack([torch.stack([p.abs().max() for p in rows.split(128, 1)]) for rows in w.split(128, 0)]) / 448
        n, k = torch.arange(w.shape[0], device="cuda") // 128, torch.arange(w.shape[1], device="cuda") // 128
        unit = s.float().double()
        return _nearest_e4m3(w / torch.where(unit == 0, 1.0, unit)[n][:, k]), torch.where(unit == 0, 1.0, s)
    if op == "act":
        y = st["xt"].double()
        if st["gate"] is not None:
            y = y * st["gate"].double() * torch.sigmoid(st["gate"].double())
        k = torch.arange(y.shape[1], device="cuda") // st["group"]
        s = torch.stack([p.abs().max(1).values for p in y.split(st["group"], 1)], 1) / _TOP[st["out"]]
        unit = s.float().double()
        s, unit = torch.where(unit == 0, 1.0, s), torch.where(unit == 0, 1.0, unit)
        return (None if st["out"] == "int8" else _nearest_e4m3(y / unit[:, k])), s
    if op == "gemm":
        k = torch.arange(st["K"], device="cuda") // 128
        n = torch.arange(st["N"], device="cuda") // 128
        return (st["xq"].double() * st["xs"].double()[:, k]) @ (st["q"].double() * st["s"].double()[n][:, k]).T
    # each token's place, sequence by sequence
    cu, starts, table, page = st["cu"].tolist(), st["starts"].tolist(), st["table"], st["page"]
    pages, rows = [], []
    for b in range(st["B"]):
        at = torch.arange(starts[b], starts[b] + cu[b + 1] - cu[b], device="cuda")
        pages.append(table[b].long()[torch.div(at, page, rounding_mode="floor")])
        rows.append(at.remainder(page))
    at = (torch.cat(pages), torch.cat(rows))
    out = []
    for i, new in ((0, st.get("k")), (2, st.get("v"))):
        codes, scales = st["cache"][i], st["cache"][i + 1]
        if op == "read":
            out.append(codes.float()[at].double() * scales.double()[at][..., None])
            continue
        s = new.double().abs().max(2).values / _TOP[st["code"]]
        unit = s.float().double()
        s, unit = torch.where(unit == 0, 1.0, s), torch.where(unit == 0, 1.0, unit)
        held = scales.double().clone()
        held[at] = s
        kept = None
        if st["code"] == "e4m3":
            kept = codes.float().double()
            kept[at] = _nearest_e4m3(new.double() / unit[..., None])
        out += [kept, held]
    return tuple(out)
