"""8-bit operators, measured: the AdamW step with its moments in 8 bits, the
moments' conversion from and to 32 bits, matrices in 8-bit floating point with
a scale for each block of 128, and their products.

`own` selects the framework's kernels; the plain forms below compute the same
from elementary torch operations in 32 bits.

Moments: a block of 256 consecutive elements of a tensor shares a word, the
exponent byte b in its low 8 bits and the number of times it was rounded in the
other 24.  Element j of the block stands for e4m3(code) * 2^(b - 127): m itself,
and for v its square root r (v = r * r).  Matrices: codes are e4m3 or e5m2, a
byte b for each block of 128 columns (of one row or of 128) scales them by
2^(b - 127).
"""
import math

import torch
import torch.nn.functional as F

own = False

LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 7
BLOCK = 256                    # elements of a moment under one word
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def listed():
    return [
        # adamw: a small model's shard at four replicas, one tensor (a call's latency) ...
        dict(name="adamw 1x2^18 W4", op="adamw", layers=0, width=512, hidden=512, vocab=512, W=4, clip=True),
        # ... odd tensors, none a multiple of the block, three replicas, the norm below the limit ...
        dict(name="adamw 1 layer 333x1111 W3", op="adamw", layers=1, width=333, hidden=1111, vocab=0, W=3, clip=False),
        # ... one layer of a model of width 4096 with all of its gradients on one replica ...
        dict(name="adamw 1 layer 4096x11008 W1", op="adamw", layers=1, width=4096, hidden=11008, vocab=0, W=1, clip=True),
        # ... and the same with an embedding at eight replicas
        dict(name="adamw 1 layer 4096x11008 vocab 32000 W8", op="adamw", layers=1, width=4096, hidden=11008, vocab=32000, W=8, clip=True),
        # moments: a small vector's conversion out of a checkpoint; a large matrix's back into one
        dict(name="encode v 100003", op="encode", n=100003, which="v"),
        dict(name="decode m 4096x11008", op="decode", n=4096 * 11008, which="m"),
        # quantize: a block of activations both ways round, for a layer's product and its gradient's;
        # a weight from its 32-bit master both ways round; odd gradients in e5m2
        dict(name="quantize 8192x4096 bf16", op="quantize", rows=8192, cols=4096, pad=0, src="bf16", block=1, code="e4m3", ways="both"),
        dict(name="quantize 11008x4096 fp32 blocks", op="quantize", rows=11008, cols=4096, pad=0, src="fp32", block=128, code="e4m3", ways="both"),
        dict(name="quantize 1001x777 bf16 e5m2", op="quantize", rows=1001, cols=777, pad=23, src="bf16", block=1, code="e5m2", ways="along"),
        # product: one token through a wide layer (the weight is read once) ...
        dict(name="product 1x11008x4096", op="product", m=1, n=11008, k=4096, a="e4m3", b_block=128, out="bf16"),
        # ... an odd batch through a small model's query-key-value projection; its input is ragged
        dict(name="product 1001x2304x777 e5m2", op="product", m=1001, n=2304, k=777, a="e5m2", b_block=1, out="fp32"),
        # ... and a full batch through a large layer
        dict(name="product 8192x11008x4096", op="product", m=8192, n=11008, k=4096, a="e4m3", b_block=128, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "encode", "decode", "quantize", "product", "product"])
    if op == "adamw":
        width, hidden = _log_int(rng, 16, 4096), _log_int(rng, 16, 11008)
        if rng.random() < 0.5:                  # widths of models are round numbers
            width, hidden = -(-width // 64) * 64, -(-hidden // 64) * 64
        return dict(op=op, layers=1, width=width, hidden=hidden, vocab=rng.choice([0, 0, _log_int(rng, 16, 32000)]),
                    W=rng.choice([1, 2, 3, 4, 5, 8]), clip=rng.random() < 0.7)
    if op in ("encode", "decode"):
        return dict(op=op, n=_log_int(rng, 1, 4096 * 11008), which=rng.choice(["m", "v"]))
    if op == "quantize":
        rows = _log_int(rng, 1, 11008)
        cols = _log_int(rng, 1, min(11008, (44 << 20) // rows))
        if rng.random() < 0.5:
            rows, cols = -(-rows // 128) * 128, -(-cols // 128) * 128
        block = rng.choice([1, 1, 128])
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 1, 8, 23]), src=rng.choice(["bf16", "fp32"]), block=block,
                    code=rng.choice(["e4m3", "e5m2"]), ways=rng.choice(["along", "across", "both"]))
    m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 16, 11008), _log_int(rng, 16, 8192)
    if rng.random() < 0.5:
        n, k = -(-n // 128) * 128, -(-k // 128) * 128
    k = max(16, min(k, (8192 * 11008 * 4096) // (m * n)))
    return dict(op=op, m=m, n=n, k=k, a=rng.choice(["e4m3", "e4m3", "e5m2"]), b_block=rng.choice([1, 128]),
                out=rng.choice(["bf16", "bf16", "fp32"]))


def _sizes(case):
    """The shard's tensors: an embedding, and of each layer four square matrices, three of the feed-forward block, two gains."""
    w, h = case["width"], case["hidden"]
    return ([case["vocab"] * w] if case["vocab"] else []) + case["layers"] * (4 * [w * w] + 3 * [w * h] + 2 * [w])


# ------------------------------------------------------------------ formats
def _exponent(amax, most):
    """The exponent byte that brings amax (>= 0, fp32) to just below 2^(most + 1)."""
    return ((amax.view(torch.int32) >> 23) - most).clamp(min=1)


def _exponent_full(amax, most):
    """The exponent byte that brings amax (>= 0, fp32) to at most 1.75 * 2^most, and over half of that."""
    u = amax.view(torch.int32)
    return ((u >> 23) - most + ((u & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp(min=1)


def _power(b):
    """2^(b - 127) of exponent bytes b >= 1; 0 for b = 0, as a block of zeros has it."""
    return (b.to(torch.int32) << 23).view(torch.float32)


def _decode(codes, words):
    """What a moment's codes stand for: [blocks, 256] in fp32."""
    return codes.view(E4M3).view(-1, BLOCK).float() * _power(words & 255)[:, None]


def _encode_nearest(x):
    """Codes and words (rounded no times) of [blocks, 256] values, to the nearest, ties to even."""
    b = _exponent(x.abs().amax(1), 7)
    y = x * _power(254 - b)[:, None]
    return y.to(E4M3).view(torch.uint8).view(-1), b


def _mix(x):
    """32 well-mixed bits of 32 (in int64): the multipliers are the fractions of the roots of 2 and 3."""
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _encode_random(x, bits, count, positive):
    """Codes and words of [blocks, 256] values: up with the probability of what lies below, by 16 random bits."""
    b = _exponent(x.abs().amax(1), 7)
    u = ((x.abs() * _power(254 - b)[:, None]) * 2.0 ** -120).view(torch.int32)
    code = (u + (bits.to(torch.int32) << 4)) >> 20
    if positive:                                # a square root that is not zero stays so
        code = torch.maximum(code, (x > 0).to(torch.int32))
    else:
        code = code | (torch.signbit(x).to(torch.int32) << 7)
    return code.to(torch.uint8).view(-1), ((count + 1) & 0xFFFFFF) << 8 | b


def _pad(x, sizes):
    return torch.cat([F.pad(t, (0, -n % BLOCK)) for t, n in zip(x.split(sizes), sizes)]).view(-1, BLOCK)


def _pieces(x, sizes, unit=1):
    """Of a padded array, each tensor's part."""
    whole = [(n + BLOCK - 1) // BLOCK * BLOCK // unit for n in sizes]
    return [t[:-(-n // unit)] for t, n in zip(x.split(whole), sizes)]


def _blocks_of(x, block):
    """[rows, cols] padded to whole blocks: [row blocks, block, column blocks, 128]."""
    rows, cols = x.shape
    x = F.pad(x, (0, -cols % 128, 0, -rows % block))
    return x.view(-1, block, x.shape[1] // 128, 128)


def _quantize(x, block, code):
    """Codes [rows, cols] and exponent bytes [row blocks, column blocks] of an fp32 matrix."""
    rows, cols = x.shape
    t = _blocks_of(x, block)
    amax = t.abs().amax((1, 3))
    b = _exponent_full(amax, 8 if code == "e4m3" else 15)    # the formats end at 1.75 * 2^8 and 1.75 * 2^15
    y = t * _power(254 - b)[:, None, :, None]
    q = y.to(E4M3 if code == "e4m3" else E5M2)
    q = q.view(torch.uint8).reshape(-1, t.shape[2] * 128)[:rows, :cols].contiguous()
    return q, b.to(torch.uint8)


def _values(q, scales, block, code):
    """What a matrix's codes stand for."""
    rows, cols = q.shape
    v = q.view(E4M3 if code == "e4m3" else E5M2).float()
    s = _power(scales).repeat_interleave(128, 1)[:, :cols]
    return v * (s.repeat_interleave(block, 0)[:rows] if block > 1 else s)


# ------------------------------------------------------------------ inputs
def _spread(gen, n, size):
    """Values as gradients and momenta are: rows of 1000 that differ by orders of magnitude."""
    rows = -(-n // 1000)
    x = torch.randn(rows, 1000, generator=gen, device="cuda")
    return (x.mul_(size * torch.exp(1.5 * torch.randn(rows, 1, generator=gen, device="cuda")))).view(-1)[:n]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "adamw":
        sizes = s["sizes"] = _sizes(case)
        total = sum(sizes)
        base = _spread(gen, total, 1e-3)
        s["grads"] = [(base * (1 + 0.5 * torch.randn(total, generator=gen, device="cuda"))).to(torch.bfloat16) for _ in range(case["W"])]
        s["m"] = _encode_nearest(_pad(base * 0.7, sizes))
        s["v"] = _encode_nearest(_pad((base * 1.2).abs() + 1e-7, sizes))
        s["m"], s["v"] = ([c, b + (STEP - 1 << 8)] for c, b in (s["m"], s["v"]))
        s["master"] = 0.02 * torch.randn(total, generator=gen, device="cuda")
        s["param"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda")
        s["max_norm"] = 1e-2 if case["clip"] else math.inf
    elif op in ("encode", "decode"):
        x = _spread(gen, case["n"], 1e-3)
        s["x"] = x.square() if case["which"] == "v" else x
        s["state"] = _encode_nearest(_pad(x.abs() if case["which"] == "v" else x, [case["n"]]))
    elif op == "quantize":
        x = _spread(gen, case["rows"] * (case["cols"] + case["pad"]), 1.0).view(case["rows"], -1)
        s["x"] = x.to(torch.bfloat16 if case["src"] == "bf16" else torch.float32)[:, :case["cols"]]
    else:
        a = _spread(gen, case["m"] * case["k"], 1.0).view(case["m"], -1)
        b = 0.02 * torch.randn(case["n"], case["k"], generator=gen, device="cuda")
        s["a"] = _quantize(a, 1, case["a"])
        s["b"] = _quantize(b, case["b_block"], "e4m3")
    if own:
        _plan(s, case)
    return s


def _plan(s, case):
    """What a program keeps: the moments' buffers and the plan over them, the quantised operands, the outputs, workspaces."""
    import zero_sharded_mixed_zero1_amd as z
    s["z"] = z
    op = s["op"]

    def buffer(codes, words, n):
        """One tensor's moment as the framework holds it, with views of its codes and words."""
        t = torch.zeros(z.state8_bytes(n), dtype=torch.uint8, device="cuda")
        blocks = -(-n // BLOCK)
        c, w = t[:n], t[-4 * blocks:].view(torch.int32)
        c.copy_(codes)
        w.copy_(words)
        return t, c.view(E4M3), w

    def matrix(rows, cols, block, code, q=None, scales=None):
        """A matrix in 8 bits as the framework holds it, with views of its codes and scales."""
        codes = torch.zeros(rows, -(-cols // 128) * 128, dtype=torch.uint8, device="cuda")
        e = torch.zeros(-(-rows // block), -(-cols // 512) * 4, dtype=torch.uint8, device="cuda")
        c, b = codes[:, :cols], e[:, :-(-cols // 128)]
        if q is not None:
            c.copy_(q)
            b.copy_(scales)
        return z.f8_matrix(rows, cols, codes, e, block_rows=block, flags=z.E5M2 if code == "e5m2" else 0), c, b, (codes, e)

    if op == "adamw":
        sizes, total = s["sizes"], sum(s["sizes"])
        m = [buffer(c, w, n) for c, w, n in zip(_pieces(s["m"][0], sizes), _pieces(s["m"][1], sizes, BLOCK), sizes)]
        v = [buffer(c, w, n) for c, w, n in zip(_pieces(s["v"][0], sizes), _pieces(s["v"][1], sizes, BLOCK), sizes)]
        at = [sum(sizes[:k]) for k in range(len(sizes))]
        pieces = [(n, o, s["param"][o:], s["master"][o:], mk[0], vk[0]) for n, o, mk, vk in zip(sizes, at, m, v)]
        s["table"] = torch.empty(z.mta_table_bytes(pieces), dtype=torch.uint8, device="cuda")
        s["plan"] = z.mta_plan(pieces, s["table"], flags=z.MV_8BIT)
        s["ws"] = torch.empty(z.mta_workspace_bytes(s["plan"], case["W"]), dtype=torch.uint8, device="cuda")
        s["sumsq"] = torch.zeros(1, dtype=torch.float64, device="cuda")
        s["hp"] = dict(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, max_norm=s["max_norm"], step=STEP)
        s["kept"] = (m, v)
        s["out"] = {"master": s["master"], "param": s["param"], "m": [t[1] for t in m], "m_words": [t[2] for t in m],
                    "v": [t[1] for t in v], "v_words": [t[2] for t in v]}
        del s["m"], s["v"]
    elif op in ("encode", "decode"):
        n = case["n"]
        s["which"] = z.STATE_V if case["which"] == "v" else z.STATE_M
        s["kept"], codes, words = buffer(s["state"][0][:n], s["state"][1], n)
        if op == "encode":
            s["kept"].zero_()
            s["out"] = {"codes": codes, "words": words}
        else:
            s["y"] = torch.empty(n, device="cuda")
            s["out"] = {"x": s["y"]}
        del s["state"]
    elif op == "quantize":
        rows, cols, block, code = case["rows"], case["cols"], case["block"], case["code"]
        dtype = E5M2 if code == "e5m2" else E4M3
        s["out"], s["q"], s["qt"] = {}, None, None
        if case["ways"] != "across":
            s["q"], c, b, s["kept"] = matrix(rows, cols, block, code)
            s["out"].update(q=c.view(dtype), scales=b)
        if case["ways"] != "along":
            s["qt"], c, b, s["kept_t"] = matrix(cols, rows, block, code)
            s["out"].update(qt=c.view(dtype), scales_t=b)
        s["flags"] = z.F32 if case["src"] == "fp32" else 0
    else:
        s["fa"], _, _, s["kept_a"] = matrix(case["m"], case["k"], 1, case["a"], *s["a"])
        s["fb"], _, _, s["kept_b"] = matrix(case["n"], case["k"], case["b_block"], "e4m3", *s["b"])
        s["flags"] = z.F32 if case["out"] == "fp32" else 0
        s["d"] = torch.empty(case["m"], case["n"], dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16, device="cuda")
        s["ws"] = torch.empty(z.f8_product_workspace_bytes(s["fa"], s["fb"], flags=s["flags"]), dtype=torch.uint8, device="cuda")
        del s["a"], s["b"]


def _run_own(s):
    z, op = s["z"], s["op"]
    if op == "adamw":
        z.mta_step(s["grads"], 0, s["plan"], s["hp"], s["sumsq"], 1, 0, ws=s["ws"])
    elif op == "encode":
        z.state8_encode(s["x"], s["case"]["n"], s["kept"], s["which"])
    elif op == "decode":
        z.state8_decode(s["kept"], s["case"]["n"], s["y"], s["which"])
    elif op == "quantize":
        z.f8_quantize(s["x"], s["case"]["rows"], s["case"]["cols"], q=s["q"], qt=s["qt"], ld=s["x"].stride(0), flags=s["flags"])
    else:
        z.f8_product(s["fa"], s["fb"], s["d"], flags=s["flags"], ws=s["ws"])
        return {"d": s["d"]}
    return s["out"]


# ------------------------------------------------------------------ plain forms
def _starts(sizes, device):
    """The shard's position of each block's first element, low 32 bits."""
    return torch.cat([torch.arange(o, o + n, BLOCK, device=device) for o, n in zip([sum(sizes[:k]) for k in range(len(sizes))], sizes)]) & 0xFFFFFFFF


def _adamw(s):
    case, sizes = s["case"], s["sizes"]
    g = sum((t.float() for t in s["grads"][1:]), s["grads"][0].float())
    g = g / torch.full((), case["W"], dtype=torch.float32, device=g.device)    # a division: a number would be inverted first
    norm = g.double().square().sum().sqrt()
    clip = s["max_norm"] / norm
    g = torch.where(norm > s["max_norm"], g * clip.float(), g)
    g = _pad(g, sizes)
    r = _decode(*s["v"])
    m = BETA1 * _decode(*s["m"]) + (1 - BETA1) * g
    v = BETA2 * (r * r) + (1 - BETA2) * (g * g)
    r = torch.sqrt(v)
    q = torch.cat(_pieces((m / (r + EPS)).view(-1), sizes))
    p = (s["master"] - LR * math.sqrt(1 - BETA2 ** STEP) / (1 - BETA1 ** STEP) * q) * (1 - LR * DECAY)
    count = (s["m"][1] >> 8) & 0xFFFFFF
    key = _mix((_mix(_starts(sizes, g.device)) + count) & 0xFFFFFFFF)
    bits = _mix((key[:, None] + torch.arange(BLOCK, device=g.device)) & 0xFFFFFFFF)
    s["m"] = _encode_random(m, bits & 0xFFFF, count, False)
    s["v"] = _encode_random(r, bits >> 16, (s["v"][1] >> 8) & 0xFFFFFF, True)
    s["master"].copy_(p)
    s["param"].copy_(p)
    return {"master": s["master"], "param": s["param"],
            "m": [c.view(E4M3) for c in _pieces(s["m"][0], sizes)], "m_words": _pieces(s["m"][1], sizes, BLOCK),
            "v": [c.view(E4M3) for c in _pieces(s["v"][0], sizes)], "v_words": _pieces(s["v"][1], sizes, BLOCK)}


def run(s):
    if own:
        return _run_own(s)
    case, op = s["case"], s["op"]
    if op == "adamw":
        return _adamw(s)
    if op == "encode":
        x = s["x"].sqrt() if case["which"] == "v" else s["x"]
        codes, words = _encode_nearest(_pad(x, [case["n"]]))
        if case["which"] == "v":                # a square root that is not zero stays so
            codes = torch.maximum(codes, (_pad(x, [case["n"]]) > 0).view(-1).to(torch.uint8))
        return {"codes": codes[:case["n"]].view(E4M3), "words": words}
    if op == "decode":
        x = _decode(*s["state"]).view(-1)[:case["n"]]
        return {"x": x * x if case["which"] == "v" else x}
    if op == "quantize":
        out, x, dtype = {}, s["x"].float(), E5M2 if case["code"] == "e5m2" else E4M3
        if case["ways"] != "across":
            q, b = _quantize(x, case["block"], case["code"])
            out.update(q=q.view(dtype), scales=b)
        if case["ways"] != "along":
            q, b = _quantize(x.t().contiguous(), case["block"], case["code"])
            out.update(qt=q.view(dtype), scales_t=b)
        return out
    d = _values(*s["a"], 1, case["a"]) @ _values(*s["b"], case["b_block"], "e4m3").t()
    return {"d": d if case["out"] == "fp32" else d.to(torch.bfloat16)}


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        words = 4 * sum(-(-k // BLOCK) for k in _sizes(case))
        return {"bytes": n * (2 * case["W"] + 8 + 2 + 4) + 4 * words, "flops": n * (case["W"] + 40)}
    if op in ("encode", "decode"):
        return {"bytes": 5 * case["n"] + 4 * -(-case["n"] // BLOCK), "flops": 6 * case["n"]}
    if op == "quantize":
        e, ways = case["rows"] * case["cols"], 2 if case["ways"] == "both" else 1
        return {"bytes": e * ((2 if case["src"] == "bf16" else 4) + ways), "flops": 4 * e}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": (m + n) * k + m * n * (4 if case["out"] == "fp32" else 2), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ 64 bits
def _rounded(y, mantissa, low, more=None):
    """y in 64 bits on a format's grid: to the nearest, ties to even, or up by the share `more` of a step; magnitudes and signs apart."""
    _, e = torch.frexp(y)
    step = torch.exp2((e.to(y.dtype) - 1).clamp(min=low) - mantissa)
    k = y.abs() / step
    return torch.copysign((torch.round(k) if more is None else torch.floor(k + more)) * step, y)


def _exact_moment(x, more=None, positive=False):
    """A moment's blocks [blocks, 256] in units of their scales, the largest in [128, 256), on e4m3's grid."""
    _, e = torch.frexp(x.abs().amax(1, keepdim=True))
    y = _rounded(x * torch.exp2(8.0 - e.to(x.dtype).clamp(min=-117)), 3, -6.0, more)
    return torch.where((x > 0) & (y == 0), 2.0 ** -9, y) if positive else y


def _shares(begins, counts):
    """Sixteen random bits twice for each element, as shares of 65536: a block's number and count, then the place in it."""
    def scatter(x):
        for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
            x = torch.remainder(torch.bitwise_xor(x, x // 2 ** shift) * factor, 2 ** 32)
        return torch.bitwise_xor(x, x // 2 ** 16)
    h = scatter(torch.remainder(begins, 2 ** 32))
    h = scatter(torch.remainder(h + counts, 2 ** 32))
    h = scatter(torch.remainder(h[:, None] + torch.arange(BLOCK, device=h.device)[None], 2 ** 32))
    return torch.remainder(h, 65536).double() / 65536, (h // 65536).double() / 65536


def exact(case, seed):
    """The definitions in 64 bits; 8-bit outputs in units of their blocks' scales."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "adamw":
        sizes = s["sizes"]
        mean = torch.zeros(sum(sizes), dtype=f64, device="cuda")
        for g in s["grads"]:
            mean += g.to(f64)
        mean /= case["W"]
        norm = float(torch.linalg.vector_norm(mean))
        if norm > s["max_norm"]:
            mean *= s["max_norm"] / norm
        mean = torch.cat([F.pad(t, (0, -len(t) % BLOCK)) for t in mean.split(sizes)]).view(-1, BLOCK)
        scale = torch.exp2((s["m"][1] & 255).to(f64) - 127)[:, None]
        m = s["m"][0].view(E4M3).to(f64).view(-1, BLOCK) * scale * BETA1 + mean * (1 - BETA1)
        scale = torch.exp2((s["v"][1] & 255).to(f64) - 127)[:, None]
        r = torch.sqrt((s["v"][0].view(E4M3).to(f64).view(-1, BLOCK) * scale) ** 2 * BETA2 + mean ** 2 * (1 - BETA2))
        begins = torch.cat([torch.arange(-(-n // BLOCK), device="cuda") * BLOCK + sum(sizes[:k]) for k, n in enumerate(sizes)])
        share_m, share_r = _shares(begins, (s["m"][1] // 256).long())
        move = torch.cat([t[:n] for t, n in zip((m / (r + EPS)).view(-1).split([-(-n // BLOCK) * BLOCK for n in sizes]), sizes)])
        p = s["master"].to(f64)
        p = (p - move * (LR * math.sqrt(1 - BETA2 ** STEP) / (1 - BETA1 ** STEP))) * (1 - LR * DECAY)
        cut = [-(-n // BLOCK) * BLOCK for n in sizes]
        return {"master": p, "param": p, "m": [t[:n] for t, n in zip(_exact_moment(m, share_m).view(-1).split(cut), sizes)], "m_words": None,
                "v": [t[:n] for t, n in zip(_exact_moment(r, share_r, True).view(-1).split(cut), sizes)], "v_words": None}
    if op == "encode":
        x = s["x"].to(f64)
        x = torch.sqrt(x) if case["which"] == "v" else x
        x = F.pad(x, (0, -case["n"] % BLOCK)).view(-1, BLOCK)
        return {"codes": _exact_moment(x, positive=case["which"] == "v").view(-1)[:case["n"]], "words": None}
    if op == "decode":
        codes, words = s["state"]
        x = (codes.view(E4M3).to(f64).view(-1, BLOCK) * torch.exp2((words & 255).to(f64) - 127)[:, None]).view(-1)[:case["n"]]
        return {"x": x ** 2 if case["which"] == "v" else x}
    if op == "quantize":
        out, (limit, mantissa, low) = {}, (448.0, 3, -6.0) if case["code"] == "e4m3" else (57344.0, 2, -14.0)
        for key, scales, x in (("q", "scales", s["x"]), ("qt", "scales_t", s["x"].t())):
            if case["ways"] in (("across",) if key == "q" else ("along",)):
                continue
            x = x.to(f64)
            rows, cols, block = x.shape[0], x.shape[1], case["block"]
            t = F.pad(x, (0, -cols % 128, 0, -rows % block))
            t = t.reshape(t.shape[0] // block, block, t.shape[1] // 128, 128)
            e = torch.ceil(torch.log2(t.abs().amax((1, 3), keepdim=True).clamp(min=2.0 ** -100) / limit)).clamp(min=-126)
            out.update({key: _rounded(t * torch.exp2(-e), mantissa, low).reshape(-1, t.shape[2] * 128)[:rows, :cols], scales: None})
        return out
    (qa, sa), (qb, sb) = s["a"], s["b"]

    def whole(q, e, block, dtype):
        e = torch.exp2(e.to(f64) - 127)
        rows = torch.arange(q.shape[0], device="cuda") // block
        cols = torch.arange(q.shape[1], device="cuda") // 128
        return q.view(dtype).to(f64) * e[rows][:, cols]

    return {"d": whole(qa, sa, 1, E5M2 if case["a"] == "e5m2" else E4M3) @ whole(qb, sb, case["b_block"], E4M3).T}
