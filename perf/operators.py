"""The Muon step's operators, measured: momentum over the W replicas' gradients,
orthogonalisation of the momentum by Newton-Schulz products, the update of the
fp32 master with the bf16 parameter, and the whole step.

One case is a number of equally shaped weight matrices owned by one
data-parallel rank.  `own` selects the framework's kernels; the plain forms
below compute the same from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

# The quintic's coefficients and the momentum of the Muon step, and the eps
# added to the Frobenius norm.
A, B, C = 3.4445, -4.7750, 2.0315
MU = 0.95
EPS = 1e-7
LR, DECAY = 3e-4, 0.1


def listed():
    return [
        # momentum: one small head's matrix on one replica (a call's latency) ...
        dict(name="momentum 1x64x64 W1", op="momentum", count=1, rows=64, cols=64, pad=0, W=1, m="fp32", u="bf16"),
        # ... odd matrices cut out of wider ones, three replicas, 16-bit state ...
        dict(name="momentum 5x1001x777 W3", op="momentum", count=5, rows=1001, cols=777, pad=23, W=3, m="bf16", u="fp32"),
        # ... and a large model's attention matrices on eight replicas
        dict(name="momentum 4x4096x4096 W8", op="momentum", count=4, rows=4096, cols=4096, pad=0, W=8, m="fp32", u="bf16"),
        # orthogonalize: one small matrix (latency), and a few heads' or adapters' matrices
        dict(name="orthogonalize 1x64x64", op="orthogonalize", count=1, rows=64, cols=64, pad=0, u="bf16", steps=5),
        dict(name="orthogonalize 24x100x1000", op="orthogonalize", count=24, rows=100, cols=1000, pad=0, u="bf16", steps=5),
        # the attention output matrices of a 12-layer model of width 768
        dict(name="orthogonalize 12x768x768", op="orthogonalize", count=12, rows=768, cols=768, pad=0, u="bf16", steps=5),
        # tall and odd, cut out of wider ones, 32-bit momentum
        dict(name="orthogonalize 3x2501x1111", op="orthogonalize", count=3, rows=2501, cols=1111, pad=5, u="fp32", steps=5),
        # two feed-forward matrices of a model of width 4096
        dict(name="orthogonalize 2x4096x11008", op="orthogonalize", count=2, rows=4096, cols=11008, pad=0, u="bf16", steps=5),
        # update: odd matrices cut out of wider ones; a large model's attention matrices
        dict(name="update 5x1001x777", op="update", count=5, rows=1001, cols=777, pad=23),
        dict(name="update 4x4096x4096", op="update", count=4, rows=4096, cols=4096, pad=0),
        # step: the fused query-key-value matrices of a 12-layer model of width 768 on eight
        # replicas; a tall matrix of a large model with 16-bit state on one replica
        dict(name="step 12x768x2304 W8", op="step", count=12, rows=768, cols=2304, pad=0, W=8, m="fp32", u="bf16", steps=5),
        dict(name="step 1x11008x4096 W1", op="step", count=1, rows=11008, cols=4096, pad=0, W=1, m="bf16", u="bf16", steps=5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["momentum", "orthogonalize", "orthogonalize", "update", "step"])
    rows = _log_int(rng, 1, 11008)
    cols = _log_int(rng, 1, min(11008, (36 << 20) // rows))
    if rng.random() < 0.5:                      # as many tall as wide ones
        rows, cols = cols, rows
    if rng.random() < 0.4:                      # widths of models are round numbers
        rows, cols = -(-rows // 64) * 64, -(-cols // 64) * 64
    W = rng.choice([1, 2, 3, 4, 5, 8]) if op in ("momentum", "step") else 1
    steps = rng.choice([3, 5, 5, 5, 6])
    # no more than the largest listed case computes, moves or holds
    k, n = min(rows, cols), max(rows, cols)
    most = min(64, (56 << 20) // (rows * cols), int(1.5e12 / (steps * (4.0 * k * k * n + k ** 3))) if op in ("orthogonalize", "step") else 64)
    count = _log_int(rng, 1, max(1, most))
    pad = rng.choice([0, 0, 1, 8, 23]) if rows > 1 else 0
    c = dict(op=op, count=count, rows=rows, cols=cols, pad=pad)
    if op in ("momentum", "step"):
        c.update(W=W, m=rng.choice(["fp32", "bf16"]))
    if op != "update":
        c.update(u=rng.choice(["bf16", "bf16", "fp32"]))
    if op in ("orthogonalize", "step"):
        c.update(steps=steps)
    return c


_TYPE = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _scale(case):
    """The update's size by the matrix's shape: entries of O have a root mean square of 1/sqrt(max side)."""
    return 0.2 * math.sqrt(max(case["rows"], case["cols"]))


def _update_like(gen, count, rows, cols, size):
    """Matrices as gradients are: a few strong directions over noise."""
    r = min(8, rows, cols)
    left = torch.randn(count, rows, r, generator=gen, device="cuda")
    right = torch.randn(count, r, cols, generator=gen, device="cuda")
    return size * (torch.bmm(left, right) + torch.randn(count, rows, cols, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    count, rows, cols = case["count"], case["rows"], case["cols"]
    ld = cols + case["pad"]
    s = {"case": case, "op": case["op"]}

    def wide(t):
        """The matrices as the first columns of wider ones (row stride ld)."""
        if not case["pad"]:
            return t
        w = torch.zeros(count, rows, ld, dtype=t.dtype, device="cuda")
        w[:, :, :cols] = t
        return w[:, :, :cols]

    if "W" in case:
        base = _update_like(gen, count, rows, cols, 1e-3)
        grads = torch.zeros(case["W"], count, rows, ld, dtype=torch.bfloat16, device="cuda")
        for w in range(case["W"]):              # the replicas share the directions, not the noise
            grads[w, :, :, :cols] = base + 1e-3 * torch.randn(count, rows, cols, generator=gen, device="cuda")
        s["grads"] = grads
        s["slices"] = [grads[w] for w in range(case["W"])]
        s["m"] = wide((5 * base + _update_like(gen, count, rows, cols, 2e-3)).to(_TYPE[case["m"]]))
    if case["op"] == "orthogonalize":
        s["u"] = wide(_update_like(gen, count, rows, cols, 1e-3).to(_TYPE[case["u"]]))
    elif case["op"] != "update":
        s["u"] = torch.zeros(count, rows, cols, dtype=_TYPE[case["u"]], device="cuda")
    if case["op"] in ("update", "step"):
        s["master"] = wide(0.02 * torch.randn(count, rows, cols, generator=gen, device="cuda"))
        s["param"] = wide(s["master"].to(torch.bfloat16))
    if case["op"] == "update":
        s["o"] = (torch.randn(count, rows, cols, generator=gen, device="cuda") / math.sqrt(max(rows, cols))).to(torch.bfloat16)
    elif case["op"] == "orthogonalize":
        s["o"] = torch.zeros(count, rows, cols, dtype=torch.bfloat16, device="cuda")
    if own:
        _plan(s, ld)
    return s


def _plan(s, ld):
    """What a training program sets up once: the plan over its matrices and the workspace."""
    import zero_sharded_mixed_zero1_amd as z
    case = s["case"]

    def at(key, k):
        return s[key][k] if key in s else None

    mats = [z.matrix(case["rows"], case["cols"], ld=ld, shard_offset=k * case["rows"] * ld, scale=_scale(case),
                     param=at("param", k), master=at("master", k), m=at("m", k),
                     u=at("u", k), ldu=s["u"].stride(1) if "u" in s else 0, o=at("o", k))
            for k in range(case["count"])]
    flags = (z.MV_BF16 if case.get("m") == "bf16" else 0) | (z.U_F32 if case.get("u") == "fp32" else 0)
    s["table"] = torch.empty(z.muon_table_bytes(mats), dtype=torch.uint8, device="cuda")
    s["plan"] = z.muon_plan(mats, s["table"], flags=flags)
    s["ws"] = torch.empty(z.muon_workspace_bytes(s["plan"]), dtype=torch.uint8, device="cuda")
    s["hp"] = dict(lr=LR, momentum=MU, weight_decay=DECAY, max_norm=math.inf, ns_steps=case.get("steps", 5),
                   ns_a=A, ns_b=B, ns_c=C, ns_eps=EPS)
    s["z"] = z


def _run_own(s):
    z, op = s["z"], s["op"]
    if op == "momentum":
        z.muon_momentum(s["slices"], 0, s["plan"], s["hp"])
        return {"m": s["m"], "u": s["u"]}
    if op == "orthogonalize":
        z.orthogonalize(s["plan"], s["hp"], ws=s["ws"])
        return {"o": s["o"]}
    if op == "update":
        z.muon_update(s["plan"], s["hp"])
        return {"master": s["master"], "param": s["param"]}
    z.muon_step(s["slices"], 0, s["plan"], s["hp"], ws=s["ws"])
    return {"m": s["m"], "master": s["master"], "param": s["param"]}


# ------------------------------------------------------------------ plain forms
def _momentum(s):
    cols = s["case"]["cols"]
    g = s["grads"][..., :cols].float().sum(0) / s["case"]["W"]
    m = MU * s["m"].float() + g
    s["m"].copy_(m)
    return g + MU * m


def _orthogonal(u, steps):
    """u: [count, rows, cols] in 32 bits."""
    norm = u.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt() + EPS
    x = u / norm.float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(steps):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = A * x + torch.bmm(B * gram + C * torch.bmm(gram, gram), x)
    return x.transpose(1, 2) if tall else x


def _update(s, o):
    p = (s["master"] - (LR * _scale(s["case"])) * o) * (1.0 - LR * DECAY)
    s["master"].copy_(p)
    s["param"].copy_(p)


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "momentum":
        u = _momentum(s)
        s["u"].copy_(u)
        return {"m": s["m"], "u": s["u"]}
    if s["op"] == "orthogonalize":
        s["o"].copy_(_orthogonal(s["u"].float(), s["case"]["steps"]))
        return {"o": s["o"]}
    if s["op"] == "update":
        _update(s, s["o"].float())
        return {"master": s["master"], "param": s["param"]}
    u = _momentum(s).to(s["u"].dtype)           # the momentum is held in u's type between the two
    s["u"].copy_(u)
    _update(s, _orthogonal(u.float(), s["case"]["steps"]))
    return {"m": s["m"], "master": s["master"], "param": s["param"]}


def work(case):
    count, rows, cols = case["count"], case["rows"], case["cols"]
    e, k, n = count * rows * cols, min(rows, cols), max(rows, cols)
    mb, ub = (4 if case.get("m") == "fp32" else 2), (4 if case.get("u") == "fp32" else 2)
    # a step of the iteration: X X^T and A A are symmetric (half of each), B X is not
    ns = float(count) * case.get("steps", 0) * (1.0 * k * k * n + 1.0 * k ** 3 + 2.0 * k * k * n)
    if case["op"] == "momentum":
        return {"bytes": e * (2 * case["W"] + 2 * mb + ub), "flops": e * (case["W"] + 4)}
    if case["op"] == "orthogonalize":
        return {"bytes": e * (ub + 2), "flops": ns}
    if case["op"] == "update":
        return {"bytes": e * 12, "flops": e * 3}
    return {"bytes": e * (2 * case["W"] + 2 * mb + 10), "flops": ns}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, one matrix after the other: with S = X^T X
    (or X X^T, whichever is smaller), a step multiplies X by aI + (bI + cS)S."""
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    out = {}
    if op in ("momentum", "step"):
        mean = torch.zeros(case["count"], case["rows"], case["cols"], dtype=f64, device="cuda")
        for w in range(case["W"]):
            mean += s["grads"][w, :, :, :case["cols"]].to(f64)
        mean /= case["W"]
        m = s["m"].to(f64) * MU + mean
        u = mean + m * MU
        out["m"] = m
        if op == "momentum":
            out["u"] = u
            return out
        u = u.to(_TYPE[case["u"]]).to(f64)      # the step hands the momentum on in u's type
    elif op == "orthogonalize":
        u = s["u"].to(f64)
    if op in ("orthogonalize", "step"):
        o = torch.empty(case["count"], case["rows"], case["cols"], dtype=f64, device="cuda")
        for i in range(case["count"]):
            x = u[i] / (torch.linalg.vector_norm(u[i]) + EPS)
            wide = case["rows"] <= case["cols"]
            eye = torch.eye(min(case["rows"], case["cols"]), dtype=f64, device="cuda")
            for _ in range(case["steps"]):
                g = x @ x.T if wide else x.T @ x
                p = A * eye + (B * eye + C * g) @ g
                x = p @ x if wide else x @ p
            o[i] = x
        if op == "orthogonalize":
            return {"o": o}
    else:
        o = s["o"].to(f64)
    master = s["master"].to(f64) - LR * _scale(case) * o
    master = master - LR * DECAY * master
    out.update(master=master, param=master)
    return out
