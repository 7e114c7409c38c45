"""The Muon step on the GPU.  Momentum and update are bit for bit the fp32
operation sequence of tests/muon_ref.py (and agree with 64 bits to the
roundings counted there); the iteration is compared with its definition in 64
bits, within the first-order bound that muon_ref.iterate_bound derives from the
matrix's singular values, and within the figures the header states."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
import synth
import zero_sharded_mixed_zero1_amd as z
from tests import muon_ref as ref
from tests.gpu_util import assert_bf16_equal, assert_f32_equal, to_dev_u16, to_np_u16, torch_cuda, ws_tensor

pytestmark = pytest.mark.gpu

HP = dict(lr=2e-3, momentum=0.95, weight_decay=0.1)
GUARD = 0x7A5A          # sentinel of the columns beside a matrix


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, dev


class Mats:
    """A plan over matrices of the given (rows, cols), each array of each in a
    buffer of its own: rows of cols + pad elements behind `skew` others, the
    elements beside the matrix holding sentinels."""

    def __init__(self, env, shapes, W=1, pad=0, skew=0, pad_u=0, pad_o=0, m_bf16=False, u_f32=False, in_place=False,
                 seed=1, u=None, flags=0, sigma=1e-2, with_o=True):
        torch, dev = self.torch, self.dev = env
        self.shapes, self.W = shapes, W
        self.m_bf16, self.u_f32, self.in_place = m_bf16, u_f32, in_place
        self.pads = dict(g=pad, param=pad, master=pad, m=pad, u=pad_u, o=pad_u if in_place else pad_o)
        self.skew = skew
        self.scale = [float(np.float32(0.2 * math.sqrt(max(s)))) for s in shapes]
        rng = np.random.default_rng(seed)
        self.offsets, at = [], 3
        for r, c in shapes:
            self.offsets.append(at)
            at += r * (c + pad) + 5
        self.G = [synth.bf16(at, synth.grad_key(seed, 1, w), 0, sigma, 1) for w in range(W)]
        self.grads = [to_dev_u16(torch, g, dev) for g in self.G]
        self.master0 = [rng.standard_normal(s).astype(np.float32) * np.float32(0.02) for s in shapes]
        self.m0 = [rng.standard_normal(s).astype(np.float32) * np.float32(2 * sigma) for s in shapes]
        if m_bf16:
            self.m0 = [ref.widen(ref.bf16(m)).reshape(m.shape) for m in self.m0]
        self.u0 = u if u is not None else [self.matrix(rng, s) for s in shapes]
        self.u0 = [x.astype(np.float32) if u_f32 else ref.widen(ref.bf16(x)).reshape(x.shape) for x in self.u0]
        self.dev_buf = {k: [] for k in ("param", "master", "m", "u", "o")}
        mats = []
        for i, (r, c) in enumerate(shapes):
            self.put("param", i, np.full((r, c), 0x3F80, np.uint16))
            self.put("master", i, self.master0[i])
            self.put("m", i, ref.bf16(self.m0[i]) if m_bf16 else self.m0[i])
            self.put("u", i, self.u0[i] if u_f32 else ref.bf16(self.u0[i]))
            if not in_place:
                self.put("o", i, np.full((r, c), 0x3F80, np.uint16))
            a = {k: self.at(k, i) for k in ("param", "master", "m", "u")}
            o = (a["u"] if in_place else self.at("o", i)) if with_o else None
            mats.append(z.matrix(r, c, ld=c + pad, shard_offset=self.offsets[i], scale=self.scale[i], o=o,
                                 ldu=c + pad_u, ldo=c + self.pads["o"], **a))
        self.mats = mats
        self.flags = (z.MV_BF16 if m_bf16 else 0) | (z.U_F32 if u_f32 else 0)
        self.table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
        self.plan = z.muon_plan(mats, self.table, flags=self.flags)

    @staticmethod
    def matrix(rng, shape, kind=None):
        """A matrix as momentum is: a few strong directions over noise."""
        r, c = shape
        k = min(4, r, c)
        return (rng.standard_normal((r, k)) @ rng.standard_normal((k, c)) * 3 + rng.standard_normal((r, c))) * 1e-3

    def put(self, name, i, a):
        r, c = self.shapes[i]
        pad = self.pads[name]
        wide = a.view(np.uint16) if a.itemsize == 2 else a.view(np.uint32)
        buf = np.full(self.skew + r * (c + pad) + 4, GUARD, wide.dtype)
        buf[self.skew:self.skew + r * (c + pad)].reshape(r, c + pad)[:, :c] = wide
        self.dev_buf[name].append(self.torch.from_numpy(buf.view(np.int16 if wide.itemsize == 2 else np.int32)).to(self.dev))

    def at(self, name, i):
        return self.dev_buf[name][i][self.skew:]

    def get(self, name, i, dtype=None):
        """The matrix's elements; the ones beside it have to be untouched."""
        if name == "o" and self.in_place:
            name = "u"
        r, c = self.shapes[i]
        pad = self.pads[name]
        a = self.dev_buf[name][i].cpu().numpy()
        a = a.view(np.uint16 if a.itemsize == 2 else np.uint32)
        body = a[self.skew:self.skew + r * (c + pad)].reshape(r, c + pad)
        assert (a[:self.skew] == GUARD).all() and (a[self.skew + r * (c + pad):] == GUARD).all(), f"{name}[{i}] guard"
        assert (body[:, c:] == GUARD).all(), f"{name}[{i}]: wrote beside its columns"
        body = np.ascontiguousarray(body[:, :c])
        return body if body.itemsize == 2 else body.view(np.float32)

    def workspace(self, fill=0xFF):
        ws = ws_tensor(self.torch, z.muon_workspace_bytes(self.plan), self.dev)
        ws.fill_(fill)      # NaNs: everything read has to be written first
        return ws

    def g(self, i, average=True, round_bf16=False):
        r, c = self.shapes[i]
        ld = c + self.pads["g"]
        n = (r - 1) * ld + c
        flat = oracle.shard_reduce([x[self.offsets[i]:self.offsets[i] + n] for x in self.G], average=average)
        full = np.zeros(r * ld, np.float32)
        full[:n] = flat
        out = np.ascontiguousarray(full.reshape(r, ld)[:, :c])
        return ref.widen(ref.bf16(out)).reshape(out.shape) if round_bf16 else out


# ------------------------------------------------------------------ momentum
SHAPES = [(1, 1), (1, 3), (3, 1), (2, 5), (7, 4), (64, 64), (33, 130), (130, 33), (1, 5000), (257, 513), (40, 2048)]


@pytest.mark.parametrize("W", [1, 2, 3, 5, 8, 9])
@pytest.mark.parametrize("m_bf16,u_f32", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("pad,skew,pad_u", [(0, 0, 0), (3, 1, 0), (8, 0, 5)])
def test_momentum(env, W, m_bf16, u_f32, pad, skew, pad_u):
    torch, dev = env
    t = Mats(env, SHAPES, W=W, pad=pad, skew=skew, pad_u=pad_u, m_bf16=m_bf16, u_f32=u_f32, seed=10 + W)
    for flags in (0, z.SUM_ONLY, z.NO_NESTEROV, z.G_BF16):
        m_before = [ref.widen(t.get("m", i)) if m_bf16 else t.get("m", i) for i in range(len(SHAPES))]
        z.muon_momentum(t.grads, 0, t.plan, HP, flags=flags)
        torch.cuda.synchronize()
        for i, s in enumerate(SHAPES):
            what = f"{s} W={W} flags={flags}"
            g = t.g(i, average=not flags & z.SUM_ONLY, round_bf16=bool(flags & z.G_BF16))
            m, u = ref.momentum32(g, m_before[i], HP["momentum"], nesterov=not flags & z.NO_NESTEROV)
            (assert_bf16_equal if m_bf16 else assert_f32_equal)(t.get("m", i), ref.bf16(m) if m_bf16 else m, "m " + what)
            (assert_f32_equal if u_f32 else assert_bf16_equal)(t.get("u", i), u if u_f32 else ref.bf16(u), "u " + what)


def test_momentum_against_64_bits(env):
    """fp32 m and u against the formulas in 64 bits.  A sum of W slices rounds
    W - 1 times, its average once, mu (as fp32) and mu m once each, and each
    addition once, every time by 2^-24 of a value that is at most the sum of
    the terms' sizes: (W + 4) of them for m; u takes mu m and an addition
    more, W + 7."""
    torch, dev = env
    for W in (1, 3, 8):
        t = Mats(env, SHAPES, W=W, u_f32=True, seed=77)
        z.muon_momentum(t.grads, 0, t.plan, HP)
        torch.cuda.synchronize()
        for i, (r, c) in enumerate(SHAPES):
            o = t.offsets[i]
            G = [ref.widen(x[o:o + r * c]).astype(np.float64).reshape(r, c) for x in t.G]
            mu, m0 = HP["momentum"], t.m0[i].astype(np.float64)
            g, size = sum(G) / W, sum(np.abs(x) for x in G) / W
            m = mu * m0 + g
            msize = mu * np.abs(m0) + size
            assert (np.abs(t.get("m", i) - m) <= (W + 4) * 2.0 ** -24 * msize + 1e-44).all()
            assert (np.abs(t.get("u", i) - (g + mu * m)) <= (W + 7) * 2.0 ** -24 * (size + mu * msize) + 1e-44).all()


@pytest.mark.parametrize("max_norm,flags", [(0.5, 0), (1e9, 0), (0.5, z.CLIP_EPS), (math.inf, 0)])
def test_momentum_clips_by_the_global_norm(env, max_norm, flags):
    torch, dev = env
    t = Mats(env, [(30, 50), (65, 9)], W=3, seed=5)
    rs = torch.tensor([1.25, 0.5, 2.0], dtype=torch.float64, device=dev)
    info = torch.zeros(4, dtype=torch.float64, device=dev)
    z.muon_momentum(t.grads, 0, t.plan, dict(HP, max_norm=max_norm), rank_sumsq=rs, n_ranks=3, flags=flags, info_out=info)
    torch.cuda.synchronize()
    norm = math.sqrt((1.25 + 0.5) + 2.0)
    raw = info.cpu().numpy()
    coef, clip = raw[2:3].view(np.float32)[0], raw[2:3].view(np.int32)[1]
    assert raw[0] == 3.75 and raw[1] == norm
    c = max_norm / (norm + 1e-6) if flags else max_norm / norm
    assert clip == (1 if max_norm < norm else 0)
    assert coef == (np.float32(c) if clip else np.float32(1.0))
    for i in range(2):
        g = t.g(i) * coef if clip else t.g(i)
        m, u = ref.momentum32(g, t.m0[i], HP["momentum"])
        assert_f32_equal(t.get("m", i), m, "m")
        assert_bf16_equal(t.get("u", i), ref.bf16(u), "u")


def test_momentum_propagates_non_finite_values(env):
    torch, dev = env
    t = Mats(env, [(5, 70)], W=2, seed=8)
    o = t.offsets[0]
    for w, k, bits in ((0, 0, 0x7F80), (1, 9, 0xFF80), (0, 9, 0x7F80), (1, 33, 0x7FC1), (0, 100, 0x7F7F), (1, 100, 0x7F7F)):
        t.G[w][o + k] = bits
    t.grads = [to_dev_u16(torch, g, dev) for g in t.G]
    z.muon_momentum(t.grads, 0, t.plan, HP)
    torch.cuda.synchronize()
    m, u = ref.momentum32(t.g(0), t.m0[0], HP["momentum"])
    assert_f32_equal(t.get("m", 0), m, "m")
    assert_bf16_equal(t.get("u", 0), ref.bf16(u), "u")
    assert np.isinf(m).any() and np.isnan(m).any()


# ------------------------------------------------------------------ update
@pytest.mark.parametrize("pad,skew,pad_o", [(0, 0, 0), (3, 1, 0), (8, 0, 5)])
@pytest.mark.parametrize("flags", [0, z.DECAY_FIRST])
def test_update(env, pad, skew, pad_o, flags):
    torch, dev = env
    t = Mats(env, SHAPES, pad=pad, skew=skew, pad_o=pad_o)
    rng = np.random.default_rng(3)
    O = []
    for i, s in enumerate(SHAPES):
        o = ref.bf16(rng.standard_normal(s).astype(np.float32) / np.float32(math.sqrt(max(s))))
        O.append(o)
        buf = t.dev_buf["o"][i].cpu().numpy()
        body = buf[skew:skew + s[0] * (s[1] + pad_o)].reshape(s[0], s[1] + pad_o)
        body[:, :s[1]] = o.view(np.int16)
        t.dev_buf["o"][i].copy_(torch.from_numpy(buf))
    z.muon_update(t.plan, HP, flags=flags)
    torch.cuda.synchronize()
    for i, s in enumerate(SHAPES):
        exp = ref.update32(t.master0[i], ref.widen(O[i]).reshape(s), HP["lr"], HP["weight_decay"], t.scale[i],
                           decay_first=bool(flags))
        got = t.get("master", i)
        assert_f32_equal(got, exp, f"master {s}")
        assert_bf16_equal(t.get("param", i), ref.bf16(exp), f"param {s}")
        # 64 bits: eta, eta o, the difference, delta and the product round by
        # 2^-24 of their value each
        o = ref.widen(O[i]).reshape(s).astype(np.float64)
        p = t.master0[i].astype(np.float64)
        eta, delta = HP["lr"] * t.scale[i], 1 - HP["lr"] * HP["weight_decay"]
        e64 = p * delta - eta * o if flags else (p - eta * o) * delta
        assert (np.abs(got - e64) <= 6 * 2.0 ** -24 * (np.abs(p) + eta * np.abs(o))).all()


# ------------------------------------------------------------------ orthogonalize
def check_o(t, i, steps=5, coef=(ref.A, ref.B, ref.C), eps=1e-7, what=""):
    o = ref.widen(t.get("o", i)).reshape(t.shapes[i]).astype(np.float64)
    exact = ref.iterate64(t.u0[i], steps, coef, eps)
    bound, size = ref.iterate_bound(t.u0[i], steps, coef, eps)
    off = np.linalg.norm(o - exact)
    assert off <= bound, f"{what} {t.shapes[i]}: off by {off:.3g}, bound {bound:.3g}, |o| {size:.3g}"
    return off / size if size else 0.0


NS_SHAPES = [(1, 1), (1, 2), (2, 1), (2, 2), (3, 7), (1, 300), (300, 1), (16, 16), (17, 31), (64, 64), (63, 200),
             (100, 127), (128, 128), (129, 128), (127, 129), (128, 257), (260, 130), (200, 600), (513, 140), (384, 384)]


@pytest.mark.parametrize("u_f32", [False, True])
@pytest.mark.parametrize("pad_u,pad_o,skew", [(0, 0, 0), (3, 5, 1)])
def test_orthogonalize(env, u_f32, pad_u, pad_o, skew):
    torch, dev = env
    t = Mats(env, NS_SHAPES, pad_u=pad_u, pad_o=pad_o, skew=skew, u_f32=u_f32)
    z.orthogonalize(t.plan, HP, ws=t.workspace())
    torch.cuda.synchronize()
    for i, s in enumerate(NS_SHAPES):
        # the header's figure, before the rounding to bf16 (at most 2^-8 of it)
        assert check_o(t, i) <= 5e-3 + ref.BF16
        u = t.get("u", i)
        assert_f32_equal(u if u_f32 else ref.widen(u), t.u0[i] if u_f32 else t.u0[i].reshape(u.shape), "u is only read")


@pytest.mark.parametrize("kind", ["gauss", "power1", "power2", "rank1", "rank8"])
@pytest.mark.parametrize("shape", [(150, 200), (400, 130)])
def test_orthogonalize_spectra(env, kind, shape):
    """Matrices of every kind of spectrum, those of a few strong directions
    among them: off by at most 0.3 % of the result where it is not yet rounded
    to bf16 (rounding one half of X only would give 2 % and more on these)."""
    torch, dev = env
    rng = np.random.default_rng(17)
    r, c = shape
    k = min(shape)
    if kind == "gauss":
        u = rng.standard_normal(shape)
    else:
        U, _ = np.linalg.qr(rng.standard_normal((r, k)))
        V, _ = np.linalg.qr(rng.standard_normal((c, k)))
        s = np.arange(1, k + 1.0)
        s = {"power1": s ** -1, "power2": s ** -2, "rank1": (s == 1) * 1.0, "rank8": np.where(s <= 8, 1.0, 1e-4)}[kind]
        u = (U * s) @ V.T
    t = Mats(env, [shape], u=[u])
    z.orthogonalize(t.plan, HP, ws=t.workspace())
    torch.cuda.synchronize()
    # two errors that do not know of each other: 0.3 % and a bf16 rounding of
    # at most 2^-8, 1/sqrt(3) of that in the mean square
    assert check_o(t, 0, what=kind) <= math.hypot(3e-3, ref.BF16 / math.sqrt(3))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("coef", [(ref.A, ref.B, ref.C), (1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (1.0, 0.0, 0.0)])
def test_orthogonalize_coefficients(env, steps, coef):
    torch, dev = env
    t = Mats(env, [(90, 140), (140, 90), (1, 5)])
    z.orthogonalize(t.plan, dict(HP, ns_steps=steps, ns_a=coef[0], ns_b=coef[1], ns_c=coef[2]), ws=t.workspace())
    torch.cuda.synchronize()
    for i in range(3):
        check_o(t, i, steps, coef, what=f"{steps} steps of {coef}")


def test_orthogonalize_in_place(env):
    torch, dev = env
    shapes = [(70, 200), (200, 70), (1, 9)]
    a = Mats(env, shapes, pad_u=3, skew=1)
    b = Mats(env, shapes, pad_u=3, skew=1, in_place=True)
    for t in (a, b):
        z.orthogonalize(t.plan, HP, ws=t.workspace())
    torch.cuda.synchronize()
    for i in range(3):
        assert_bf16_equal(b.get("o", i), a.get("o", i), "in place")


def test_orthogonalize_is_the_same_alone_and_again(env):
    """A matrix's result does not depend on the others of its plan, and a rerun
    on another workspace gives the same bits."""
    torch, dev = env
    shapes = [(60, 300), (129, 500), (500, 129), (5, 5)]
    t = Mats(env, shapes)
    first = []
    for run in range(2):
        z.orthogonalize(t.plan, HP, ws=t.workspace(fill=run * 0x55))
        torch.cuda.synchronize()
        got = [t.get("o", i) for i in range(4)]
        first = first or got
        for i in range(4):
            assert_bf16_equal(got[i], first[i], "again")
    for i in range(4):
        one = Mats(env, [shapes[i]], u=[t.u0[i]])
        z.orthogonalize(one.plan, HP, ws=one.workspace())
        torch.cuda.synchronize()
        assert_bf16_equal(one.get("o", 0), first[i], "alone")


def test_orthogonalize_non_finite_and_extreme_sizes(env):
    """A matrix with an infinity or a NaN becomes NaN throughout, a zero matrix
    zero; the sizes at the ends of the type's range (whose squares do not fit
    fp32) are matrices like others; neighbours are not touched by any of it."""
    torch, dev = env
    rng = np.random.default_rng(9)
    base = rng.standard_normal((40, 150))
    us = [base.copy() for _ in range(9)]
    us[1][3, 7] = np.inf
    us[2][39, 149] = np.nan
    us[3][:] = 0.0
    us[4] *= 1e36
    us[5] *= 1e-36
    us[6] *= 0.0
    us[6][20, 100] = -3e38
    us[7][1, 1], us[7][2, 2] = np.inf, -np.inf
    for u_f32 in (False, True):
        t = Mats(env, [b.shape for b in us], u=[u.astype(np.float32) for u in us], u_f32=u_f32)
        z.orthogonalize(t.plan, dict(HP, ns_eps=0.0), ws=t.workspace())
        torch.cuda.synchronize()
        o = [ref.widen(t.get("o", i)) for i in range(9)]
        for i in (1, 2, 3, 7):      # 0 / 0 with eps = 0
            assert np.isnan(o[i]).all(), i
        for i in (0, 4, 5, 6, 8):
            check_o(t, i, eps=0.0, what=f"matrix {i}")
        assert_f32_equal(o[8], o[0], "the same matrix")
        z.orthogonalize(t.plan, HP, ws=t.workspace())
        torch.cuda.synchronize()
        assert (t.get("o", 3) == 0).all()               # 0 / eps
        check_o(t, 5, eps=1e-7, what="much smaller than eps")


def test_subnormal_matrix(env):
    torch, dev = env
    u = np.random.default_rng(2).standard_normal((20, 33)) * 1e-40
    t = Mats(env, [(20, 33)], u=[u], u_f32=True)
    z.orthogonalize(t.plan, dict(HP, ns_eps=0.0), ws=t.workspace())
    torch.cuda.synchronize()
    check_o(t, 0, eps=0.0)


def test_groups_of_matrices(env):
    """More matrices than one group of the workspace holds: the workspace stays
    within a group's size, and every group's results are right."""
    torch, dev = env
    rng = np.random.default_rng(4)
    shapes = [(2050, 2100)] * 14 + [(20, 30)] * 3
    us = [Mats.matrix(rng, shapes[0]).astype(np.float32), Mats.matrix(rng, shapes[-1]).astype(np.float32)]
    u = [us[0] * np.float32(1 + i) for i in range(14)] + [us[1]] * 3
    t = Mats(env, shapes, u=u, sigma=1e-2)
    assert t.plan.n_groups >= 2
    assert z.muon_workspace_bytes(t.plan) < (600 << 20)
    z.orthogonalize(t.plan, HP, ws=t.workspace())
    torch.cuda.synchronize()
    for i in range(14):
        x = torch.from_numpy(t.u0[i]).to(dev).double()      # the iteration in 64 bits, on the GPU for its size
        x = x / (torch.linalg.vector_norm(x) + 1e-7)
        for _ in range(5):
            s = x @ x.T
            x = ref.A * x + (ref.B * s + ref.C * (s @ s)) @ x
        o = torch.from_numpy(ref.widen(t.get("o", i))).to(dev).double()
        off, size = float(torch.linalg.vector_norm(o - x)), float(torch.linalg.vector_norm(x))
        assert off <= math.hypot(3e-3, ref.BF16) * size, (i, off, size)
    for i in range(14, 17):
        check_o(t, i)


# ------------------------------------------------------------------ together
def expect_step(t, i, flags=0, hp=HP, m_before=None):
    """m, u as the momentum gives them; the update from the iteration in 64 bits."""
    m0 = m_before if m_before is not None else t.m0[i]
    m, u = ref.momentum32(t.g(i), m0, hp["momentum"], nesterov=not flags & z.NO_NESTEROV)
    return m, u


def check_step(t, i, master_before, m_before, hp=HP, flags=0):
    torch = t.torch
    m, u = expect_step(t, i, flags, hp, m_before)
    (assert_bf16_equal if t.m_bf16 else assert_f32_equal)(t.get("m", i), ref.bf16(m) if t.m_bf16 else m, "m")
    uh = u if t.u_f32 else ref.widen(ref.bf16(u)).reshape(u.shape)
    (assert_f32_equal if t.u_f32 else assert_bf16_equal)(t.get("u", i), u if t.u_f32 else ref.bf16(u), "u")
    exact = ref.iterate64(uh)
    bound, size = ref.iterate_bound(uh)
    eta, delta = hp["lr"] * t.scale[i], 1 - hp["lr"] * hp["weight_decay"]
    p = master_before.astype(np.float64)
    want = p * delta - eta * exact if flags & z.DECAY_FIRST else (p - eta * exact) * delta
    got = t.get("master", i)
    # the update's own roundings, 6 * 2^-24 of the terms, and eta times o's
    room = 6 * 2.0 ** -24 * (np.linalg.norm(p) + eta * size) + eta * bound
    assert np.linalg.norm(got - want) <= room, (t.shapes[i], np.linalg.norm(got - want), room)
    assert_bf16_equal(t.get("param", i), ref.bf16(got), "param")


STEP_SHAPES = [(1, 1), (5, 300), (300, 5), (64, 64), (130, 400), (400, 130), (128, 256)]


@pytest.mark.parametrize("W,m_bf16,u_f32,pad,skew,pad_u,flags", [
    (1, False, False, 0, 0, 0, 0), (8, False, False, 0, 0, 0, 0), (3, True, False, 3, 1, 2, 0),
    (4, False, True, 8, 0, 0, z.DECAY_FIRST), (2, True, True, 0, 0, 0, z.NO_NESTEROV)])
def test_step(env, W, m_bf16, u_f32, pad, skew, pad_u, flags):
    """Three steps in a row, the gradients the same: each against the formulas
    from the state that it found."""
    torch, dev = env
    t = Mats(env, STEP_SHAPES, W=W, m_bf16=m_bf16, u_f32=u_f32, pad=pad, skew=skew, pad_u=pad_u, with_o=False, seed=30 + W)
    ws = t.workspace()
    n = len(STEP_SHAPES)
    for _ in range(3):
        master = [t.get("master", i) for i in range(n)]
        m = [ref.widen(t.get("m", i)).reshape(STEP_SHAPES[i]) if m_bf16 else t.get("m", i) for i in range(n)]
        z.muon_step(t.grads, 0, t.plan, HP, flags=flags, ws=ws)
        torch.cuda.synchronize()
        for i in range(n):
            check_step(t, i, master[i], m[i], flags=flags)


def test_step_equals_its_three_calls_but_for_o(env):
    """The step's master is the three calls' to the rounding of o to bf16."""
    torch, dev = env
    shapes = [(130, 260), (260, 130)]
    a, b = Mats(env, shapes, W=2, seed=3), Mats(env, shapes, W=2, seed=3)
    z.muon_step(a.grads, 0, a.plan, HP, ws=a.workspace())
    z.muon_momentum(b.grads, 0, b.plan, HP)
    z.orthogonalize(b.plan, HP, ws=b.workspace())
    z.muon_update(b.plan, HP)
    torch.cuda.synchronize()
    for i in range(2):
        assert_f32_equal(a.get("m", i), b.get("m", i), "m")
        assert_bf16_equal(a.get("u", i), b.get("u", i), "u")
        o = np.abs(ref.widen(b.get("o", i)).astype(np.float64))
        eta = HP["lr"] * a.scale[i]
        room = eta * 2 * ref.BF16 * o + 4 * 2.0 ** -24 * (np.abs(a.master0[i]) + eta * o)
        assert (np.abs(a.get("master", i).astype(np.float64) - b.get("master", i)) <= room).all()


def test_begin_offsets_the_gradients(env):
    torch, dev = env
    a, b = Mats(env, [(20, 30)], W=2, seed=6), Mats(env, [(20, 30)], W=2, seed=6)
    moved = [torch.cat([torch.full((11,), 0x4000, dtype=torch.int16, device=dev), g]) for g in b.grads]
    z.muon_momentum(a.grads, 0, a.plan, HP)
    z.muon_momentum(moved, 11, b.plan, HP)
    torch.cuda.synchronize()
    assert_f32_equal(b.get("m", 0), a.get("m", 0), "m")


def test_captured_step_replays(env):
    """Two steps with workspaces of their own captured into two graphs, their
    scalars in device memory, replayed with eager steps of a third set of
    matrices between: every replay equals the eager step bit for bit."""
    torch, dev = env
    shapes = [(130, 300), (64, 64), (300, 140)]
    sets = [Mats(env, shapes, W=3, seed=12) for _ in range(3)]
    ws = [t.workspace() for t in sets]
    scal = torch.zeros(6, dtype=torch.int32, device=dev)
    def set_scalars(hp):
        raw = np.frombuffer(bytes(z.muon_scalars_derive(hp)), np.int32)
        scal.copy_(torch.from_numpy(raw.copy()))
    def step(k, hp):
        z.muon_step(sets[k].grads, 0, sets[k].plan, hp, ws=ws[k])
    set_scalars(HP)
    for k in range(3):
        step(k, HP)
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(k, dict(device_scalars=scal))
        graphs.append(g)
    torch.cuda.synchronize()
    other = torch.ones(1 << 20, device=dev)
    for it in range(4):
        hp = dict(lr=1e-3 * (it + 1), momentum=0.9 + 0.02 * it, weight_decay=0.05 * it)
        set_scalars(hp)
        step(2, hp)
        for g in graphs:
            g.replay()
        other.mul_(1.0001).add_(1.0)
        torch.cuda.synchronize()
        for i in range(3):
            for k in range(2):
                assert_f32_equal(sets[k].get("master", i), sets[2].get("master", i), f"replay {it} graph {k}")
                assert_f32_equal(sets[k].get("m", i), sets[2].get("m", i), f"replay {it} graph {k}")
                assert_bf16_equal(sets[k].get("param", i), sets[2].get("param", i), f"replay {it} graph {k}")


def test_two_streams_with_their_own_workspaces(env):
    torch, dev = env
    shapes = [(260, 520), (520, 260)]
    a, b, c = (Mats(env, shapes, W=2, seed=s) for s in (21, 22, 21))
    z.muon_step(c.grads, 0, c.plan, HP, ws=c.workspace())
    wa, wb = a.workspace(), b.workspace()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    z.muon_step(a.grads, 0, a.plan, HP, ws=wa, stream=s1)
    z.muon_step(b.grads, 0, b.plan, HP, ws=wb, stream=s2)
    torch.cuda.synchronize()
    for i in range(2):
        assert_f32_equal(a.get("master", i), c.get("master", i), "two streams")
        check_step(b, i, b.master0[i], b.m0[i])


def test_plan_of_another_device_is_refused(env):
    torch, dev = env
    t = Mats(env, [(4, 5)])
    t.plan.device = 5
    for call in (lambda: z.muon_momentum(t.grads, 0, t.plan, HP), lambda: z.muon_update(t.plan, HP),
                 lambda: z.orthogonalize(t.plan, HP, ws=t.workspace()),
                 lambda: z.muon_step(t.grads, 0, t.plan, HP, ws=t.workspace())):
        with pytest.raises(z.Zero1Error) as e:
            call()
        assert e.value.name == "ZERO1_EINVAL" and "device 5" in e.value.message


def test_column_blocks_of_one_parameter(env):
    """The three square blocks of a fused [d, 3 d] weight, orthogonalised apart:
    one array of each kind, a common stride, nothing between them disturbed."""
    torch, dev = env
    d, W = 96, 2
    rng = np.random.default_rng(40)
    G = [synth.bf16(3 * d * d, synth.grad_key(41, 1, w), 0, 1e-2, 1) for w in range(W)]
    master = (rng.standard_normal((d, 3 * d)) * 0.02).astype(np.float32)
    grads = [to_dev_u16(torch, g, dev) for g in G]
    dm = torch.from_numpy(master.copy()).to(dev)
    mom = torch.zeros_like(dm)
    par = torch.zeros(d, 3 * d, dtype=torch.int16, device=dev)
    u = torch.zeros(d, 3 * d, dtype=torch.int16, device=dev)
    mats = [z.matrix(d, d, ld=3 * d, shard_offset=k * d, scale=1.0, param=par[:, k * d:], master=dm[:, k * d:],
                     m=mom[:, k * d:], u=u[:, k * d:], ldu=3 * d) for k in range(3)]
    table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
    plan = z.muon_plan(mats, table)
    z.muon_step(grads, 0, plan, HP, ws=ws_tensor(torch, z.muon_workspace_bytes(plan), dev))
    torch.cuda.synchronize()
    g = oracle.shard_reduce(G).reshape(d, 3 * d)
    m, uu = ref.momentum32(g, np.zeros_like(g), HP["momentum"])
    assert_f32_equal(mom.cpu().numpy(), m, "m")
    uh = ref.widen(ref.bf16(uu)).reshape(d, 3 * d)
    for k in range(3):
        blk = slice(k * d, (k + 1) * d)
        exact = ref.iterate64(uh[:, blk])
        bound, size = ref.iterate_bound(uh[:, blk])
        eta, delta = HP["lr"], 1 - HP["lr"] * HP["weight_decay"]
        want = (master[:, blk].astype(np.float64) - eta * exact) * delta
        room = 6 * 2.0 ** -24 * (np.linalg.norm(master[:, blk]) + eta * size) + eta * bound
        assert np.linalg.norm(dm.cpu().numpy()[:, blk] - want) <= room
    assert_bf16_equal(to_np_u16(par), ref.bf16(dm.cpu().numpy()), "param")


# ------------------------------------------------------------------ o before its rounding
class Steps:
    """Matrices u (fp32, each entry the exact sum of two bf16 slices) whose o
    muon_step leaves in the master unrounded: momentum and master are zero, lr
    and scale 1, so m = u = g and p = 0 - o."""

    def __init__(self, env, us, u_f32):
        torch, dev = self.torch, self.dev = env
        self.hi = [ref.bf16(u.astype(np.float32)).reshape(u.shape) for u in us]
        self.u = [ref.widen(h).reshape(h.shape) for h in self.hi]
        parts = [self.hi]
        if u_f32:
            lo = [ref.bf16(u.astype(np.float32) - w).reshape(u.shape) for u, w in zip(us, self.u)]
            self.u = [w + ref.widen(x).reshape(x.shape) for w, x in zip(self.u, lo)]
            parts.append(lo)
        self.grads = [to_dev_u16(torch, np.concatenate([h.ravel() for h in p]), dev) for p in parts]
        self.bufs, mats, at = [], [], 0
        for u in us:
            b = dict(param=torch.zeros(u.shape, dtype=torch.int16, device=dev), master=torch.zeros(u.shape, device=dev),
                     m=torch.zeros(u.shape, device=dev),
                     u=torch.zeros(u.shape, dtype=torch.float32 if u_f32 else torch.int16, device=dev))
            self.bufs.append(b)
            mats.append(z.matrix(*u.shape, shard_offset=at, **b))
            at += u.size
        self.table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
        self.plan = z.muon_plan(mats, self.table, flags=z.U_F32 if u_f32 else 0)
        self.ws = ws_tensor(torch, z.muon_workspace_bytes(self.plan), dev)

    def o(self, steps, coef=(ref.A, ref.B, ref.C), eps=1e-7):
        for b in self.bufs:
            b["master"].zero_()
            b["m"].zero_()
        self.ws.fill_(0xFF)
        hp = dict(lr=1.0, momentum=0.5, weight_decay=0.0, ns_steps=steps, ns_a=coef[0], ns_b=coef[1], ns_c=coef[2],
                  ns_eps=eps)
        z.muon_step(self.grads, 0, self.plan, hp, flags=z.NO_NESTEROV | z.SUM_ONLY, ws=self.ws)
        self.torch.cuda.synchronize()
        return [-b["master"].cpu().numpy().astype(np.float64) for b in self.bufs]


def spectrum(rng, shape, kind):
    r, c = shape
    k = min(shape)
    if kind == "gauss":
        return rng.standard_normal(shape) * 1e-3
    U, _ = np.linalg.qr(rng.standard_normal((r, k)))
    V, _ = np.linalg.qr(rng.standard_normal((c, k)))
    s = np.arange(1, k + 1.0)
    return (U * (s ** -1 if kind == "power" else np.where(s <= 4, 1.0, 1e-3))) @ V.T


EDGE_SHAPES = [(32, 200), (33, 200), (200, 33), (64, 255), (64, 256), (64, 257), (257, 64), (65, 65), (128, 300), (300, 128),
               (128, 128), (129, 300), (3, 1000), (1000, 3), (1, 700), (700, 2), (20, 5000), (5000, 100), (127, 4200)]


@pytest.mark.parametrize("u_f32", [False, True])
@pytest.mark.parametrize("kind", ["gauss", "power", "low"])
def test_o_before_rounding(env, kind, u_f32):
    """Around every size where the path changes (32, 64 and 128 rows; 256
    columns; one part of the gram sum or several; one segment of steps or two):
    within the first-order bound without the last rounding, and where the
    smaller side is at most 128 within the header's 0.05 % of a segment of
    five default steps."""
    rng = np.random.default_rng(77)
    t = Steps(env, [spectrum(rng, s, kind) for s in EDGE_SHAPES], u_f32)
    for steps in (1, 2, 5, 8):
        for got, u in zip(t.o(steps), t.u):
            exact = ref.iterate64(u, steps)
            bound, size = ref.iterate_bound(u, steps)
            off = np.linalg.norm(got - exact)
            what = (u.shape, steps, off / size)
            assert off <= (bound - ref.BF16 * size) / (1 + ref.BF16), what
            if min(u.shape) <= 128 and steps <= 5:
                assert off <= 5e-4 * size, what


@pytest.mark.parametrize("coef,steps", [((1.5, -0.5, 0.0), 20), ((1.5, -0.5, 0.0), 64), ((1.875, -1.25, 0.375), 16)])
def test_many_steps_converge(env, coef, steps):
    """Coefficients that converge (p(1) = 1, p'(1) = 0): after enough steps every
    singular value is 1 whatever the roundings before, so o is U V^T.  What stays
    are the last steps' own roundings, which the bound counts."""
    rng = np.random.default_rng(5)
    us = [spectrum(rng, s, "gauss") for s in [(20, 90), (90, 20), (60, 300), (100, 700), (150, 400)]]
    t = Steps(env, us, True)
    for got, u in zip(t.o(steps, coef), t.u):
        exact = ref.iterate64(u, steps, coef)
        bound, size = ref.iterate_bound(u, steps, coef)
        off = np.linalg.norm(got - exact)
        assert off <= (bound - ref.BF16 * size) / (1 + ref.BF16), (u.shape, off / size, bound / size)


def test_zero_matrices_and_tiny_eps(env):
    """0 / (0 + eps) is zero for every eps > 0, however small, on every path."""
    shapes = [(5, 9), (50, 60), (40, 700), (100, 300), (150, 200)]
    t = Steps(env, [np.zeros(s) for s in shapes], True)
    for eps in (1e-7, 1e-20, 1e-200, 1e-308):
        for o in t.o(5, eps=eps):
            assert (o == 0.0).all(), (eps, o.shape)
    for o in t.o(5, eps=0.0):
        assert np.isnan(o).all(), o.shape


def test_plan_of_every_path_equals_each_alone(env):
    """Dense matrices and thin ones of every class in one plan: each has the bits
    that it has in a plan of its own."""
    rng = np.random.default_rng(8)
    us = [spectrum(rng, s, "gauss") for s in EDGE_SHAPES + [(400, 500), (260, 1300)]]
    for u_f32 in (False, True):
        t = Steps(env, us, u_f32)
        assert t.plan.n_groups >= 4 and t.plan.n_dense == 3
        for steps in (5, 7):
            together = t.o(steps)
            for i, u in enumerate(us):
                alone = Steps(env, [u], u_f32).o(steps)[0]
                assert np.array_equal(alone, together[i]), (u.shape, steps)


# ------------------------------------------------------------------ the ends of the range
@pytest.mark.parametrize("W", [16, 127, 128])
def test_momentum_of_many_slices(env, W):
    torch, dev = env
    t = Mats(env, [(33, 130), (7, 2), (40, 300)], W=W, pad=1, skew=1, seed=W)
    z.muon_momentum(t.grads, 0, t.plan, HP)
    torch.cuda.synchronize()
    for i in range(3):
        m, u = ref.momentum32(t.g(i), t.m0[i], HP["momentum"])
        assert_f32_equal(t.get("m", i), m, f"m {i}")
        assert_bf16_equal(t.get("u", i), ref.bf16(u), f"u {i}")


def test_rows_shorter_than_four(env):
    """Tall matrices of one to three columns, contiguous and cut out of wider
    rows: every call on them."""
    torch, dev = env
    shapes = [(3000, 1), (1000, 2), (2049, 3), (5, 3)]
    for pad, W in ((0, 2), (2, 2), (1, 3), (5, 9)):
        t = Mats(env, shapes, W=W, pad=pad, pad_u=pad, pad_o=2 * pad, skew=1)
        ws = t.workspace()
        z.muon_momentum(t.grads, 0, t.plan, HP)
        z.orthogonalize(t.plan, HP, ws=ws)
        z.muon_update(t.plan, HP)
        torch.cuda.synchronize()
        for i, s in enumerate(shapes):
            m, u = ref.momentum32(t.g(i), t.m0[i], HP["momentum"])
            assert_f32_equal(t.get("m", i), m, f"m {s}")
            assert_bf16_equal(t.get("u", i), ref.bf16(u), f"u {s}")
            t.u0[i] = ref.widen(ref.bf16(u)).reshape(s)
            check_o(t, i)
            o = ref.widen(t.get("o", i)).reshape(s)
            p = ref.update32(t.master0[i], o, HP["lr"], HP["weight_decay"], t.scale[i])
            assert_f32_equal(t.get("master", i), p, f"master {s}")
            assert_bf16_equal(t.get("param", i), ref.bf16(p), f"param {s}")
        b = Mats(env, shapes, W=W, pad=pad, pad_u=pad, skew=1, with_o=False)
        z.muon_step(b.grads, 0, b.plan, HP, ws=b.workspace())
        torch.cuda.synchronize()
        for i in range(len(shapes)):
            check_step(b, i, b.master0[i], b.m0[i])


@pytest.mark.parametrize("W", [2, 3])
def test_more_tiles_than_workgroups(env, W):
    """A plan of more than 8192 tiles, which the workgroups walk in one part per
    XCD: an odd matrix, a flat one and short rows, bit for bit (the fp32
    operations of the contract, one torch operation each)."""
    torch, dev = env
    gen = torch.Generator(device=dev).manual_seed(3)
    shapes, pads = [(3001, 5003), (1024, 2048), (40001, 3)], [2, 0, 1]
    total = sum(r * (c + p) for (r, c), p in zip(shapes, pads))
    grads = [(torch.randn(total, generator=gen, device=dev) * 1e-2).bfloat16() for _ in range(W)]
    mats, state, at = [], [], 0
    for (r, c), p in zip(shapes, pads):
        ld = c + p
        def arr(dtype):
            return (torch.randn(r, ld, generator=gen, device=dev) * 1e-2).to(dtype)
        b = dict(param=arr(torch.bfloat16), master=arr(torch.float32), m=arr(torch.float32), u=arr(torch.bfloat16),
                 o=arr(torch.bfloat16))
        state.append((at, c, ld, b, {k: v.clone() for k, v in b.items()}))
        mats.append(z.matrix(r, c, ld=ld, ldu=ld, ldo=ld, shard_offset=at, scale=0.5, **b))
        at += r * ld
    table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
    plan = z.muon_plan(mats, table)
    assert plan.n_tiles > 8192
    z.muon_momentum(grads, 0, plan, HP)
    z.muon_update(plan, HP)
    torch.cuda.synchronize()
    mu = torch.tensor(HP["momentum"], dtype=torch.float32, device=dev)
    eta = torch.tensor(float(np.float32(HP["lr"]) * np.float32(0.5)), dtype=torch.float32, device=dev)
    delta = torch.tensor(1.0 - HP["lr"] * HP["weight_decay"], dtype=torch.float32, device=dev)
    for at, c, ld, b, old in state:
        n = b["m"].shape[0] * ld
        g = grads[0][at:at + n].float()
        for w in range(1, W):
            g = g + grads[w][at:at + n].float()
        g = (g / torch.tensor(float(W), device=dev)).reshape(-1, ld)   # (a true division)
        m = mu * old["m"] + g
        u = g + mu * m
        p = (old["master"] - eta * old["o"].float()) * delta
        for name, want in (("m", m), ("u", u.bfloat16()), ("master", p), ("param", p.bfloat16())):
            assert torch.equal(b[name][:, :c], want[:, :c]), (name, c)
            assert torch.equal(b[name][:, c:], old[name][:, c:]), (name, c, "beside the columns")


@pytest.mark.parametrize("rows,cols,ld", [(5, 200, (1 << 30) + 1), (140, 130, (1 << 25) + 3), (300, 60, (1 << 24) + 5)])
def test_offsets_past_32_bits(env, rows, cols, ld):
    """Rows so far apart that the last ones lie past 2^32 elements of every
    array, gradients at a `begin` beyond that as well."""
    torch, dev = env
    n = (rows - 1) * ld + cols
    assert n > 1 << 32
    rng = np.random.default_rng(2)
    begin = 7
    def strided(dtype, values):
        flat = torch.empty(n + begin, dtype=dtype, device=dev)
        view = torch.as_strided(flat, (rows, cols), (ld, 1), begin)
        view.copy_(torch.from_numpy(values))
        return flat, view
    G = synth.bf16(rows * cols, synth.grad_key(4, 1, 0), 0, 1e-2, 1).reshape(rows, cols)
    m0 = rng.standard_normal((rows, cols)).astype(np.float32) * np.float32(1e-2)
    p0 = rng.standard_normal((rows, cols)).astype(np.float32) * np.float32(2e-2)
    zero = np.zeros((rows, cols), np.int16)
    g, _ = strided(torch.int16, G.view(np.int16))
    m, mv = strided(torch.float32, m0)
    p, pv = strided(torch.float32, p0)
    bufs = {k: strided(torch.int16, zero) for k in ("param", "u", "o")}
    def plan_of(**kw):
        mats = [z.matrix(rows, cols, ld=ld, ldu=ld, ldo=ld, scale=0.3, param=bufs["param"][0][begin:], master=p[begin:],
                         m=m[begin:], u=bufs["u"][0][begin:], **kw)]
        table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
        plan = z.muon_plan(mats, table)
        return plan, table, ws_tensor(torch, z.muon_workspace_bytes(plan), dev)
    plan, table, ws = plan_of(o=bufs["o"][0][begin:])
    z.muon_momentum([g], begin, plan, HP)
    z.orthogonalize(plan, HP, ws=ws)
    z.muon_update(plan, HP)
    torch.cuda.synchronize()
    me, ue = ref.momentum32(ref.widen(G).reshape(rows, cols), m0, HP["momentum"])
    assert_f32_equal(mv.cpu().numpy(), me, "m")
    u = bufs["u"][1].cpu().numpy().view(np.uint16)
    assert_bf16_equal(u, ref.bf16(ue), "u")
    u = ref.widen(u).reshape(rows, cols)
    o = ref.widen(bufs["o"][1].cpu().numpy().view(np.uint16)).reshape(rows, cols)
    bound, size = ref.iterate_bound(u)
    exact = ref.iterate64(u)
    assert np.linalg.norm(o - exact) <= bound
    pe = ref.update32(p0, o, HP["lr"], HP["weight_decay"], 0.3)
    assert_f32_equal(pv.cpu().numpy(), pe, "master")
    assert_bf16_equal(bufs["param"][1].cpu().numpy().view(np.uint16), ref.bf16(pe), "param")
    # the step in one call, from the first state
    mv.copy_(torch.from_numpy(m0))
    pv.copy_(torch.from_numpy(p0))
    z.muon_step([g], begin, plan, HP, ws=ws)
    torch.cuda.synchronize()
    assert_f32_equal(mv.cpu().numpy(), me, "m of the step")
    eta, delta = HP["lr"] * 0.3, 1 - HP["lr"] * HP["weight_decay"]
    want = (p0.astype(np.float64) - eta * exact) * delta
    # eta's own rounding is one of the six counted
    room = 6 * 2.0 ** -24 * (np.linalg.norm(p0) + eta * size) + eta * bound
    assert np.linalg.norm(pv.cpu().numpy() - want) <= room
    del plan, table, ws, g, m, mv, p, pv, bufs
    torch.cuda.empty_cache()


def test_captured_clip_reads_its_device_scalars(env):
    """A captured step that clips by the max_norm of its device scalars, the sum
    of squares formed by the library's own reduction in the same graph: every
    replay equals the eager step with that max_norm."""
    torch, dev = env
    shapes = [(130, 300), (40, 64)]
    a, b = Mats(env, shapes, W=2, seed=51), Mats(env, shapes, W=2, seed=51)
    wa, wb = a.workspace(), b.workspace()
    n = a.G[0].size
    sumsq = torch.zeros(1, dtype=torch.float64, device=dev)
    rws = ws_tensor(torch, z.workspace_bytes(n, 2), dev)
    z.shard_reduce(b.grads, 0, n, sumsq_out=sumsq, ws=rws)
    torch.cuda.synchronize()
    norm = math.sqrt(float(sumsq[0]))
    scal = torch.zeros(6, dtype=torch.int32, device=dev)
    def set_scalars(hp):
        scal.copy_(torch.from_numpy(np.frombuffer(bytes(z.muon_scalars_derive(hp)), np.int32).copy()))
    first = dict(HP, max_norm=0.5 * norm)
    set_scalars(first)
    for t, ws in ((a, wa), (b, wb)):
        z.muon_step(t.grads, 0, t.plan, first, rank_sumsq=sumsq, n_ranks=1, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z.shard_reduce(a.grads, 0, n, sumsq_out=sumsq, ws=rws)
        z.muon_step(a.grads, 0, a.plan, dict(device_scalars=scal), rank_sumsq=sumsq, n_ranks=1, ws=wa)
    results = []
    for f in (0.25, 2.0, 0.75):
        hp = dict(HP, max_norm=f * norm)
        set_scalars(hp)
        g.replay()
        torch.cuda.synchronize()
        z.muon_step(b.grads, 0, b.plan, hp, rank_sumsq=sumsq, n_ranks=1, ws=wb)
        torch.cuda.synchronize()
        for i in range(2):
            assert_f32_equal(a.get("master", i), b.get("master", i), f"master, {f}")
            assert_f32_equal(a.get("m", i), b.get("m", i), f"m, {f}")
            assert_bf16_equal(a.get("u", i), b.get("u", i), f"u, {f}")
        results.append(a.get("u", 0).copy())
    assert not np.array_equal(results[0], results[1])


@pytest.mark.parametrize("rows,cols,count,tiles", [(4090, 4101, 1, (1, 1)), (5103, 5003, 1, (2, 2)), (4099, 2051, 3, (0, 2)),
                                                   (1111, 2501, 3, (0, 1))])
def test_every_tile_shape(env, rows, cols, count, tiles):
    """Sizes that take the larger tiles of the products, ragged against all of them,
    cut out of wider arrays: the iteration in 64 bits (on the GPU for its size),
    o's neighbours untouched, a captured replay the same bits, and the update in
    the last product's epilogue."""
    torch, dev = env
    gen = torch.Generator(device=dev).manual_seed(7)
    ld, ldo = cols + 3, cols + 5
    u = torch.zeros(count, rows, ld, dtype=torch.bfloat16, device=dev)
    o = torch.full((count, rows, ldo), 7.0, dtype=torch.bfloat16, device=dev)
    for k in range(count):
        low = torch.randn(rows, 8, generator=gen, device=dev) @ torch.randn(8, cols, generator=gen, device=dev)
        u[k, :, :cols] = ((3 * low + torch.randn(rows, cols, generator=gen, device=dev)) * 1e-3).bfloat16()
    mats = [z.matrix(rows, cols, u=u[k], ldu=ld, o=o[k], ldo=ldo) for k in range(count)]
    table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
    plan = z.muon_plan(mats, table)
    assert (plan.groups[0].sym_tile, plan.groups[0].full_tile) == tiles and plan.n_groups == 1
    ws = ws_tensor(torch, z.muon_workspace_bytes(plan), dev)
    ws.fill_(0xFF)
    z.orthogonalize(plan, HP, ws=ws)
    torch.cuda.synchronize()
    assert (o[:, :, cols:] == 7.0).all()
    exact = []
    for k in range(count):
        x = u[k, :, :cols].double()
        x = x / (torch.linalg.vector_norm(x) + 1e-7)
        for _ in range(5):
            if rows <= cols:
                s = x @ x.T
                x = ref.A * x + (ref.B * s + ref.C * (s @ s)) @ x
            else:
                s = x.T @ x
                x = ref.A * x + x @ (ref.B * s + ref.C * (s @ s))
        off, size = (float(torch.linalg.vector_norm(v)) for v in (o[k, :, :cols].double() - x, x))
        assert off <= math.hypot(3e-3, ref.BF16) * size, (k, off / size)
        exact.append(x)
    first = o.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z.orthogonalize(plan, HP, ws=ws)
    for _ in range(2):
        o.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[:, :, :cols], first[:, :, :cols])
    # the step: u = g of one slice, so that its o is the same but for the rounding
    mom, master = torch.zeros(count, rows, ld, device=dev), torch.zeros(count, rows, ld, device=dev)
    param = torch.full((count, rows, ld), 7.0, dtype=torch.bfloat16, device=dev)
    u2 = torch.zeros_like(u)
    mats = [z.matrix(rows, cols, ld=ld, shard_offset=k * rows * ld, param=param[k], master=master[k], m=mom[k], u=u2[k],
                     ldu=ld) for k in range(count)]
    table2 = ws_tensor(torch, z.muon_table_bytes(mats), dev)
    plan2 = z.muon_plan(mats, table2)
    z.muon_step([u], 0, plan2, dict(lr=1.0, momentum=0.5, weight_decay=0.0), flags=z.NO_NESTEROV, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(u2, u)
    assert (param[:, :, cols:] == 7.0).all() and (master[:, :, cols:] == 0).all()
    assert torch.equal(param[:, :, :cols], master[:, :, :cols].bfloat16())
    for k in range(count):
        off = float(torch.linalg.vector_norm(-master[k, :, :cols].double() - exact[k]))
        assert off <= 3e-3 * float(torch.linalg.vector_norm(exact[k])), k
        # and is what orthogonalize rounds
        assert torch.equal((-master[k, :, :cols]).bfloat16(), first[k, :, :cols])


@pytest.mark.parametrize("steps", [1, 5, 7])
def test_in_place_on_every_path(env, steps):
    """o in place of u: thin matrices of one part and of several, in one segment of
    steps and in two, wide and tall, and others."""
    torch, dev = env
    shapes = [(30, 40), (64, 250), (250, 64), (100, 1001), (1001, 100), (3, 700), (200, 600), (601, 203)]
    a = Mats(env, shapes, pad_u=3, skew=1)
    b = Mats(env, shapes, pad_u=3, skew=1, in_place=True)
    for t in (a, b):
        z.orthogonalize(t.plan, dict(HP, ns_steps=steps), ws=t.workspace())
    torch.cuda.synchronize()
    for i in range(len(shapes)):
        assert_bf16_equal(b.get("o", i), a.get("o", i), f"in place {shapes[i]}")


@pytest.mark.parametrize("u_f32", [False, True])
def test_split_gram(env, u_f32):
    """Matrices whose gram's inner dimension is split between waves (few block rows,
    a long other side, any remainder of it by four), around both ends of the rule:
    within the bound before the last rounding, and the same bits in a plan of its
    own."""
    rng = np.random.default_rng(21)
    shapes = [(129, 1024), (140, 1030), (1100, 200), (300, 1217), (512, 961), (511, 960), (513, 1000), (1345, 321)]
    us = [spectrum(rng, s, k) for s, k in zip(shapes, ["gauss", "power", "low", "gauss", "power", "gauss", "gauss", "low"])]
    t = Steps(env, us, u_f32)
    assert sum(t.plan.groups[i].split for i in range(t.plan.n_groups)) == 1 and t.plan.n_groups == 2
    for steps in (1, 5):
        together = t.o(steps)
        for i, u in enumerate(t.u):
            exact = ref.iterate64(u, steps)
            bound, size = ref.iterate_bound(u, steps)
            off = np.linalg.norm(together[i] - exact)
            assert off <= (bound - ref.BF16 * size) / (1 + ref.BF16), (shapes[i], steps, off / size)
            assert np.array_equal(Steps(env, [us[i]], u_f32).o(steps)[0], together[i]), (shapes[i], steps)
