"""Moments in 8 bits on the GPU: conversions and the AdamW step with 8-bit m and
v, bit for bit against tests/state8_ref.py and the oracle's fp32 step on the
widened moments, and against 64 bits within the roundings counted here."""
from __future__ import annotations

import math

import numpy as np
import pytest

import oracle
import synth
import zero_sharded_mixed_zero1_amd as z
from tests import state8_ref as ref
from tests.gpu_util import assert_bf16_equal, assert_f32_equal, to_dev_u16, to_np_u16, torch_cuda, ws_tensor

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, max_norm=1.0)
GUARD = 64


@pytest.fixture(scope="module")
def env():
    torch = torch_cuda()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, dev


def bf16_bits(x):
    u = x.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)).astype(np.uint16)
    return np.where(np.isnan(x), (u >> np.uint64(16)).astype(np.uint16) | 0x40, r).astype(np.uint16)


def widen(h):
    return (h.astype(np.uint32) << 16).view(np.float32)


def values(n, seed, spread=3.0):
    rng = np.random.default_rng(seed)
    return (1e-3 * rng.standard_normal(n) * np.exp(spread * rng.standard_normal(n))).astype(np.float32)


class Buf:
    """A device buffer of bytes between guards, `skew` bytes off its 256-byte alignment."""

    def __init__(self, torch, dev, n, skew=0, fill=0xA7):
        self.t = torch.full((n + 2 * 256 + skew,), fill, dtype=torch.uint8, device=dev)
        self.view = self.t[256 + skew:256 + skew + n]
        self.fill, self.n, self.skew = fill, n, skew

    def guards_hold(self):
        a = self.t.cpu().numpy()
        lo = 256 + self.skew
        return (a[:lo] == self.fill).all() and (a[lo + self.n:] == self.fill).all()

    def put(self, a):
        import torch
        self.view.copy_(torch.from_numpy(np.ascontiguousarray(a).view(np.uint8)))

    def get(self, dtype=np.uint8):
        return self.view.cpu().numpy().view(dtype)


# ------------------------------------------------------------------ conversions
@pytest.mark.parametrize("which", [z.STATE_M, z.STATE_V])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [0, 1, 3, 64, 255, 256, 257, 1000, 2047, 2048, 2049, 100_003])
@pytest.mark.parametrize("skew", [0, 1])
def test_encode_and_decode(env, n, bf16, which, skew):
    torch, dev = env
    flags, e = (z.MV_BF16, 2) if bf16 else (0, 4)
    x = values(n, n + which)
    if which == z.STATE_V:
        x = x * x
    if bf16:
        x = widen(bf16_bits(x))
    src = Buf(torch, dev, n * e, skew=skew * e)
    src.put(bf16_bits(x) if bf16 else x)
    buf = Buf(torch, dev, ref.size(n))
    z.state8_encode(src.view, n, buf.view, which, flags=flags)
    codes, words = ref.encode_nearest(np.sqrt(x) if which == z.STATE_V else x, which)
    got_c, got_w = ref.split(buf.get(), n)
    assert np.array_equal(got_w, words) and np.array_equal(got_c, codes)
    assert (buf.get()[n:ref.words_at(n)] == 0xA7).all(), "the bytes between codes and words are left alone"
    out = Buf(torch, dev, n * e, skew=skew * e)
    z.state8_decode(buf.view, n, out.view, which, flags=flags)
    y = ref.decode(codes, words, which)
    got = out.get(np.uint16 if bf16 else np.float32)
    assert np.array_equal(got, bf16_bits(y) if bf16 else y)
    assert src.guards_hold() and buf.guards_hold() and out.guards_hold()
    # against 64 bits: half a code's step (2^-4) for m, on the root for v, where the value reaches 2^-13 of the block's
    # largest (2^-13 of the root's); a bf16 rounding more
    if n:
        r = np.sqrt(x.astype(np.float64)) if which == z.STATE_V else np.abs(x.astype(np.float64))
        top = np.repeat(np.pad(r, (0, -n % 256)).reshape(-1, 256).max(1), 256)[:n]
        big = r >= 2.0 ** -13 * top
        back = np.abs((widen(got) if bf16 else got).astype(np.float64))
        back = np.sqrt(back) if which == z.STATE_V else back
        assert (np.abs(back - r)[big] <= (2.0 ** -4 + (2.0 ** -8 if bf16 else 2.0 ** -22)) * r[big]).all()


def test_conversion_of_special_values(env):
    torch, dev = env
    x = np.tile(values(256, 5), 6)
    x[0], x[1], x[2] = np.nan, np.inf, -np.inf             # block 0: beside finite ones
    x[256:512] = np.nan                                    # block 1: nothing else
    x[512:768] = 0.0                                       # block 2: zeros of both signs
    x[600] = -0.0
    x[768:1024] = np.float32(2.0 ** -149) * np.arange(256)  # block 3: subnormals
    x[1024] = np.finfo(np.float32).max                     # block 4: the largest values there are
    x[1025] = -np.finfo(np.float32).max
    x[1030] = np.float32(2.0 ** 127)
    n = x.size
    for which in (z.STATE_M, z.STATE_V):
        t = torch.from_numpy(x).to(dev)
        buf = Buf(torch, dev, ref.size(n))
        z.state8_encode(t, n, buf.view, which)
        with np.errstate(invalid="ignore"):
            codes, words = ref.encode_nearest(np.sqrt(x) if which == z.STATE_V else x, which)
        got_c, got_w = ref.split(buf.get(), n)
        assert np.array_equal(got_w, words) and np.array_equal(got_c, codes)
        out = torch.full((n,), 7.0, device=dev)
        z.state8_decode(buf.view, n, out, which)
        y = out.cpu().numpy()
        assert_f32_equal(y, ref.decode(codes, words, which), "decode")
        bad = ~np.isfinite(x) | ((x < 0) if which == z.STATE_V else False)
        assert np.array_equal(np.isnan(y), bad) and not np.isinf(y).any()


def test_zero_bytes_stand_for_zeros(env):
    torch, dev = env
    n = 1000
    buf = torch.zeros(z.state8_bytes(n), dtype=torch.uint8, device=dev)
    for which in (z.STATE_M, z.STATE_V):
        out = torch.full((n,), 7.0, device=dev)
        z.state8_decode(buf, n, out, which)
        assert (out == 0).all()


def test_every_code_decodes(env):
    torch, dev = env
    codes = np.arange(256, dtype=np.uint8)
    for b in (0, 1, 2, 127, 200, 247):
        words = np.array([b | 0x123400], np.uint32)
        buf = torch.from_numpy(ref.join(codes, words)).to(dev)
        for which in (z.STATE_M, z.STATE_V):
            out = torch.empty(256, device=dev)
            z.state8_decode(buf, 256, out, which)
            want = ref.decode(codes, words, which)
            if b == 247:                                   # codes that no encoding gives stand for more than binary32 holds
                keep = np.abs(ref.E4M3[codes]) <= 240
                assert_f32_equal(out.cpu().numpy()[keep], want[keep], "decode")
            else:
                assert_f32_equal(out.cpu().numpy(), want, f"decode b={b}")


# ------------------------------------------------------------------ the step
class Shard8:
    """One rank's shard with 8-bit moments: each tensor's part in buffers of its own between guards."""

    def __init__(self, env, numels, W, rank, seed, start=True, skew=0):
        torch, dev = self.torch, self.dev = env
        N = sum(numels)
        self.W, self.rank = W, rank
        self.begin, self.S = z.shard_range(N, W, rank)
        self.pl = z.shard_pieces(numels, self.begin, self.begin + self.S)
        self.master_np = synth.f32(N, synth.master_key(seed), 0, 0.02)[self.begin:self.begin + self.S].copy()
        self.param_np = np.zeros(self.S, np.uint16)
        self.master, self.param, self.m, self.v, self.np8 = [], [], [], [], []
        pieces = []
        for ti, off, so, n in self.pl:
            ms, pr = Buf(torch, dev, 4 * n, skew=4 * skew), Buf(torch, dev, 2 * n, skew=2 * skew)
            ms.put(self.master_np[so:so + n])
            m, v = Buf(torch, dev, ref.size(n)), Buf(torch, dev, ref.size(n))
            if start:                                      # as a run in its middle has them
                mc, mw = ref.encode_nearest(values(n, seed + so), ref.M)
                vc, vw = ref.encode_nearest(np.abs(values(n, seed + so + 1)), ref.V)
                mw, vw = mw | np.uint32(5 << 8), vw | np.uint32(5 << 8)
            else:
                mc, vc = np.zeros(n, np.uint8), np.zeros(n, np.uint8)
                mw, vw = np.zeros(ref.blocks(n), np.uint32), np.zeros(ref.blocks(n), np.uint32)
            m.put(ref.join(mc, mw))
            v.put(ref.join(vc, vw))
            self.np8.append([mc, mw, vc, vw])
            for lst, x in ((self.master, ms), (self.param, pr), (self.m, m), (self.v, v)):
                lst.append(x)
            pieces.append((n, so, pr.view, ms.view, m.view, v.view))
        self.pieces = pieces
        self.table = ws_tensor(torch, z.mta_table_bytes(pieces), dev)
        self.plan = z.mta_plan(pieces, self.table, flags=z.MV_8BIT)

    def workspace(self, flags=0):
        return ws_tensor(self.torch, z.mta_workspace_bytes(self.plan, self.W, flags), self.dev)

    def expect(self, G, hp, rs, average=True, variant=0):
        """The oracle's fp32 step on the widened moments, rounded back by the reference."""
        m = np.concatenate([ref.decode(q[0], q[1], ref.M) for q in self.np8]) if self.np8 else np.zeros(0, np.float32)
        v = np.concatenate([ref.decode(q[2], q[3], ref.V) for q in self.np8]) if self.np8 else np.zeros(0, np.float32)
        with np.errstate(all="ignore"):
            info = oracle.step([g[self.begin:self.begin + self.S] for g in G], self.master_np, m, v, self.param_np, hp, rs,
                               self.rank, average=average, variant=variant)
            r = np.sqrt(v)
        for (ti, off, so, n), q in zip(self.pl, self.np8):
            q[:] = ref.round_step(m[so:so + n], r[so:so + n], q[1], q[3], so)
        return info

    def check(self, what):
        for k, (ti, off, so, n) in enumerate(self.pl):
            assert_f32_equal(self.master[k].get(np.float32), self.master_np[so:so + n], f"master {what}")
            assert_bf16_equal(self.param[k].get(np.uint16), self.param_np[so:so + n], f"param {what}")
            for buf, c, w, name in ((self.m[k], 0, 1, "m"), (self.v[k], 2, 3, "v")):
                gc, gw = ref.split(buf.get(), n)
                assert np.array_equal(gw, self.np8[k][w]), f"{name} words, piece {k} {what}"
                assert np.array_equal(gc, self.np8[k][c]), f"{name} codes, piece {k} {what}: {(gc != self.np8[k][c]).sum()} of {n}"
                assert (buf.get()[n:ref.words_at(n)] == np.frombuffer(ref.join(self.np8[k][c], self.np8[k][w]), np.uint8)[n:ref.words_at(n)]).all()
            for buf in (self.master[k], self.param[k], self.m[k], self.v[k]):
                assert buf.guards_hold(), f"written beside a buffer of piece {k} {what}"


def grads_of(torch, dev, N, W, seed, t, sigma=0.02):
    G = [synth.bf16(N, synth.grad_key(seed, t, w), 0, sigma, 1) for w in range(W)]
    return G, [to_dev_u16(torch, g, dev) for g in G]


LISTS = {
    "ragged": [3000, 17, 5000, 8, 2203, 1, 255, 256, 257, 70_001],
    "round": [4096, 2048, 8192, 16384, 256],
    "one": [1],
}


@pytest.mark.parametrize("numels", list(LISTS), ids=list(LISTS))
@pytest.mark.parametrize("W,rank,design", [(1, 0, 0), (2, 1, 0), (3, 0, z.STORE_G), (4, 3, z.RECOMPUTE_G), (5, 2, 0), (8, 7, 0), (8, 0, z.RECOMPUTE_G)])
def test_step_is_the_oracles_rounded(env, numels, W, rank, design):
    torch, dev = env
    numels = LISTS[numels]
    N, seed = sum(numels), 0x8B00 + W
    if numels == [1]:
        rank = 0                                           # the others own nothing
    sh = Shard8(env, numels, W, rank, seed)
    ws = sh.workspace(design)
    for t in range(6, 9):
        G, gd = grads_of(torch, dev, N, W, seed, t)
        rs = np.full(W, 0.3)
        rsd = torch.from_numpy(rs.copy()).to(dev)
        hp = dict(HP, step=t)
        z.mta_step(gd, sh.begin, sh.plan, hp, rsd, W, rank, flags=design, ws=ws)
        sh.expect(G, hp, rs)
        sh.check(f"t={t}")


@pytest.mark.parametrize("skew", [1, 3])
def test_misaligned_master_and_param(env, skew):
    torch, dev = env
    numels, W, rank = [5000, 2048, 9000], 3, 1
    sh = Shard8(env, numels, W, rank, 77, skew=skew)
    G, gd = grads_of(torch, dev, sum(numels), W, 77, 1)
    rs = np.zeros(W)
    rsd = torch.zeros(W, dtype=torch.float64, device=dev)
    for t in (1, 2):
        z.mta_step(gd, sh.begin, sh.plan, dict(HP, step=t), rsd, W, rank, ws=sh.workspace())
        sh.expect(G, dict(HP, step=t), rs)
        sh.check(f"t={t}")


@pytest.mark.parametrize("flags,variant,average", [(z.DECAY_FIRST, oracle.DECAY_FIRST, True), (z.CLIP_EPS, oracle.CLIP_EPS, True),
                                                   (z.G_BF16, oracle.G_BF16, True), (z.SUM_ONLY, 0, False)])
def test_variants(env, flags, variant, average):
    torch, dev = env
    numels, W, rank = [3000, 4096, 77], 2, 0
    sh = Shard8(env, numels, W, rank, 91)
    G, gd = grads_of(torch, dev, sum(numels), W, 91, 1)
    rs, rsd = np.zeros(W), torch.zeros(W, dtype=torch.float64, device=dev)
    z.mta_step(gd, sh.begin, sh.plan, dict(HP, step=3), rsd, W, rank, flags=flags, ws=sh.workspace())
    sh.expect(G, dict(HP, step=3), rs, average=average, variant=variant)
    sh.check("")


@pytest.mark.parametrize("change", [dict(beta1=0.0), dict(beta2=0.0), dict(beta1=0.0, beta2=0.0), dict(lr=0.0), dict(max_norm=math.inf),
                                    dict(beta2=0.999, eps=1e-15)])
def test_edge_hyper_parameters(env, change):
    torch, dev = env
    numels = [3000, 2048, 5]
    sh = Shard8(env, numels, 1, 0, 17)
    G, gd = grads_of(torch, dev, sum(numels), 1, 17, 1)
    rs, rsd = np.zeros(1), torch.zeros(1, dtype=torch.float64, device=dev)
    hp = {**HP, **change, "step": 4}
    z.mta_step(gd, 0, sh.plan, hp, rsd, 1, 0, ws=sh.workspace())
    sh.expect(G, hp, rs)
    sh.check(str(change))


def test_first_steps_from_zero_bytes(env):
    """Zero bytes are the state before the first step; all-zero gradients leave zeros, with no NaN."""
    torch, dev = env
    numels = [3000, 2048, 5]
    N = sum(numels)
    sh = Shard8(env, numels, 1, 0, 23, start=False)
    rs, rsd = np.zeros(1), torch.zeros(1, dtype=torch.float64, device=dev)
    zero = np.zeros(N, np.uint16)
    G, gd = grads_of(torch, dev, N, 1, 23, 1)
    for t, (g, d) in enumerate([([zero], [to_dev_u16(torch, zero, dev)]), (G, gd), (G, gd)], 1):
        z.mta_step(d, 0, sh.plan, dict(HP, step=t), rsd, 1, 0, ws=sh.workspace())
        sh.expect(g, dict(HP, step=t), rs)
        sh.check(f"t={t}")
        assert np.isfinite(sh.master_np).all()


def test_nan_and_infinite_gradients(env):
    """They reach their own elements' moments as NaN (and the norm); the other elements of their blocks stay finite."""
    torch, dev = env
    numels = [4096, 300]
    N = sum(numels)
    sh = Shard8(env, numels, 1, 0, 29)
    G, _ = grads_of(torch, dev, N, 1, 29, 1)
    G[0][[5, 700, 4200]] = [0x7FC0, 0x7F80, 0xFF80]
    gd = [to_dev_u16(torch, G[0], dev)]
    rs, rsd = np.zeros(1), torch.zeros(1, dtype=torch.float64, device=dev)
    hp = dict({**HP, "max_norm": math.inf}, step=2)
    for _ in range(2):
        z.mta_step(gd, 0, sh.plan, hp, rsd, 1, 0, ws=sh.workspace())
        sh.expect(G, hp, rs)
        sh.check("")
    bad = np.zeros(N, bool)
    bad[[5, 700, 4200]] = True
    assert np.array_equal(np.isnan(sh.master_np), bad)


def test_a_root_that_is_not_zero_stays_so(env):
    """Gradients far below their block's largest: the held root keeps the update bounded step after step."""
    torch, dev = env
    n = 2048
    g = np.full(n, 1e-12, np.float32)
    g[::256] = 1e3
    G = [bf16_bits(g)]
    gd = [to_dev_u16(torch, G[0], dev)]
    sh = Shard8(env, [n], 1, 0, 31, start=False)
    rs, rsd = np.zeros(1), torch.zeros(1, dtype=torch.float64, device=dev)
    for t in range(1, 30):
        hp = {**HP, "max_norm": math.inf, "weight_decay": 0.0, "step": t}
        before = sh.master_np.copy()
        z.mta_step(gd, 0, sh.plan, hp, rsd, 1, 0, ws=sh.workspace())
        sh.expect(G, hp, rs)
        sh.check(f"t={t}")
        # |m| is at most a code above what the largest gradients leave, r at least the smallest code of the same block:
        # lr sqrt(bc2) / bc1 times m / r stays below 2 lr * 2^17 / 2^17 ... a few learning rates
        assert np.abs(sh.master_np - before).max() <= 8 * HP["lr"]
    assert (sh.np8[0][2] > 0).all()


def test_flat_step_g_given_or_recomputed(env):
    torch, dev = env
    for n in (1, 255, 2048, 100_003):
        G, gd = grads_of(torch, dev, n, 3, n, 1)
        g = oracle.shard_reduce(G)
        rs = np.array([oracle.sumsq(g), 0.2])
        for given in (True, False):
            mc, mw = ref.encode_nearest(values(n, n), ref.M)
            vc, vw = ref.encode_nearest(np.abs(values(n, n + 1)), ref.V)
            master = values(n, n + 2)
            m, v = Buf(torch, dev, ref.size(n)), Buf(torch, dev, ref.size(n))
            m.put(ref.join(mc, mw))
            v.put(ref.join(vc, vw))
            md = torch.from_numpy(master.copy()).to(dev)
            param = torch.zeros(n, dtype=torch.int16, device=dev)
            hp = dict(HP, step=5)
            z.adamw_step(torch.from_numpy(g).to(dev) if given else None, None if given else gd, 0, n, md, m.view, v.view, param,
                         hp, torch.from_numpy(rs).to(dev), 2, flags=z.MV_8BIT)
            mm, vv, p = ref.decode(mc, mw, ref.M), ref.decode(vc, vw, ref.V), np.zeros(n, np.uint16)
            clip, coef = oracle.clip_coef(oracle.global_norm(rs), HP["max_norm"])
            oracle.adamw(g, master, mm, vv, p, oracle.adamw_scalars(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"], 5), clip, coef)
            want = ref.round_step(mm, np.sqrt(vv), mw, vw, 0)
            assert_f32_equal(md.cpu().numpy(), master, "master")
            assert_bf16_equal(to_np_u16(param), p, "param")
            for buf, c, w in ((m, 0, 1), (v, 2, 3)):
                gc, gw = ref.split(buf.get(), n)
                assert np.array_equal(gw, want[w]) and np.array_equal(gc, want[c]) and buf.guards_hold()


def test_long_shard(env):
    """Past the size where each XCD walks its own part of the tiles; a ragged tail; multi-tensor and flat."""
    torch, dev = env
    numels = [(1 << 24) + 2053, 777]
    N = sum(numels)
    sh = Shard8(env, numels, 1, 0, 41)
    G, gd = grads_of(torch, dev, N, 1, 41, 1)
    rs, rsd = np.zeros(1), torch.zeros(1, dtype=torch.float64, device=dev)
    z.mta_step(gd, 0, sh.plan, dict(HP, step=2), rsd, 1, 0, ws=sh.workspace())
    sh.expect(G, dict(HP, step=2), rs)
    sh.check("long")


@pytest.mark.parametrize("design", [z.STORE_G, z.RECOMPUTE_G])
def test_captured_step_replays(env, design):
    """One captured step replayed four times between eager work equals the eager steps: the rounding's bits come from
    the words, so every replay takes new ones."""
    torch, dev = env
    numels, W, rank = [30_001, 7, 2_048 * 5, 9_000], 4, 2
    G, gd = grads_of(torch, dev, sum(numels), W, 51, 1)
    sh = Shard8(env, numels, W, rank, 51)
    ws = sh.workspace(design)
    rsd = torch.full((W,), 0.3, dtype=torch.float64, device=dev)
    rs = np.full(W, 0.3)
    scal = torch.zeros(40, dtype=torch.uint8, device=dev)
    z.mta_step(gd, sh.begin, sh.plan, dict(HP, step=1), rsd, W, rank, flags=design, ws=ws)
    sh.expect(G, dict(HP, step=1), rs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z.mta_step(gd, sh.begin, sh.plan, {"device_scalars": scal}, rsd, W, rank, flags=design, ws=ws)
    noise = torch.ones(1 << 20, device=dev)
    for t in range(2, 6):
        scal.copy_(torch.from_numpy(np.frombuffer(bytes(z.step_scalars_derive(dict(HP, step=t))), np.uint8).copy()))
        graph.replay()
        noise.mul_(1.0001).add_(1.0)
        torch.cuda.synchronize()
        sh.expect(G, dict(HP, step=t), rs)
        sh.check(f"replay t={t}")
    del graph


def test_bucketed_and_static_flows(env):
    torch, dev = env
    numels, W, rank = [30_001, 7, 2_048 * 5, 9_000], 8, 3
    N = sum(numels)
    G, gd = grads_of(torch, dev, N, W, 61, 1)
    rs = np.full(W, 0.3)
    a, b = Shard8(env, numels, W, rank, 61), Shard8(env, numels, W, rank, 61)
    rsd = torch.full((W,), 0.3, dtype=torch.float64, device=dev)
    ws = a.workspace(z.STORE_G)
    parts = torch.zeros(2, dtype=torch.float64, device=dev)
    cut = 3333
    for k, (lo, hi) in enumerate([(cut, a.S), (0, cut)]):
        z.mta_reduce_range([g[a.begin + lo:] for g in gd], a.plan, lo, hi, parts[k:], ws=ws)
    z.partials_sum(parts, 2, rsd[rank:])
    z.mta_update(gd, a.begin, a.plan, dict(HP, step=1), rsd, W, flags=z.STORE_G, ws=ws)
    a.expect(G, dict(HP, step=1), rs)
    a.check("bucketed")
    rsd = torch.full((W,), 0.3, dtype=torch.float64, device=dev)
    z.mta_step_static(gd, b.begin, b.plan, dict(HP, step=1), rsd, W, rank)
    b.expect(G, dict(HP, step=1), np.full(W, 0.3))
    b.check("static")


def test_arena_holds_8_bit_moments(env):
    torch, dev = env
    S, W = 70_001, 3
    a = z.arena_tensors(S, W, S, 0, S, 0, flags=z.MV_8BIT, device=dev, capacity=64 << 20)
    assert a.m.numel() == z.state8_bytes(S) == a.v.numel()
    for t in (a.m, a.v, a.params):
        t.zero_()
    master = synth.f32(S, synth.master_key(7), 0, 0.02)
    a.master.copy_(torch.from_numpy(master))
    G, gd = grads_of(torch, dev, S, W, 7, 1)
    for w in range(W):
        a.grads[w].copy_(gd[w])
    pieces = [(S, 0, a.params, a.master, a.m, a.v)]
    table = ws_tensor(torch, z.mta_table_bytes(pieces), dev)
    plan = z.mta_plan(pieces, table, flags=z.MV_8BIT)
    rsd = torch.zeros(1, dtype=torch.float64, device=dev)
    z.mta_step(a.grads, 0, plan, dict(HP, step=1), rsd, 1, 0, ws=a.ws)
    m, v, p, rs = np.zeros(S, np.float32), np.zeros(S, np.float32), np.zeros(S, np.uint16), np.zeros(1)
    oracle.step(G, master, m, v, p, dict(HP, step=1), rs, 0)
    zero = np.zeros(ref.blocks(S), np.uint32)
    want = ref.round_step(m, np.sqrt(v), zero, zero, 0)
    assert_f32_equal(a.master.cpu().numpy(), master, "master")
    for t, c, w in ((a.m, 0, 1), (a.v, 2, 3)):
        gc, gw = ref.split(t.cpu().numpy(), S)
        assert np.array_equal(gc, want[c]) and np.array_equal(gw, want[w])


def test_two_streams_and_a_rerun(env):
    """Two shards stepped at once on two streams, and again from copies of their state: the same bits."""
    torch, dev = env
    numels = [200_003, 4096]
    G, gd = grads_of(torch, dev, sum(numels), 1, 71, 1)
    shards = [Shard8(env, numels, 1, 0, 71 + k) for k in range(2)]
    ws = [s.workspace() for s in shards]
    rsd = [torch.zeros(1, dtype=torch.float64, device=dev) for _ in shards]
    streams = [torch.cuda.Stream() for _ in shards]
    torch.cuda.synchronize()
    for t in range(1, 5):
        for s, w, r, st in zip(shards, ws, rsd, streams):
            z.mta_step(gd, 0, s.plan, dict(HP, step=t), r, 1, 0, ws=w, stream=st)
    torch.cuda.synchronize()
    for s in shards:
        rs = np.zeros(1)
        for t in range(1, 5):
            s.expect(G, dict(HP, step=t), rs)
        s.check("streams")


def test_small_changes_add_up(env):
    """beta2 = 0.999: a step changes v by a thousandth, a code's distance is an eighth.  Over 3000 steps of random
    gradients the mean of v follows the exact average.  The held root is right on average, so r^2 is high by its
    variance: a step moves r by (1 - beta2)/2 |g^2/v - 1| of itself, 0.97 (1 - beta2)/2 on average for normal g; its
    rounding's variance is at most that times a step of 1/8, which beta2 forgets at the rate (1 - beta2): 6 % of v.
    (65,536 elements: the mean's own spread is under 0.3 %.)"""
    torch, dev = env
    n, steps = 65_536, 3000
    gen = torch.Generator(device=dev).manual_seed(3)
    m, v = (torch.zeros(z.state8_bytes(n), dtype=torch.uint8, device=dev) for _ in range(2))
    master, param = torch.zeros(n, device=dev), torch.zeros(n, dtype=torch.bfloat16, device=dev)
    rs = torch.ones(1, dtype=torch.float64, device=dev)
    exact = torch.zeros(n, dtype=torch.float64, device=dev)
    exact_m = torch.zeros(n, dtype=torch.float64, device=dev)
    hp = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_norm=math.inf)
    for t in range(1, steps + 1):
        g = torch.randn(n, generator=gen, device=dev).bfloat16()
        z.adamw_step(None, [g], 0, n, master, m, v, param, dict(hp, step=t), rs, 1, flags=z.MV_8BIT)
        exact = exact * 0.999 + 0.001 * g.double().square()
        exact_m = exact_m * 0.9 + 0.1 * g.double()
    out = torch.empty(n, device=dev)
    z.state8_decode(v, n, out, z.STATE_V)
    ratio = float((out.double() / exact).mean())
    assert 0.99 <= ratio <= 1.07, ratio
    z.state8_decode(m, n, out, z.STATE_M)
    # m: one step's rounding is at most 1/8 of the value and is forgotten at the rate 0.1: its variance is at most
    # (m/8)^2/4 / (1 - 0.81) of the mean square, 2 % of it
    d = out.double() - exact_m
    assert float(d.square().mean() / exact_m.square().mean()) <= 0.021
    # (mean of 65,536: six standard errors)
    assert abs(float(d.mean())) <= 6 * float(d.std()) / n ** 0.5


def test_calls_run_on_torchs_current_stream(env):
    from zero_sharded_mixed_zero1_amd import binding
    torch, dev = env
    side = torch.cuda.Stream()
    assert binding._stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert binding._stream(None) == side.cuda_stream == torch.cuda.current_stream().cuda_stream
    assert binding._stream(side) == side.cuda_stream
    assert binding._stream(None) == torch.cuda.current_stream().cuda_stream != side.cuda_stream


def test_rounding_at_its_borders(env):
    """Magnitudes and bits at which the sum just reaches, or just misses, the next code, in every binade of the codes and
    below the smallest normal one, where binary32's scaled bits are rounded to 2^-29 of a unit first."""
    torch, dev = env
    rng = np.random.default_rng(9)
    n = 256 * 512
    first, counts = 0, np.zeros(ref.blocks(n), np.uint32)
    bits = ref.random_bits(first, counts, n).astype(np.int64)
    for which, half in ((ref.M, bits & 0xFFFF), (ref.V, bits >> 16)):
        # a value whose fraction of a code's step is 1 - u / 65536 give or take less than 2^-20
        e = rng.integers(-9, 7, n)
        step = 2.0 ** (np.maximum(e, -6) - 3)
        k = np.floor(2.0 ** e / step + rng.integers(0, 8, n) * (e >= -6))
        near = (1 - half / 65536.0) + rng.choice([-1, -0.75, -0.5, -0.25, 0, 0.25, 0.5, 1], n) * 2.0 ** -20
        y = (k + np.clip(near, 0, 1 - 2.0 ** -20)) * step
        y[::256] = 200.0                                   # the block's largest
        x = y.astype(np.float32)
        # a step that leaves x: m = 0 * m + 1 * g (beta1 = 0), r = sqrt(0 * v + 1 * g^2); g fp32
        hp = dict(lr=0.0, beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0, max_norm=math.inf, step=1)
        m, v = (torch.zeros(z.state8_bytes(n), dtype=torch.uint8, device=dev) for _ in range(2))
        master, param = torch.zeros(n, device=dev), torch.zeros(n, dtype=torch.int16, device=dev)
        z.adamw_step(torch.from_numpy(x).to(dev), None, 0, n, master, m, v, param, hp, torch.ones(1, dtype=torch.float64, device=dev),
                     1, flags=z.MV_8BIT)
        r = np.sqrt(x * x) if which == ref.V else np.sqrt(x * x)
        want = ref.round_step(x, r, np.zeros(ref.blocks(n), np.uint32), np.zeros(ref.blocks(n), np.uint32), first)
        gc, gw = ref.split(m.cpu().numpy(), n)
        assert np.array_equal(gw, want[1]) and np.array_equal(gc, want[0]), f"m: {(gc != want[0]).sum()} differ"
        gc, gw = ref.split(v.cpu().numpy(), n)
        assert np.array_equal(gw, want[3]) and np.array_equal(gc, want[2]), f"v: {(gc != want[2]).sum()} differ"


def test_param_is_the_nearest_bf16_of_any_master(env):
    """Masters of every kind of bits through a step that changes none of them."""
    torch, dev = env
    n = 1 << 20
    u = np.random.default_rng(4).integers(0, 1 << 32, n, dtype=np.uint64).astype(np.uint32)
    u[:8] = [0x3F808000, 0x3F818000, 0x7F7FFFFF, 0x7F7F8000, 0x00008000, 0x00018000, 0x80000000, 0x7F800000]
    u[2048:4096] &= 0x807FFFFF                             # subnormals
    x = u.view(np.float32)
    hp = dict(lr=0.0, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, max_norm=math.inf, step=1)
    m, v = (torch.zeros(z.state8_bytes(n), dtype=torch.uint8, device=dev) for _ in range(2))
    master, param = torch.from_numpy(x.copy()).to(dev), torch.zeros(n, dtype=torch.int16, device=dev)
    g = torch.full((n,), 1e-3, device=dev)
    z.adamw_step(g, None, 0, n, master, m, v, param, hp, torch.ones(1, dtype=torch.float64, device=dev), 1, flags=z.MV_8BIT)
    assert_f32_equal(master.cpu().numpy(), x, "master")
    assert_bf16_equal(to_np_u16(param), bf16_bits(x), "param")


@pytest.mark.parametrize("given", [True, False])
def test_long_flat_step(env, given):
    """The flat step past the size where each XCD walks its own part of the tiles, with a ragged tail."""
    torch, dev = env
    n, W = (1 << 24) + 2053, 2
    G, gd = grads_of(torch, dev, n, W, 43, 1)
    g = oracle.shard_reduce(G)
    rs = np.array([0.3])
    mc, mw = ref.encode_nearest(values(n, 1), ref.M)
    vc, vw = ref.encode_nearest(np.abs(values(n, 2)), ref.V)
    master = values(n, 3)
    m, v = Buf(torch, dev, ref.size(n)), Buf(torch, dev, ref.size(n))
    m.put(ref.join(mc, mw))
    v.put(ref.join(vc, vw))
    md = torch.from_numpy(master.copy()).to(dev)
    param = torch.zeros(n, dtype=torch.int16, device=dev)
    hp = dict(HP, step=5)
    z.adamw_step(torch.from_numpy(g).to(dev) if given else None, None if given else gd, 0, n, md, m.view, v.view, param, hp,
                 torch.from_numpy(rs).to(dev), 1, flags=z.MV_8BIT)
    mm, vv, p = ref.decode(mc, mw, ref.M), ref.decode(vc, vw, ref.V), np.zeros(n, np.uint16)
    clip, coef = oracle.clip_coef(oracle.global_norm(rs), HP["max_norm"])
    oracle.adamw(g, master, mm, vv, p, oracle.adamw_scalars(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"], 5), clip, coef)
    want = ref.round_step(mm, np.sqrt(vv), mw, vw, 0)
    assert_f32_equal(md.cpu().numpy(), master, "master")
    assert_bf16_equal(to_np_u16(param), p, "param")
    for buf, c, w in ((m, 0, 1), (v, 2, 3)):
        gc, gw = ref.split(buf.get(), n)
        assert np.array_equal(gw, want[w]) and np.array_equal(gc, want[c]) and buf.guards_hold()


@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("W", [1, 3, 6, 64])
def test_flat_step_of_misaligned_slices(env, W, skew):
    """Slices, master and parameters off every vector's alignment; lengths around the tile and the quad."""
    torch, dev = env
    for n in (1, 2, 3, 5, 2047, 2049, 2050, 2051, 4099):
        begin = 3 * skew
        G = [synth.bf16(n + begin, synth.grad_key(7, 1, w), 0, 0.02, 1) for w in range(W)]
        gd = [to_dev_u16(torch, x, dev) for x in G]
        g = oracle.shard_reduce([x[begin:] for x in G])
        rs = np.array([oracle.sumsq(g)])
        mc, mw = ref.encode_nearest(values(n, n), ref.M)
        vc, vw = ref.encode_nearest(np.abs(values(n, n + 1)), ref.V)
        master, p = values(n, n + 2), np.zeros(n, np.uint16)
        m, v, ms, pr = Buf(torch, dev, ref.size(n)), Buf(torch, dev, ref.size(n)), Buf(torch, dev, 4 * n, skew=4 * skew), Buf(torch, dev, 2 * n, skew=2 * skew)
        m.put(ref.join(mc, mw))
        v.put(ref.join(vc, vw))
        ms.put(master)
        z.adamw_step(None, gd, begin, n, ms.view, m.view, v.view, pr.view, dict(HP, step=2), torch.from_numpy(rs).to(dev), 1, flags=z.MV_8BIT)
        mm, vv = ref.decode(mc, mw, ref.M), ref.decode(vc, vw, ref.V)
        clip, coef = oracle.clip_coef(oracle.global_norm(rs), HP["max_norm"])
        oracle.adamw(g, master, mm, vv, p, oracle.adamw_scalars(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"], 2), clip, coef)
        want = ref.round_step(mm, np.sqrt(vv), mw, vw, 0)
        assert_f32_equal(ms.get(np.float32), master, f"master n={n}")
        assert_bf16_equal(pr.get(np.uint16), p, f"param n={n}")
        for buf, c, w in ((m, 0, 1), (v, 2, 3)):
            gc, gw = ref.split(buf.get(), n)
            assert np.array_equal(gw, want[w]) and np.array_equal(gc, want[c]) and buf.guards_hold()
        assert ms.guards_hold() and pr.guards_hold()
