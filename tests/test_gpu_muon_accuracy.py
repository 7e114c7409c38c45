"""What o is before its rounding to bf16, on the GPU, against the iteration in 64
bits: inputs at the ends of the formats' ranges and the figures that the header
states."""
from __future__ import annotations

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests import muon_formats as fmt
from tests import muon_ref as ref
from tests.gpu_util import ws_tensor
from tests.test_gpu_muon import Steps, env  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("u_f32", [False, True])
@pytest.mark.parametrize("size", [1.0, 1e-20, 1e-30])
def test_parts_of_the_gram_sum_that_hold_only_zeros(env, u_f32, size):  # noqa: F811
    """Thin matrices whose gram is summed in several parts, some of them zero: the
    zeros say nothing about the size of the others, however small these are.
    eps = 0, and an eps of a millionth of the matrix's size."""
    rng = np.random.default_rng(31)
    zeros = [((100, 1000), slice(256, 384)), ((100, 1000), slice(0, 128)), ((100, 1000), slice(128, 1000)),
             ((60, 700), slice(500, 700)), ((20, 5000), slice(0, 4900)), ((1, 900), slice(100, 900))]
    us = []
    for shape, cols in zeros:
        u = rng.standard_normal(shape) * size
        u[:, cols] = 0.0
        us += [u, u.T.copy()]
    t = Steps(env, us, u_f32)
    for eps in (0.0, 1e-6 * size):
        for got, u in zip(t.o(5, eps=eps), t.u):
            exact = ref.iterate64(u, 5, eps=eps)
            off = np.linalg.norm(got - exact)
            assert off <= 5e-4 * np.linalg.norm(exact), (u.shape, size, eps, off)
    # nothing but zeros in every part
    for got in Steps(env, [np.zeros((100, 1000)), np.zeros((1000, 20))], u_f32).o(5, eps=1e-6 * size):
        assert (got == 0.0).all()


def one_step(env, shape, value, u_f32):  # noqa: F811
    """muon_step on a matrix of equal elements with coefficients (1, 0, 0): the
    master it leaves is -u / |u|."""
    torch, dev = env
    g = torch.full(shape, value, dtype=torch.bfloat16, device=dev)
    b = dict(param=torch.zeros_like(g), master=torch.zeros(shape, device=dev), m=torch.zeros(shape, device=dev),
             u=torch.zeros(shape, dtype=torch.float32 if u_f32 else torch.bfloat16, device=dev))
    mats = [z.matrix(*shape, **b)]
    table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
    plan = z.muon_plan(mats, table, flags=z.U_F32 if u_f32 else 0)
    ws = ws_tensor(torch, z.muon_workspace_bytes(plan), dev)
    ws.fill_(0xFF)
    hp = dict(lr=1.0, momentum=0.5, weight_decay=0.0, ns_steps=1, ns_a=1.0, ns_b=0.0, ns_c=0.0, ns_eps=0.0)
    z.muon_step([g], 0, plan, hp, flags=z.NO_NESTEROV, ws=ws)
    torch.cuda.synchronize()
    return b["master"]


@pytest.mark.parametrize("value", [1.2578125, 1.40625, 1.7109375])
@pytest.mark.parametrize("shape,u_f32", [((1, 1 << 26), False), ((3, 1 << 22), False), ((1 << 22, 3), True),
                                         ((100, 1 << 20), False), ((1, 300001), True)])
def test_norm_of_long_matrices(env, shape, u_f32, value):  # noqa: F811
    """The norm of a thin matrix is summed in fp32: parts in runs of at most 8192
    columns, a part's runs, then the parts.  The matrix cores round once every 8
    products (an fp32 u: three products of its halves), every addition by at most
    2^-24 of the sum so far; the norm is off by half of what its square is.  Equal
    elements are the worst: all roundings of a binade have the same sign.  o's own
    arithmetic (r, two halves of X, the product with r) adds at most 8 * 2^-24."""
    torch, _ = env
    p = one_step(env, shape, value, u_f32)
    n = max(shape)
    runs = -(-n // 32 // 8192)
    room = ((1024 * (3 if u_f32 else 1) + runs + 31) / 2 + 8) * 2.0 ** -24
    want = 1.0 / float(np.sqrt(float(shape[0]) * shape[1]))
    lo, hi = float(-p.max()), float(-p.min())
    assert want * (1 - room) <= lo <= hi <= want * (1 + room), (lo / want - 1, hi / want - 1, room)


@pytest.mark.parametrize("u_f32", [False, True])
def test_long_matrices_of_uneven_size(env, u_f32):  # noqa: F811
    """Parts of several runs whose sizes rise and fall by 2^100, with zeros between:
    the runs before are scaled to the largest so far."""
    rng = np.random.default_rng(12)
    n = 32 * 8192 * 3 + 777
    j = np.arange(n)
    us = []
    for sign in (1, -1):
        u = rng.standard_normal((2, n)) * 2.0 ** (sign * 50 * np.cos(j / 9000.0))
        u[:, (j // 8192) % 4 == 1] = 0.0
        us.append(u)
    us.append(np.where(j < n - 5000, 0.0, 1e-25) * rng.standard_normal((2, n)))
    us.append(rng.standard_normal((n, 2)) * 1e-3)
    t = Steps(env, us, u_f32)
    for steps in (5, 8):        # (eight: a second segment, whose X comes from the workspace)
        for got, u in zip(t.o(steps, eps=0.0), t.u):
            exact = ref.iterate64(u, steps, eps=0.0)
            assert np.linalg.norm(got - exact) <= fmt.stated(u.shape, steps) * np.linalg.norm(exact), (u.shape, steps)
    us[0][1, n - 3], us[1][0, 5] = np.inf, np.nan
    with np.errstate(invalid="ignore"):     # (the second slice of an infinity is a NaN)
        got = Steps(env, us, u_f32).o(5, eps=0.0)
    assert np.isnan(got[0]).all() and np.isnan(got[1]).all() and np.isfinite(got[2]).all() and np.isfinite(got[3]).all()


DENSE = [(129, 129), (400, 130), (150, 200), (256, 512), (200, 1217), (1100, 300), (513, 700)]
THIN = [(5, 300), (30, 40), (65, 65), (64, 255), (300, 100), (128, 128), (100, 1001), (127, 2100)]


@pytest.mark.parametrize("u_f32", [False, True])
@pytest.mark.parametrize("kind", fmt.KINDS)
def test_o_is_as_exact_as_stated(env, kind, u_f32):  # noqa: F811
    """Within the header's figures of the iteration in 64 bits, on every path.

    Of matrices that are not thin the formats' roundings (muon_formats.dense) explain
    it in up to five steps, but for the fp32 sums.  Where these differ by their order,
    an entry of A, B or X within 2^-24 sqrt(n) of a border of fp16's steps (2^-11) is
    rounded to the other side, one in some hundred, by a step of which the others are
    off by 1/sqrt(12) in the mean square: a third more at most.  And X itself is off
    by the sums of B X (k/8 additions, each rounding by at most 2^-24 of a partial
    sum, |b s^2 + c s^4| < 3 of X; of either sign, so their squares add) and by the
    epilogue's own operations (a X and the last sum, within 8 * 2^-24 of X).  Like
    every rounding of X that is a direction X did not have, which the steps after it
    multiply by a = 3.44 each; X is within 1.8 times o in size.  In eight steps this
    alone may reach 2 %, so there the stated figure is all that is asked."""
    rng = np.random.default_rng(41)
    t = Steps(env, [fmt.spectrum(rng, s, kind) for s in DENSE + THIN], u_f32)
    worst = {}
    for steps in (1, 5, 6, 8):
        for got, u in zip(t.o(steps), t.u):
            exact = ref.iterate64(u, steps)
            size = np.linalg.norm(exact)
            off = np.linalg.norm(got - exact) / size
            assert off <= fmt.stated(u.shape, steps), (u.shape, steps, off)
            if min(u.shape) > 128 and steps <= 5:
                formats = np.linalg.norm(fmt.dense(u, steps) - exact) / size
                sums = 1.8 * 2.0 ** -24 * (3 * np.sqrt(min(u.shape) / 8) + 8) * sum(ref.A ** j for j in range(steps))
                assert off <= 4 / 3 * formats + sums, (u.shape, steps, off, formats, sums)
            key = (min(u.shape) <= 128, steps)
            worst[key] = max(worst.get(key, 0.0), off)
    print(kind, "fp32" if u_f32 else "bf16", {("thin " if k[0] else "dense ") + str(k[1]): f"{v:.2e}" for k, v in worst.items()})


@pytest.mark.parametrize("u_f32", [False, True])
@pytest.mark.parametrize("shape", [(130, 170), (300, 1100), (2200, 2100)])
def test_ends_of_the_range_of_matrices_that_are_not_thin(env, shape, u_f32):  # noqa: F811
    """Sizes whose squares fp32 does not hold, zeros, infinities and NaNs, on the
    paths of k > 128 (a gram of tiles and a split one; norms in prepare and in a
    launch of their own): a NaN takes its own matrix only."""
    torch, dev = env
    rng = np.random.default_rng(19)
    base = rng.standard_normal(shape).astype(np.float32)
    us = [base, base * np.float32(1e36), base * np.float32(1e-36), np.zeros_like(base), base.copy(), base.copy(), base]
    us[4][-1, -1], us[5][0, 7] = np.inf, np.nan
    if shape[0] > 2000:
        us = us[1:6]
    bf = [torch.from_numpy(ref.bf16(u).reshape(shape).view(np.int16)).to(dev).view(torch.bfloat16) for u in us]
    u = [x.float() if u_f32 else x for x in bf]
    o = [torch.full(shape, 7.0, dtype=torch.bfloat16, device=dev) for _ in us]
    mats = [z.matrix(*shape, u=a, o=b) for a, b in zip(u, o)]
    table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
    plan = z.muon_plan(mats, table, flags=z.U_F32 if u_f32 else 0)
    ws = ws_tensor(torch, z.muon_workspace_bytes(plan), dev)
    ws.fill_(0xFF)
    z.orthogonalize(plan, dict(lr=0.0, momentum=0.0, weight_decay=0.0, ns_eps=0.0), ws=ws)
    torch.cuda.synchronize()
    for a, b in zip(u, o):
        x = a.double()
        if not bool((x != 0).any()) or not bool(torch.isfinite(x).all()):     # 0 / 0; the formulas' NaN
            assert bool(torch.isnan(b).all())
            continue
        x = x / torch.linalg.vector_norm(x)
        x = x.T.contiguous() if shape[0] > shape[1] else x
        for _ in range(5):
            s = x @ x.T
            x = ref.A * x + (ref.B * s + ref.C * (s @ s)) @ x
        x = x.T if shape[0] > shape[1] else x
        off = float(torch.linalg.vector_norm(b.double() - x) / torch.linalg.vector_norm(x))
        assert off <= fmt.stated(shape, 5) + ref.BF16, off      # (and the rounding to bf16)
    if shape[0] < 2000:
        assert torch.equal(o[0], o[-1])
