"""Host-side checks of the Muon entry points (no GPU): what they refuse, the
derived scalars, table and workspace sizes, and the tests' own plain forms."""
from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import pytest

import zero_sharded_mixed_zero1_amd as z
from tests import muon_ref as ref

FAKE = 1 << 40
MB = 1 << 20


def _einval(fn, name="ZERO1_EINVAL"):
    with pytest.raises(z.Zero1Error) as e:
        fn()
    assert e.value.name == name, e.value
    return e.value.message


def _mat(rows=10, cols=20, at=FAKE, **kw):
    d = dict(param=at, master=at + MB, m=at + 2 * MB, u=at + 3 * MB, o=at + 4 * MB)
    d.update(kw)
    return z.matrix(rows, cols, **d)


def _plan(**kw):
    d = dict(table=FAKE, elems=200, n_mats=1, n_tiles=1, n_groups=1, has=15,
             area_bytes=1 << 17)
    d.update(kw)
    return z.MatrixPlan(**d)


def _hp(**kw):
    d = dict(lr=1e-3, momentum=0.95, weight_decay=0.1)
    d.update(kw)
    return d


def _valid(mats, flags=0):
    """Plans up to the table's size, which is refused after everything else."""
    assert "needs" in _einval(lambda: z.muon_plan(mats, FAKE, 0, flags=flags), "ZERO1_EWORKSPACE")
    return True


def test_table_bytes_and_layout():
    # 192 bytes a matrix; streaming tiles of 512 quads (16 bytes each); of
    # a thin matrix a part of the gram sum and 64 columns (32 bytes each)
    assert z.muon_table_bytes([_mat()]) == 256 + 256 + 32 * (1 + 1)
    assert z.muon_table_bytes([_mat(100, 1000)]) == 256 + -(-49 * 16 // 256) * 256 + 32 * (8 + 16)
    # of others product tiles of 128 x 128: A's upper triangle, X; X's blocks of
    # 64 x 64 (32 bytes each)
    # 300 x 700: 3 x 6 tiles of X, 6 of A's 3 x 3, 5 x 11 blocks; 52500 quads
    assert z.muon_table_bytes([_mat(300, 700)]) == 256 + -(-103 * 16 // 256) * 256 + 32 * (6 + 18 + 55)
    # without u there is nothing to iterate
    assert z.muon_table_bytes([_mat(u=None)]) == 256 + 256
    # a tall matrix has the tiles of its transpose
    assert z.muon_table_bytes([_mat(700, 300)]) == z.muon_table_bytes([_mat(300, 700)])


def test_workspace_bytes_follow_the_plan():
    assert z.muon_workspace_bytes(z.MatrixPlan()) == 0
    assert z.muon_workspace_bytes(_plan()) == 256 + 256 + (1 << 17)
    assert z.muon_workspace_bytes(_plan(n_tiles=33, n_mats=33, area_bytes=1)) == 512 + 512 + 256


def test_matrices_refused():
    def tb(mats, flags=0):
        return z.muon_plan(mats, FAKE, 0, flags=flags)
    assert "at least one" in _einval(lambda: tb([]))
    for rows, cols in ((0, 5), (5, 0), (-1, 5), (1 << 31, 1)):
        assert "must be in" in _einval(lambda: tb([_mat(rows, cols)]))
    assert "smaller side" in _einval(lambda: tb([_mat(32769, 32769, u=FAKE << 2, o=None, m=None, master=None, param=None)]))
    # the table's size needs the shapes only
    for bad in ([], [_mat(0, 5)], [_mat(), _mat(o=None)], [z.matrix(3, 4)], [_mat(ld=19)]):
        _einval(lambda: z.muon_table_bytes(bad))
    assert "ld=19" in _einval(lambda: tb([_mat(ld=19)]))
    assert "ldu=5" in _einval(lambda: tb([_mat(ldu=5)]))
    assert "ldo=-1" in _einval(lambda: tb([_mat(ldo=-1)]))
    assert "shard_offset" in _einval(lambda: tb([_mat(shard_offset=-1)]))
    assert "scale" in _einval(lambda: tb([_mat(scale=math.nan)]))
    assert "scale" in _einval(lambda: tb([_mat(scale=math.inf)]))
    assert "together" in _einval(lambda: tb([_mat(master=None)]))
    assert "together" in _einval(lambda: tb([_mat(param=None)]))
    assert "no buffer" in _einval(lambda: tb([z.matrix(3, 4)]))
    assert "same buffers" in _einval(lambda: tb([_mat(), _mat(at=FAKE + 64 * MB, o=None)]))
    assert "master is not aligned" in _einval(lambda: tb([_mat(master=FAKE + MB + 2)]))
    assert "param_bf16 is not aligned" in _einval(lambda: tb([_mat(param=FAKE + 1)]))
    assert "m is not aligned" in _einval(lambda: tb([_mat(m=FAKE + 2 * MB + 2)]))
    assert _valid([_mat(m=FAKE + 2 * MB + 2)], flags=z.MV_BF16)
    assert "u is not aligned" in _einval(lambda: tb([_mat(u=FAKE + 3 * MB + 2)], flags=z.U_F32))
    assert "unknown flag" in _einval(lambda: tb([_mat()], flags=0x1000))
    assert "unknown flag" in _einval(lambda: z.muon_plan([_mat()], FAKE, 1 << 20, flags=0x100))


def test_overlapping_buffers_refused():
    def tb(mats, flags=0):
        return z.muon_plan(mats, FAKE, 0, flags=flags)
    assert "overlap" in _einval(lambda: tb([_mat(u=FAKE + 2 * MB + 100)]))          # u inside m
    assert "overlap" in _einval(lambda: tb([_mat(o=FAKE + 3 * MB + 2)]))            # o shifted against u
    assert _valid([_mat(o=FAKE + 3 * MB)])                                              # o in place of u
    assert "overlap" in _einval(lambda: tb([_mat(o=FAKE + 3 * MB)], flags=z.U_F32))  # not of an fp32 u
    assert "overlap" in _einval(lambda: tb([_mat(o=FAKE + 3 * MB, ldo=21)]))        # not at another stride
    assert "overlap" in _einval(lambda: tb([_mat(), _mat()]))                       # the same matrix twice

    # blocks of columns of one array of 60 columns
    def cols(first, n, rows=10, first_row=0):
        e = 60 * first_row + first
        return _mat(rows, n, ld=60, ldu=60, ldo=60, param=FAKE + 2 * e, master=FAKE + MB + 4 * e,
                    m=FAKE + 2 * MB + 4 * e, u=FAKE + 3 * MB + 2 * e, o=FAKE + 4 * MB + 2 * e)
    assert _valid([cols(0, 20), cols(20, 20), cols(40, 20)])
    assert _valid([cols(40, 20), cols(0, 40)])
    assert "overlap" in _einval(lambda: tb([cols(0, 21), cols(20, 20)]))
    assert "overlap" in _einval(lambda: tb([cols(20, 20), cols(0, 60, rows=1, first_row=4)]))
    assert _valid([cols(0, 60, rows=4), cols(0, 60, rows=4, first_row=4)])
    # the second begins in the last row's tail and goes on with the columns after it
    assert _valid([cols(0, 30, rows=3), cols(30, 30, rows=3, first_row=1)])
    assert "overlap" in _einval(lambda: tb([cols(10, 50, rows=3), cols(0, 11, rows=2, first_row=2)]))


def test_overlap_decision_matches_element_sets():
    """Random pairs of blocks of one array: refused exactly when they share an
    element (wrapping past a row's end included)."""
    rng = np.random.default_rng(5)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        ld = int(rng.integers(1, 9))
        blocks = []
        for _ in range(2):
            r, c = int(rng.integers(1, 6)), int(rng.integers(1, ld + 1))
            blocks.append((int(rng.integers(0, 40)), r, c))
        sets = [{off + i * ld + j for i in range(r) for j in range(c)} for off, r, c in blocks]
        mats = [z.matrix(r, c, u=FAKE + 2 * off, ldu=ld) for off, r, c in blocks]
        hit = bool(sets[0] & sets[1])
        seen[hit] += 1
        if hit:
            assert "overlap" in _einval(lambda: z.muon_plan(mats, FAKE, 0)), (ld, blocks)
        else:
            assert _valid(mats), (ld, blocks)
    assert min(seen.values()) > 300


def test_plan_refuses_its_table():
    need = z.muon_table_bytes([_mat()])
    assert "NULL" in _einval(lambda: z.muon_plan([_mat()], None), "ZERO1_EWORKSPACE")
    assert "aligned" in _einval(lambda: z.muon_plan([_mat()], FAKE + 128, need), "ZERO1_EWORKSPACE")
    assert "needs" in _einval(lambda: z.muon_plan([_mat()], FAKE, need - 1), "ZERO1_EWORKSPACE")
    L = z.lib()
    assert L.zero1_muon_plan((z.Matrix * 1)(_mat()), 1, 0, FAKE, need, None) == 1


def test_hyper_parameters_refused():
    g, p = [FAKE], _plan()
    def mom(**kw):
        return lambda: z.muon_momentum(g, 0, p, _hp(**kw), stream=0)
    assert "lr" in _einval(mom(lr=-1.0))
    assert "lr" in _einval(mom(lr=math.inf))
    assert "momentum" in _einval(mom(momentum=1.0))
    assert "momentum" in _einval(mom(momentum=math.nan))
    assert "weight_decay" in _einval(mom(weight_decay=-0.1))
    assert "max_norm" in _einval(mom(max_norm=0.0))
    assert "aligned" in _einval(mom(device_scalars=FAKE + 4))
    assert "W=0" in _einval(lambda: z.muon_momentum([], 0, p, _hp(), stream=0))
    assert "begin" in _einval(lambda: z.muon_momentum(g, -1, p, _hp(), stream=0))
    assert "grads[0]" in _einval(lambda: z.muon_momentum([0], 0, p, _hp(), stream=0))
    assert "unknown flag" in _einval(lambda: z.muon_momentum(g, 0, p, _hp(), flags=0x800, stream=0))
    assert "no m" in _einval(lambda: z.muon_momentum(g, 0, _plan(has=13), _hp(), stream=0))
    assert "plan" in _einval(lambda: z.muon_momentum(g, 0, z.MatrixPlan(), _hp(), stream=0))
    def upd(plan=p, **kw):
        return lambda: z.muon_update(plan, _hp(**kw), stream=0)
    assert "lr" in _einval(upd(lr=math.nan))
    assert "no o" in _einval(upd(plan=_plan(has=7)))
    assert "no master" in _einval(upd(plan=_plan(has=14)))
    def step(plan=p, ws=FAKE, ws_bytes=1 << 30, **kw):
        return lambda: z.muon_step(g, 0, plan, _hp(**kw), ws=ws, ws_bytes=ws_bytes, stream=0)
    assert "no u" in _einval(step(plan=_plan(has=11)))
    assert "ns_steps=0" in _einval(step(ns_steps=0))
    assert "needs" in _einval(step(ws_bytes=1000), "ZERO1_EWORKSPACE")
    assert "aligned" in _einval(step(ws=FAKE + 8), "ZERO1_EWORKSPACE")
    assert "NULL" in _einval(step(ws=None), "ZERO1_EWORKSPACE")


def test_iteration_refused():
    p = _plan()
    def orth(**kw):
        return lambda: z.orthogonalize(p, _hp(**kw), ws=FAKE, ws_bytes=1000, stream=0)
    assert "ns_steps=65" in _einval(orth(ns_steps=65))
    assert "ns_steps=-1" in _einval(orth(ns_steps=-1))
    assert "ns_eps" in _einval(orth(ns_eps=-1e-9))
    assert "ns_eps" in _einval(orth(ns_eps=math.inf))
    assert "finite" in _einval(orth(ns_a=math.nan))
    # coefficients whose singular values leave the operands' range
    assert "singular values" in _einval(orth(ns_a=3.5, ns_b=0.0, ns_c=0.0, ns_steps=1))
    assert "singular values" in _einval(orth(ns_a=2.0, ns_b=0.0, ns_c=0.0, ns_steps=2))
    assert "singular values" in _einval(orth(ns_a=13.1, ns_b=-13.0, ns_c=0.0, ns_steps=1))
    # those in use pass (and are then refused for the workspace's size)
    for a, b, c, n in ((3.4445, -4.7750, 2.0315, 64), (1.5, -0.5, 0.0, 20), (1.875, -1.25, 0.375, 64),
                       (2.0, -1.5, 0.5, 10), (1.0, 0.0, 0.0, 5), (2.9, 0.0, 0.0, 1), (0.0, 0.0, 0.0, 3)):
        assert "needs" in _einval(orth(ns_a=a, ns_b=b, ns_c=c, ns_steps=n), "ZERO1_EWORKSPACE"), (a, b, c)


def test_range_check_covers_every_singular_value():
    """Whatever the check lets through stays within it: the largest |p(s)| over
    a fine grid of s, step after step, never passes 3, nor |b s^2 + c s^4| 12."""
    rng = np.random.default_rng(11)
    passed = 0
    for _ in range(400):
        a, b, c = rng.uniform(-3, 4), rng.uniform(-8, 4), rng.uniform(-3, 4)
        steps = int(rng.integers(1, 7))
        msg = None
        with pytest.raises(z.Zero1Error) as e:
            z.orthogonalize(_plan(), _hp(ns_a=a, ns_b=b, ns_c=c, ns_steps=steps), ws=FAKE, ws_bytes=1, stream=0)
        msg = e.value
        top, fits = 1.0, True
        for _ in range(steps):
            s = np.linspace(0, top, 20001)
            q = np.abs(b * s ** 2 + c * s ** 4).max()
            top = np.abs(a * s + b * s ** 3 + c * s ** 5).max()
            fits = q <= 12.0 and top <= 3.0
            if not fits:
                break
        if msg.name == "ZERO1_EWORKSPACE":
            passed += 1
            assert top <= 3.0 + 1e-6 and fits, (a, b, c, steps)
        elif fits:
            assert top > 2.99 or q > 11.99, (a, b, c, steps, msg.message)
    assert passed > 50


def test_scalars_derive():
    s = z.muon_scalars_derive(dict(lr=3e-4, momentum=0.95, weight_decay=0.1, max_norm=0.5))
    assert s.lr == np.float32(3e-4) and s.momentum == np.float32(0.95)
    assert s.decay == np.float32(1.0 - 3e-4 * 0.1) and s.max_norm == 0.5 and s.reserved == 0.0
    assert ctypes.sizeof(z.MuonScalars) == 24
    assert "lr" in _einval(lambda: z.muon_scalars_derive(_hp(lr=-1.0)))


def test_reference_iteration_orthogonalises():
    """The tests' 64-bit iteration does what the operator is for: singular
    values above 0.01 of the norm end within 0.68..1.21, and the singular
    vectors stay."""
    rng = np.random.default_rng(3)
    for shape in ((40, 70), (70, 40), (1, 9)):
        u = rng.standard_normal(shape)
        o = ref.iterate64(u)
        s = np.linalg.svd(o, compute_uv=False)
        assert s.max() < 1.21 and s.min() > 0.68
        U, _, Vt = np.linalg.svd(u, full_matrices=False)
        d = U.T @ o @ Vt.T
        assert np.abs(d - np.diag(np.diag(d))).max() < 1e-9


def test_header_documents_every_muon_flag():
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "zero1.h")).read()
    for name, bit in (("U_F32", z.U_F32), ("NO_NESTEROV", z.NO_NESTEROV)):
        assert f"#define ZERO1_{name}" in src and hex(bit) + "u" in src


def test_clip_arguments_refused():
    g, p = [FAKE], _plan()
    for call in (lambda **kw: z.muon_momentum(g, 0, p, _hp(), stream=0, **kw),
                 lambda **kw: z.muon_step(g, 0, p, _hp(), ws=FAKE, ws_bytes=1 << 30, stream=0, **kw)):
        assert "n_ranks=0" in _einval(lambda: call(rank_sumsq=FAKE))
        assert "info_out" in _einval(lambda: call(info_out=FAKE, n_ranks=1))


def test_sizes_out_of_reach_refused():
    """What no memory holds is refused, not laid out: spans past 2^44 elements,
    more tiles or blocks than a plan or a launch takes."""
    def tb(*mats):
        return lambda: z.muon_table_bytes(list(mats))
    u = dict(u=FAKE, param=None, master=None, m=None, o=None)
    assert "2^44" in _einval(tb(_mat(1 << 20, 3, ld=1 << 30)))
    assert "2^44" in _einval(tb(_mat(1 << 20, 3, ldo=1 << 30)))
    assert "too many elements" in _einval(tb(_mat(32768, (1 << 23))))
    assert "iterated together" in _einval(tb(_mat(1, (1 << 29), **u)))
    assert z.muon_table_bytes([_mat(1, 1 << 28, **u)]) > 0
    # (there is nothing to iterate without u)
    assert z.muon_table_bytes([_mat(1, 1 << 29, u=None)]) > 0
