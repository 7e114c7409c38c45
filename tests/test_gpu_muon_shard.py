"""Both optimizers on one rank's shard: AdamW over the tensors, Muon over the weight
matrices, clipped together by the norm of all gradients."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
import synth
import zero_sharded_mixed_zero1_amd as z
from tests import muon_formats as fmt
from tests import muon_ref as ref
from tests.gpu_util import assert_bf16_equal, assert_f32_equal, rel_close, to_dev_u16, to_np_u16, ws_tensor
from tests.test_gpu_muon import env  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

W, RANK = 3, 1
ADAM = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
MUON = dict(lr=2e-3, momentum=0.95, weight_decay=0.1)


@pytest.mark.parametrize("layout", ["matrices last", "matrices between"])
@pytest.mark.parametrize("max_norm", [0.05, 1e9])
def test_one_shard_with_both_optimizers(env, layout, max_norm):  # noqa: F811
    """The shard is cut at tensors' borders.  AdamW's plan tiles a contiguous run of
    it, so tensors in front of the matrices and behind them are two plans, each with
    the run's own `begin`; the sums of squares of all runs make this rank's entry of
    rank_sumsq."""
    torch, dev = env
    front, back = [1000, 8, 3000], [40, 512]
    shapes = [(130, 200), (64, 96), (33, 500)]
    runs = [("adam", front), ("muon", shapes), ("adam", back)]
    if layout == "matrices last":
        runs = [("adam", front + back), ("muon", shapes)]
    begin, at, spans = 11, 0, []
    for kind, items in runs:
        n = sum(int(np.prod(i)) for i in items)
        spans.append((kind, items, at, n))
        at += n
    S = at
    rng = np.random.default_rng(8)
    master0 = (rng.standard_normal(S) * 0.02).astype(np.float32)
    master, m, v = (torch.from_numpy(a.copy()).to(dev) for a in (master0, np.zeros(S, np.float32), np.zeros(S, np.float32)))
    u = torch.zeros(S, dtype=torch.int16, device=dev)
    param = torch.zeros(S, dtype=torch.int16, device=dev)
    parts = torch.zeros(len(spans), dtype=torch.float64, device=dev)
    plans = []
    for kind, items, lo, n in spans:
        offs = lo + np.cumsum([0] + [int(np.prod(i)) for i in items])
        if kind == "adam":
            pieces = [(k, int(o) - lo, param[o:], master[o:], m[o:], v[o:]) for k, o in zip(items, offs)]
            table = ws_tensor(torch, z.mta_table_bytes(pieces), dev)
            plan = z.mta_plan(pieces, table)
            ws = ws_tensor(torch, z.mta_workspace_bytes(plan, W), dev)
        else:
            mats = [z.matrix(*s, shard_offset=int(o), scale=0.2 * max(s) ** 0.5, param=param[o:], master=master[o:],
                             m=m[o:], u=u[o:]) for s, o in zip(items, offs)]
            table = ws_tensor(torch, z.muon_table_bytes(mats), dev)
            plan = z.muon_plan(mats, table)
            ws = ws_tensor(torch, max(z.muon_workspace_bytes(plan), z.workspace_bytes(n, W)), dev)
        plans.append((plan, table, ws))
    others = np.array([0.4, 0.0, 0.7])          # the other ranks' entries
    em, ev, emaster, eparam = np.zeros(S, np.float32), np.zeros(S, np.float32), master0.copy(), np.zeros(S, np.uint16)
    for t in (1, 2):
        G = [synth.bf16(begin + S + 5, synth.grad_key(60 + t, 1, w), 0, 1e-2, 1) for w in range(W)]
        grads = [to_dev_u16(torch, g, dev) for g in G]
        rank_sumsq = torch.from_numpy(others.copy()).to(dev)
        info = torch.zeros(4, dtype=torch.float64, device=dev)
        for k, ((kind, items, lo, n), (plan, _, ws)) in enumerate(zip(spans, plans)):
            if kind == "adam":
                z.mta_reduce(grads, begin + lo, plan, parts[k:], ws=ws)
            else:
                z.shard_reduce(grads, begin + lo, n, sumsq_out=parts[k:], ws=ws)
        z.partials_sum(parts, len(spans), rank_sumsq[RANK:])
        before = master.cpu().numpy()
        for (kind, items, lo, n), (plan, _, ws) in zip(spans, plans):
            if kind == "adam":
                z.mta_update(grads, begin + lo, plan, dict(ADAM, max_norm=max_norm, step=t), rank_sumsq, W, ws=ws)
            else:
                z.muon_step(grads, begin, plan, dict(MUON, max_norm=max_norm), rank_sumsq, W, info_out=info, ws=ws)
        torch.cuda.synchronize()
        g = oracle.shard_reduce([x[begin:begin + S] for x in G])
        entries = others.copy()
        entries[RANK] = oracle.sumsq(g)
        norm = oracle.global_norm(entries)
        clip, coef = oracle.clip_coef(norm, max_norm)
        raw = info.cpu().numpy()
        assert rel_close(float(rank_sumsq[RANK]), entries[RANK], 1e-12) and rel_close(raw[1], norm, 1e-12)
        assert raw[2:3].view(np.float32)[0] == coef and clip == (max_norm < norm)
        got = {k: x.cpu().numpy() for k, x in (("master", master), ("m", m), ("v", v))}
        got["u"], got["param"] = to_np_u16(u), to_np_u16(param)
        for kind, items, lo, n in spans:
            run = slice(lo, lo + n)
            if kind == "adam":
                a = [x[run].copy() for x in (emaster, em, ev, eparam)]
                oracle.adamw(g[run], *a, oracle.adamw_scalars(**ADAM, t=t), clip, coef)
                emaster[run], em[run], ev[run], eparam[run] = a
                for name, want in zip(("master", "m", "v"), a):
                    assert_f32_equal(got[name][run], want, f"{name} t={t}")
                assert_bf16_equal(got["param"][run], a[3], f"param t={t}")
                continue
            gm, eu = ref.momentum32(g[run] * coef if clip else g[run], em[run], MUON["momentum"])
            em[run] = gm
            assert_f32_equal(got["m"][run], gm, f"m t={t}")
            assert_bf16_equal(got["u"][run], ref.bf16(eu), f"u t={t}")
            assert_bf16_equal(got["param"][run], ref.bf16(got["master"][run]), f"param t={t}")
            o = lo
            for s in items:
                e = slice(o, o + s[0] * s[1])
                o = e.stop
                exact = ref.iterate64(ref.widen(got["u"][e]).reshape(s)).ravel()
                eta, delta = MUON["lr"] * 0.2 * max(s) ** 0.5, 1 - MUON["lr"] * MUON["weight_decay"]
                p, size = before[e].astype(np.float64), np.linalg.norm(exact)
                # the update's own roundings and eta times o's, as the header states it
                room = 6 * 2.0 ** -24 * (np.linalg.norm(p) + eta * size) + eta * fmt.stated(s, 5) * size
                assert np.linalg.norm(got["master"][e] - (p - eta * exact) * delta) <= room, (s, t)
            emaster[run] = got["master"][run]
