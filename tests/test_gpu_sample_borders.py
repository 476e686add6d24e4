"""Token sampling where borders are near and errors alike: a few thousand tokens that stand out over a tail of one repeated
value, whose every mass is off by the same amount in single precision.  The settings are chosen such that the
border of what is kept, or the draw, comes to within 1e-6 of the tail's mass of where the next token begins.

The library counts p in units of 2^-42 of the largest, off by at most one unit and 2^-40: all V tokens together move a border by
no more than V 2^-42 of the largest p and 2^-40 of the sum.  The reference is the definition in 64 bits; no case lies nearer than
NEAREST of the sum, which is that for the smallest sum here (120 times the largest p), and a tenth."""
import math

import numpy as np
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

pytestmark = pytest.mark.gpu
V, OUT, TOP = 131072, 3500, 140
NEAREST = 1.1 * (V * 2.0 ** -42 / 120 + 2.0 ** -40)


def tails():
    """bf16 values 16.5 to 20 octaves below 0 whose exponent rounds furthest in single precision, down and up."""
    x = -np.arange(11.5, 13.8, 0.0625)
    y = x * np.log2(np.e)
    off = np.float32(y).astype(np.float64) - y
    order = np.argsort(off)
    return [float(x[i]) for i in (*order[:4], *order[-4:])]


def row(tail, share):
    """Logits (bf16 values, 64 bits) of one row: TOP tokens near 0, OUT tokens that hold all but `share` of the rest, spread over
    the row in falling order, and the tail."""
    x = np.full(V, tail)
    w = (V - OUT - TOP) * math.exp(tail) * (1 - share) / share / OUT  # a token's mass
    at = np.linspace(0, V - 1, OUT + TOP).astype(int)
    rng = np.random.default_rng(0)
    out = np.sort(math.log(w) + 0.3 * rng.standard_normal(OUT))[::-1]
    x[at] = np.concatenate([-0.002 * np.arange(TOP), out])
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


def ordered(x):
    """(tokens in order of probability, their masses, the masses' sums up to each)."""
    v = x.double().numpy()
    order = np.argsort(-v, kind="stable")
    m = np.exp(v[order])
    return order, m, np.cumsum(m.astype(np.longdouble)).astype(np.float64)


def nearest_settings(target, lo, hi, how_many, reach):
    """float32 numbers nearest to some of `target`, with |difference| within (NEAREST, reach), spread over the list."""
    t = target[(target > lo) & (target < hi)]
    f = t.astype(np.float32)
    near = np.abs(f.astype(np.float64) - t)
    f = f[(near < reach) & (near > NEAREST)]
    return f[:: max(1, len(f) // how_many)][:how_many]


def run(x, n, u, **kw):
    return [t.cpu() for t in q.qerl_sample(x.cuda().repeat(n, 1), torch.tensor(u, device="cuda"), **kw)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tail", tails())
@pytest.mark.parametrize("share", [0.2, 0.9])
def test_nucleus(dtype, tail, share):
    x = row(tail, share)
    order, m, upto = ordered(x)
    Z, below = upto[-1], m[TOP + OUT:].sum()
    assert Z > 120 * m[0]
    ps = nearest_settings(upto / Z, upto[TOP + 10] / Z, upto[TOP + OUT - 10] / Z, 200, 1e-6 * below / Z)
    assert len(ps) >= 50
    ids, _, logq = run(x.to(dtype), len(ps), [1 - 2.0 ** -24] * len(ps), top_p=torch.tensor(ps, device="cuda"))
    wrong = []
    for i, p in enumerate(ps):
        n = int((upto < float(p) * Z).sum()) + 1  # kept
        kept = np.sort(order[:n])
        c = np.cumsum(np.exp(x.double().numpy()[kept]).astype(np.longdouble))
        want = kept[int((c <= (1 - 2.0 ** -24) * c[-1]).sum())]
        if int(ids[i]) != want:
            wrong.append((i, float(p), int(ids[i]), int(want)))
    assert not wrong, (len(wrong), len(ps), wrong[:3])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tail", tails()[::3])
@pytest.mark.parametrize("share", [0.2, 0.9])
@pytest.mark.parametrize("cut", [dict(), dict(top_p=0.98)])
def test_draws(dtype, tail, share, cut):
    x = row(tail, share)
    order, m, upto = ordered(x)
    kept = np.sort(order[:int((upto < float(np.float32(cut.get("top_p", 2.0))) * upto[-1]).sum()) + 1])
    c = np.cumsum(np.exp(x.double().numpy()[kept]).astype(np.longdouble)).astype(np.float64)
    assert c[-1] > 120 * m[0]
    us = nearest_settings(c / c[-1], 0.01, 0.999, 300, 1e-7)
    assert len(us) >= 100
    ids, _, _ = run(x.to(dtype), len(us), [float(u) for u in us], **cut)
    want = [int(kept[int((c <= float(u) * c[-1]).sum())]) for u in us]
    wrong = [(i, float(us[i]), int(ids[i]), w) for i, w in enumerate(want) if int(ids[i]) != w]
    assert not wrong, (len(wrong), len(us), wrong[:3])
