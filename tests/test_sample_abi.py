"""Token sampling refuses bad arguments on the host before any CUDA call (CPU only)."""
import ctypes as C
import math

import pytest

import nvfp4_weight_only_quantize_gb300 as q

FAKE = 1 << 20  # never dereferenced: every call fails its host check first


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


def sample(L, x=FAKE, dtype=1, T=4, V=100, ld=100, u=FAKE, ids=FAKE, lp=FAKE, lq=FAKE, opts=True, tau=1.0, p=1.0, m=0.0, k=0, taus=None, ps=None, ms=None,
           ks=None):
    o = q._SampleOpts(tau, p, m, k, taus, ps, ms, ks)
    return L.qerl_sample(x, dtype, T, V, ld, u, C.byref(o) if opts else None, ids, lp, lq, None)


def test_sample_refusals(L):
    for kw in (dict(x=None), dict(u=None), dict(ids=None), dict(lp=None), dict(lq=None), dict(opts=False), dict(dtype=2), dict(T=-1), dict(V=0),
               dict(ld=99), dict(tau=0.0), dict(tau=-1.0), dict(tau=math.nan), dict(tau=math.inf), dict(p=-0.1), dict(p=1.5), dict(p=math.nan),
               dict(m=-0.1), dict(m=1.5), dict(m=math.nan), dict(k=-1)):
        assert sample(L, **kw) == 1, kw
    for kw in (dict(V=(1 << 20) + 1, ld=1 << 21), dict(T=1 << 30), dict(ld=1 << 41)):
        assert sample(L, **kw) == 2, kw
    for kw in (dict(x=FAKE + 1), dict(x=FAKE + 2, dtype=0), dict(u=FAKE + 2), dict(ids=FAKE + 4), dict(lp=FAKE + 1), dict(lq=FAKE + 2),
               dict(taus=FAKE + 1), dict(ps=FAKE + 2), dict(ms=FAKE + 2), dict(ks=FAKE + 3)):
        assert sample(L, **kw) == 3, kw
    # a row's own settings stand in for the call's
    assert sample(L, tau=math.nan, taus=FAKE, u=FAKE + 2) == 3 and sample(L, p=2.0, ps=FAKE, u=FAKE + 2) == 3
    assert sample(L, m=2.0, ms=FAKE, u=FAKE + 2) == 3 and sample(L, k=-1, ks=FAKE, u=FAKE + 2) == 3
