"""The 4-bit cache's entry points refuse bad arguments on the host before any CUDA call (CPU only)."""
import ctypes as C
import math

import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

FAKE = 1 << 20  # never dereferenced: every call fails its host check first


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


def cache(n=8, T=100, Hkv=4, D=128, stride=(1 << 20, 1 << 16, 36 * 128), ks=1.0, vs=1.0, data=FAKE):
    return q._Kv4Cache(data, n, T, Hkv, D, (C.c_int64 * 3)(*stride), ks, vs)


BAD_CACHES = [(dict(data=None), 1), (dict(ks=0.0), 1), (dict(vs=-1.0), 1), (dict(ks=math.nan), 1), (dict(vs=math.inf), 1), (dict(n=0), 2),
              (dict(T=0), 2), (dict(T=1 << 40), 2), (dict(Hkv=0), 2), (dict(D=96), 2), (dict(stride=(-16, 16, 16)), 2),
              (dict(stride=(8, 16, 16)), 3), (dict(data=FAKE + 8), 3)]


def tokens(L, c, n=3, call="append", k=FAKE, ks=(1024, 512, 128), v=FAKE, vs=(1024, 512, 128), lens=FAKE, counts=None):
    st = C.c_int64 * 3
    c = None if c is None else C.byref(c)
    ks, vs = (None if s is None else st(*s) for s in (ks, vs))
    if call == "append":
        return L.qerl_kv4_append(c, n, k, ks, v, vs, lens, counts, None)
    return L.qerl_kv4_read(c, n, lens, k, ks, v, vs, None)


@pytest.mark.parametrize("call", ["append", "read"])
def test_tokens_refusals(L, call):
    for kw, status in BAD_CACHES:
        assert tokens(L, cache(**kw), call=call) == status, kw
    assert tokens(L, None, call=call) == 1
    for kw, status in ((dict(k=None), 1), (dict(v=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(lens=None), 1), (dict(n=-1), 2),
                       (dict(n=1 << 40), 2), (dict(ks=(1024, -8, 128)), 2), (dict(vs=(1 << 41, 8, 8)), 2), (dict(ks=(1024, 516, 128)), 3),
                       (dict(k=FAKE + 2), 3), (dict(v=FAKE + 8), 3), (dict(lens=FAKE + 2), 3)):
        assert tokens(L, cache(), call=call, **kw) == status, kw
    assert tokens(L, cache(n=1 << 20, Hkv=4096), n=1 << 20, call=call) == 2
    if call == "append":
        assert tokens(L, cache(), counts=FAKE + 1) == 3


def attn(L, B=8, Lq=1, Hq=28, pre=cache(n=2), suf=cache(), q_=FAKE, qs=(4096, 512, 128), os_=(4096, 512, 128), pl=FAKE, sl=FAKE, scale=0.1, out=FAKE,
         lse=None, ws=FAKE, ws_bytes=1 << 40, dims=True):
    st = C.c_int64 * 3
    d = C.byref(q._Kv4AttnDims(B, Lq, Hq, st(*qs), st(*os_))) if dims else None
    p, s = (None if c is None else C.byref(c) for c in (pre, suf))
    return L.qerl_kv4_attention(d, q_, p, pl if pre is not None else None, s, sl, scale, out, lse, ws, ws_bytes, None), L.qerl_kv4_attention_ws_bytes(d, p, s)


def test_attention_refusals(L):
    for kw in (dict(dims=False), dict(q_=None), dict(out=None), dict(sl=None), dict(pre=None, suf=None, sl=None), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e30, suf=cache(ks=1e10)),
               dict(scale=1e-20, suf=cache(ks=1e-30))):
        assert attn(L, **kw)[0] == 1, kw
    for kw, status in BAD_CACHES:
        for side in ("pre", "suf"):
            got, need = attn(L, **{side: cache(**kw)})
            assert got == status and need == 0, (kw, side)
    for kw in (dict(B=0), dict(B=7), dict(Lq=0), dict(Hq=0), dict(Hq=30), dict(Hq=1 << 20), dict(B=1 << 40), dict(Lq=1 << 30), dict(pre=cache(n=3)),
               dict(suf=cache(n=4)), dict(pre=cache(n=2, Hkv=2)), dict(pre=cache(n=2, D=64))):
        got, need = attn(L, **kw)
        assert got == 2 and need == 0, kw
    assert attn(L, qs=(-8, 8, 8))[0] == 2 and attn(L, os_=(1 << 41, 8, 8))[0] == 2
    for kw in (dict(qs=(4096, 512, 132)), dict(os_=(4100, 512, 128)), dict(q_=FAKE + 8), dict(out=FAKE + 2), dict(lse=FAKE + 2),
               dict(pl=FAKE + 1), dict(sl=FAKE + 2), dict(ws=FAKE + 4)):
        assert attn(L, **kw)[0] == 3, kw
    need = attn(L, ws=None)[1]
    assert need >= 8 * 28 * (128 * 4 + 8) * 2  # a part of each kind a row
    assert attn(L, ws=None)[0] == 8 and attn(L, ws_bytes=need - 1)[0] == 8


def test_binding_refuses_other_shapes_and_types(L):
    c = q.Kv4Cache(2, 40, 2, 64, device="cpu")
    lens, k = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    for bad in (k.float(), k[:1], k[:, :, :1], k[..., :32], k.transpose(2, 3)):
        with pytest.raises(AssertionError):
            c.append(bad, bad, lens)
    for bad in (lens.long(), lens[:1]):
        with pytest.raises(AssertionError):
            c.append(k, k, bad)
    with pytest.raises(AssertionError):
        c.append(k, k, lens, counts=lens.long())
    with pytest.raises(AssertionError):
        q.Kv4Cache(2, 40, 2, 64, data=torch.zeros(2, 2, 2, 36 * 128, dtype=torch.uint8))
    with pytest.raises(q.QerlError):
        q.Kv4Attention(c, 3)
