"""The RL-step entry points (prefix attention, policy loss, AdamW) refuse bad arguments on the host before any CUDA
call (CPU only)."""
import ctypes as C
import math

import pytest

import nvfp4_weight_only_quantize_gb300 as q

FAKE = 1 << 20  # never dereferenced: every call fails its host check first


@pytest.fixture(scope="module")
def L():
    q.build()
    return q.lib()


def dims(**kw):
    d = dict(B=8, Lq=1, Hq=28, Hkv=4, D=128, n_prefix=2, P=100, S=50)
    d.update({k: v for k, v in kw.items() if not k.endswith("stride")})
    a = q._AttnDims(*d.values())
    for n in ("q_stride", "out_stride", "k_prefix_stride", "v_prefix_stride", "k_suffix_stride", "v_suffix_stride"):
        setattr(a, n, (C.c_int64 * 3)(*kw.get(n, (4096, 512, 128))))
    return a


def attn(L, d, scale=0.1, ws=FAKE, ws_bytes=1 << 40, **kw):
    p = dict(q=FAKE, kp=FAKE, vp=FAKE, pl=FAKE, ks=FAKE, vs=FAKE, sl=FAKE, out=FAKE, lse=FAKE)
    p.update(kw)
    return L.qerl_prefix_attention(C.byref(d) if d is not None else None, p["q"], p["kp"], p["vp"], p["pl"], p["ks"], p["vs"],
                                   p["sl"], scale, p["out"], p["lse"], ws, ws_bytes, None)


def test_prefix_attention_refusals(L):
    assert attn(L, None) == 1
    assert attn(L, dims(), q=None) == 1 and attn(L, dims(), out=None) == 1
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert attn(L, dims(), scale=scale) == 1
    # a missing cache or length only where its capacity is not 0
    assert attn(L, dims(), kp=None) == 1 and attn(L, dims(), vs=None) == 1 and attn(L, dims(), sl=None) == 1
    for bad in (dict(D=96), dict(D=256), dict(Hkv=3), dict(Hkv=0), dict(B=0), dict(B=7), dict(n_prefix=0), dict(Lq=0), dict(P=-1),
                dict(S=-1), dict(S=1 << 40), dict(k_suffix_stride=(-8, 512, 128))):
        assert attn(L, dims(**bad)) == 2, bad
        if "k_suffix_stride" not in bad:
            assert L.qerl_prefix_attention_ws_bytes(C.byref(dims(**bad))) == 0
    assert attn(L, dims(q_stride=(4096, 512, 132))) == 3
    assert attn(L, dims(v_prefix_stride=(4096, 516, 128))) == 3
    assert attn(L, dims(), q=FAKE + 8) == 3 and attn(L, dims(), ks=FAKE + 2) == 3 and attn(L, dims(), lse=FAKE + 2) == 3
    assert attn(L, dims(), ws=None) == 8 and attn(L, dims(), ws_bytes=0) == 8
    need = L.qerl_prefix_attention_ws_bytes(C.byref(dims()))
    assert attn(L, dims(), ws_bytes=need - 1) == 8 and attn(L, dims(), ws=FAKE + 4) == 3
    assert L.qerl_prefix_attention_ws_bytes(None) == 0


def test_prefix_attention_workspace_holds_every_part(L):
    """At least one FP32 part (o, m, l) per row and segment."""
    d = dims(P=5000, S=3000)
    rows = 8 * 1 * 28
    assert L.qerl_prefix_attention_ws_bytes(C.byref(d)) >= 2 * rows * (128 * 4 + 8)
    assert L.qerl_prefix_attention_ws_bytes(C.byref(dims(P=0, S=0))) > 0


def loss(L, T=4, V=100, ld=100, dtype=1, bits=64, opts=(0.2, 0.2, 0.04, 1.0, 1.0), ldd=100, ws=FAKE, ws_bytes=1 << 30, **kw):
    p = dict(x=FAKE, ids=FAKE, old=FAKE, ref=FAKE, adv=FAKE, w=FAKE, sums=FAKE, logp=FAKE, ent=FAKE, dx=1 << 30)
    p.update(kw)
    o = None if opts is None else C.byref(q._PolicyOpts(*opts))
    return L.qerl_policy_loss(p["x"], dtype, T, V, ld, p["ids"], bits, p["old"], p["ref"], p["adv"], p["w"], o, p["sums"], p["logp"],
                              p["ent"], p["dx"], ldd, ws, ws_bytes, None)


def test_policy_loss_refusals(L):
    for kw in (dict(x=None), dict(ids=None), dict(old=None), dict(adv=None), dict(sums=None), dict(logp=None), dict(opts=None),
               dict(dtype=2), dict(bits=16), dict(T=-1), dict(V=0), dict(ref=None)):
        assert loss(L, **kw) == 1, kw
    inf, nan = math.inf, math.nan
    for o in ((-0.1, 0.2, 0, 1, 1), (1.5, 0.2, 0, 1, 1), (nan, 0.2, 0, 1, 1), (0.2, -0.1, 0, 1, 1), (0.2, inf, 0, 1, 1),
              (0.2, 0.2, -1, 1, 1), (0.2, 0.2, nan, 1, 1), (0.2, 0.2, 0, 0, 1), (0.2, 0.2, 0, -1, 1), (0.2, 0.2, 0, inf, 1),
              (0.2, 0.2, 0, 1, nan), (0.2, 0.2, 0, 1, inf)):
        assert loss(L, opts=o) == 1, o
    assert loss(L, ld=99) == 2 and loss(L, ldd=99) == 2 and loss(L, T=1 << 31) == 2
    assert loss(L, x=FAKE + 1) == 3 and loss(L, dtype=0, x=FAKE + 2) == 3 and loss(L, ids=FAKE + 4) == 3
    assert loss(L, w=FAKE + 2) == 3 and loss(L, sums=FAKE + 1) == 3 and loss(L, dx=(1 << 30) + 1) == 3
    # in place only as a whole
    assert loss(L, dx=FAKE + 2) == 1 and loss(L, dx=FAKE, ldd=128) == 1 and loss(L, dx=FAKE - 4 * 100 * 2 + 2) == 1
    assert loss(L, ws=None) == 8
    need = q.workspace_bytes(q.OP_POLICY_LOSS, 1000, 100, 0, 0)
    assert need >= 1000 * 12 and loss(L, T=1000, dx=1 << 32, ws_bytes=need - 1) == 8
    assert loss(L, ws=FAKE + 4) == 3


def test_token_logp_refusals(L):
    def call(x=FAKE, dtype=1, T=4, V=100, ld=100, ids=FAKE, bits=32, w=None, tau=1.0, logp=FAKE, ent=None):
        return L.qerl_token_logp(x, dtype, T, V, ld, ids, bits, w, tau, logp, ent, None)
    assert call(x=None) == 1 and call(ids=None) == 1 and call(logp=None) == 1 and call(dtype=7) == 1 and call(bits=8) == 1
    assert call(tau=0.0) == 1 and call(tau=math.nan) == 1 and call(T=-1) == 1 and call(V=0) == 1
    assert call(ld=99) == 2 and call(x=FAKE + 1) == 3 and call(ids=FAKE + 2) == 3 and call(ent=FAKE + 1) == 3
    assert call(T=0) == 0  # nothing to do


def tensors(count=1, **kw):
    t = dict(n=1000, param=FAKE, master=None, grad=FAKE, m=FAKE, v=FAKE, m_scale=None, v_scale=None, lr_scale=1.0, weight_decay=0.0)
    t.update(kw)
    return (q._AdamTensor * count)(*[q._AdamTensor(*t.values()) for _ in range(count)])


def plan(L, t, n=None, fmt=(0, 0, 32), ws=FAKE, ws_bytes=1 << 30):
    h = C.c_void_p(123)
    st = L.qerl_adamw_plan(C.cast(t, C.c_void_p) if t is not None else None, len(t) if n is None else n,
                           C.byref(q._AdamFormat(*fmt)) if fmt else None, ws, ws_bytes, C.byref(h))
    assert st == 0 or h.value is None  # no handle beside an error
    return st


def test_adamw_plan_refusals(L):
    assert plan(L, None, n=1) == 1 and plan(L, tensors(), n=0) == 1 and plan(L, tensors(), fmt=None) == 1
    assert L.qerl_adamw_plan(C.cast(tensors(), C.c_void_p), 1, C.byref(q._AdamFormat(0, 0, 32)), FAKE, 1 << 30, None) == 1
    for fmt in ((2, 0, 32), (0, -1, 32), (0, 0, 16)):
        assert plan(L, tensors(), fmt=fmt) == 1
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(master=FAKE), dict(lr_scale=math.nan),
               dict(weight_decay=math.inf)):
        assert plan(L, tensors(**kw)) == 1, kw
    assert plan(L, tensors(), fmt=(1, 0, 32)) == 1  # a bf16 parameter needs its master
    assert plan(L, tensors(), fmt=(0, 0, 8)) == 1   # 8-bit states need their scales
    assert plan(L, tensors(), ws=None) == 8
    for kw in (dict(param=FAKE + 8), dict(grad=FAKE + 4), dict(m=FAKE + 1), dict(v=FAKE + 8)):
        assert plan(L, tensors(**kw)) == 3, kw
    assert plan(L, tensors(m_scale=FAKE + 2, v_scale=FAKE), fmt=(0, 0, 8)) == 3
    t = tensors(3)
    need = L.qerl_adamw_ws_bytes(C.cast(t, C.c_void_p), 3)
    assert need > 0 and plan(L, t, ws_bytes=need - 1) == 8 and plan(L, t, ws=FAKE + 8) == 3
    assert plan(L, tensors(n=-1)) == 2
    neg = tensors(n=-1)
    assert L.qerl_adamw_ws_bytes(C.cast(neg, C.c_void_p), 1) == 0 and L.qerl_adamw_ws_bytes(None, 1) == 0


def test_adamw_step_refusals(L):
    hy = q._AdamHyper(1e-3, 0.9, 0.999, 1e-8, 0.0, 1, 0)
    assert L.qerl_adamw_step(None, C.byref(hy), None, None) == 1
    assert L.qerl_adamw_read_state(None, FAKE, FAKE, 0, None) == 1
    L.qerl_adamw_destroy(None)
    assert q.status_string(10) != q.status_string(99)
