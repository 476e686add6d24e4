"""The edge cases of the attention and of the policy loss on the kernels that carry their large calls: every test states the
kernel that its shape has to take, so that a change of the rule that chooses cannot leave a kernel untested.  References and
tolerances are those of the operators' own tests."""
import contextlib
import math

import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q
import test_gpu_policy_loss as pl
import test_gpu_prefix_attn as at

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@contextlib.contextmanager
def takes(*kernels):
    """Every one of these kernels is launched inside, and no other one of a choice."""
    every = range(4)
    before = [q.kernel_launch_count(k) for k in every]
    yield
    assert tuple(k for k in every if q.kernel_launch_count(k) > before[k]) == kernels


# ------------------------------------------------------------------ attention
# both segments on tcgen05; the prefix there and the suffixes beside it; the suffixes there and no prefix
BOTH, MIXED, OWN = (q.KERNEL_ATTN_ROWS128,), (q.KERNEL_ATTN_ROWS16, q.KERNEL_ATTN_ROWS128), (q.KERNEL_ATTN_ROWS128,)
SHAPES = [((8, 2, 129, 16, 2, 128, 1000, 700), BOTH), ((8, 2, 129, 16, 2, 64, 1000, 700), BOTH), ((3, 1, 97, 28, 4, 128, 1500, 333), BOTH),
          ((64, 1, 1, 28, 4, 128, 8192, 300), MIXED), ((64, 1, 1, 28, 4, 64, 8192, 300), MIXED), ((4, 1, 200, 8, 2, 128, 0, 512), OWN)]
shapes = pytest.mark.parametrize("shape,kernels", SHAPES)


def lens(shape):
    B, n, Lq, _, _, _, P, S = shape
    return at.spread(n, P // 2, P), at.spread(B, Lq, S)


def test_the_other_kernel_alone():
    with takes(q.KERNEL_ATTN_ROWS16):
        at.check(*at.inputs(8, 1, 1, 28, 4, 128, 512, 300, 1), [500], [300] * 8)


@shapes
@pytest.mark.parametrize("qscale", [0.0, 30.0, 1000.0])
def test_flat_and_peaked(shape, kernels, qscale):
    with takes(*kernels):
        at.check(*at.inputs(*shape, 31, qscale), *lens(shape))


@shapes
@pytest.mark.parametrize("sign", [1, -1])
def test_growing_logits(shape, kernels, sign):
    """Each tile's largest logit exceeds all before it by more than the step at which the maximum is raised, and the reverse."""
    B, n, Lq, Hq, Hkv, D, P, S = shape
    qq, kp, vp, ks, vs = at.inputs(*shape, 32)
    qq.fill_(1.0)
    ramp = lambda t: (sign * torch.linspace(-8, 8, t, device="cuda")).view(1, t, 1, 1).to(torch.bfloat16)  # noqa: E731
    if P:
        kp.copy_(ramp(P).expand_as(kp))
    ks.copy_(ramp(S).expand_as(ks))
    with takes(*kernels):
        at.check(qq, kp, vp, ks, vs, [P] * n, [S] * B)


@shapes
@pytest.mark.parametrize("junk", [NAN, INF, 3e38])
def test_what_lies_beyond_the_lengths_is_not_used(shape, kernels, junk):
    B, n, Lq, _, _, _, P, S = shape
    x = at.inputs(*shape, 33)
    # lengths that end everywhere inside a tile, a full cache among them
    pn, sn = [max(0, P - 1 - 37 * k) for k in range(n)], [S - (k * 29) % (S - Lq + 1) for k in range(B)]
    with takes(*kernels):
        want, wl = at.check(*x, pn, sn)
    for t, ends in ((x[1], pn), (x[2], pn), (x[3], sn), (x[4], sn)):
        for i, m in enumerate(ends):
            t[i, m:] = junk
    with takes(*kernels):
        got, gl = at.check(*x, pn, sn)
    assert torch.equal(got, want) and torch.equal(gl, wl)


@shapes
def test_rows_that_see_nothing(shape, kernels):
    """No prefix; no own tokens; fewer of them than new ones; lengths past the capacities and below zero."""
    B, n, Lq, _, _, _, P, S = shape
    x = at.inputs(*shape, 34)
    own = [(0, S, Lq // 2, 1)[k % 4] for k in range(B)]
    with takes(*kernels):
        out, lse = at.check(*x, [0] * n, own)
    assert bool(torch.isinf(lse[0]).all()) and bool((out[0] == 0).all())
    with takes(*kernels):
        at.check(*x, [P] * n, own)
        at.check(*x, [P] * n, [0] * B)
        want, _ = at.check(*x, [0] + [P] * (n - 1), [0] + [S] * (B - 1))
        got, _ = at.check(*x, [-5] + [1 << 30] * (n - 1), [-1] + [2147483647] * (B - 1))
    assert torch.equal(got, want)


@shapes
def test_layouts(shape, kernels):
    """Queries inside a fused q|k|v row, caches laid out head first, an output with its own strides."""
    B, n, Lq, Hq, Hkv, D, P, S = shape
    _, kp, vp, ks, vs = at.inputs(*shape, 35)
    g = torch.Generator(device="cuda").manual_seed(36)
    qkv = torch.randn(B, Lq, Hq + 2 * Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
    first = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    pn, sn = lens(shape)
    with takes(*kernels):
        want, _ = at.check(qkv[:, :, :Hq].contiguous(), kp, vp, ks, vs, pn, sn)
        got, _ = at.check(qkv[:, :, :Hq], first(kp), first(vp), first(ks), vs, pn, sn)
    assert torch.equal(got, want)
    wide = torch.full((B, Lq, 2 * Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q.qerl_prefix_attention(qkv[:, :, :Hq], kp, vp, ks, vs, at.i32(sn), at.i32(pn), out=wide[:, :, :Hq])
    assert torch.equal(wide[:, :, :Hq], want) and bool((wide[:, :, Hq:] == 7.0).all())


def test_one_cache_for_every_sequence():
    """Stride 0 in the suffix and in the prefix, whichever kernel takes it."""
    shape, kernels = SHAPES[0]
    B, n = shape[:2]
    x = list(at.inputs(*shape, 37))
    for k, m in ((1, n), (2, n), (3, B), (4, B)):
        x[k] = x[k][:1].expand(m, -1, -1, -1)
    pn, sn = lens(shape)
    got, _ = at.check(*x, pn, sn)
    with takes(*kernels):
        want, _ = at.check(x[0], *[t.contiguous() for t in x[1:]], pn, sn)
    assert bool(((got.float() - want.float()).abs() <= 2.0 ** -6 * want.float().abs() + 2.0 ** -8).all())


def test_offsets_past_32_bits():
    """Two sequences 2^31 elements apart in the cache, and a prefix whose keys span more than that."""
    B, n, Lq, Hq, Hkv, D, P, S = shape = (2, 1, 129, 16, 2, 128, 1000, 700)
    qq, kp0, vp0, k0, v0 = at.inputs(*shape, 38)
    far = torch.zeros((1 << 31) + (1 << 28), dtype=torch.bfloat16, device="cuda")
    at_ = lambda t, stride, first: far.as_strided(t.shape, stride, first)  # noqa: E731
    ks, vs = at_(k0, ((1 << 31) - 8, Hkv * D, D, 1), 0), at_(v0, ((1 << 31) - 8, Hkv * D, D, 1), 1 << 20)
    step = (1 << 21) + (1 << 18)
    kp, vp = at_(kp0, (0, step, D, 1), 1 << 18), at_(vp0, (0, step, D, 1), (1 << 18) + 4096)
    assert (P - 1) * step > 1 << 31
    for t, u in ((ks, k0), (vs, v0), (kp, kp0), (vp, vp0)):
        t.copy_(u)
    assert all(torch.equal(t, u) for t, u in ((ks, k0), (vs, v0), (kp, kp0), (vp, vp0)))  # they do not overlap
    with takes(q.KERNEL_ATTN_ROWS128):
        got, _ = at.check(qq, kp, vp, ks, vs, [P], [S, S - 3])
        want, _ = at.check(qq, kp0, vp0, k0, v0, [P], [S, S - 3])
    assert torch.equal(got, want)


@shapes
def test_other_stream_repeats_and_graph(shape, kernels):
    """The same bits on every run, on another stream, and from a captured graph whose lengths move on."""
    B, n, Lq, Hq, Hkv, D, P, S = shape
    x = at.inputs(*shape, 39)
    pn, sn = lens(shape)
    want, wl = at.check(*x, pn, sn)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, gl = at.check(*x, pn, sn)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    plan = q.PrefixAttention(*x[1:], Hq, Lq)
    own, pre, out = at.i32(sn), at.i32(pn), torch.empty_like(x[0])
    plan.run(x[0], own, pre, out=out)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with takes(*kernels), torch.cuda.graph(g):
        plan.run(x[0], own, pre, out=out)
    for step in (0, 1, 77):
        own.copy_(at.i32([max(0, m - step) for m in sn]))
        pre.copy_(at.i32([max(0, m - 2 * step) for m in pn]))
        for _ in range(3):
            out.fill_(NAN)
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, q.qerl_prefix_attention(*x, own, pre))
    assert q.get_error() == 0


# ------------------------------------------------------------------ policy loss
RING = [(160, 40001, torch.bfloat16), (160, 40001, torch.float32), (400, 9001, torch.bfloat16), (77, 100003, torch.float32)]
rings = pytest.mark.parametrize("T,V,dtype", RING)
ring = lambda: takes(q.KERNEL_LOSS_RING)  # noqa: E731


def test_one_cluster_per_row_alone():
    with takes(q.KERNEL_LOSS_ROW):
        pl.check(*pl.make(12, 9000, torch.bfloat16, 40))


@rings
def test_masked_vocabulary(T, V, dtype):
    """Logits at -inf and at the type's lowest value; rows of lowest values; rows that are all -inf."""
    x, ids, old, ref, adv, w = pl.make(T, V, dtype, 41, masked=0.1)
    rows = torch.arange(T, device="cuda")
    keep = torch.zeros(T, V, dtype=torch.bool, device="cuda")
    keep[:, ::3] = True
    keep[rows, ids] = True
    for junk in (-INF, torch.finfo(dtype).min):
        y = torch.where(keep, x, torch.full_like(x, junk))
        lp = torch.log_softmax(y.double(), -1)[rows, ids]
        with ring():
            got = pl.check(y, ids, (lp - 0.05).float(), (lp + 0.1).float(), adv, w)
        assert bool((got[3][~keep] == 0).all())
    # a row of lowest values is a row of zeros (in 64 bits, ln V would drown beside the type's lowest value)
    old = torch.full_like(old, -math.log(V))
    want = pl.reference(torch.zeros_like(x), ids, old, old + 0.1, adv, w, 0.2, 0.28, 0.04, 1.0, 1.0)
    with ring():
        got = q.qerl_policy_loss(torch.full_like(x, torch.finfo(dtype).min), ids, old, adv, w, ref_logp=old + 0.1, clip_low=0.2,
                                 clip_high=0.28, beta=0.04)
    for k, v in zip(("sums", "logp", "entropy", "dlogits"), got):
        pl.close(k, v, want[k])
    gone = torch.zeros(T, dtype=torch.bool, device="cuda")
    gone[2::5] = True
    x, ids, old, ref, adv, w = pl.make(T, V, dtype, 42, masked=0.0)
    x[gone] = -INF
    with ring():
        lp, ent = q.qerl_token_logp(x, ids)
        got = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, beta=0.04)
    assert bool((lp[gone] == -INF).all()) and bool((ent[gone] == 0).all()) and bool(torch.isfinite(lp[~gone]).all())
    rest = q.qerl_policy_loss(x, ids, old, adv, w.masked_fill(gone, 0.0), ref_logp=ref, beta=0.04)
    assert torch.equal(got[0], rest[0]) and torch.equal(got[3], rest[3]) and bool((got[3][gone] == 0).all())


@rings
def test_nan_and_inf_show_in_their_rows_only(T, V, dtype):
    x, ids, old, ref, adv, w = pl.make(T, V, dtype, 43, masked=0.0)
    clean = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, beta=0.04)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    for row, col, v in ((2, 77, NAN), (5, V - 1, INF), (T - 1, 0, NAN), (T // 2, int(ids[T // 2]), INF)):
        x[row, col] = v
        bad[row] = True
    with ring():
        sums, lp, ent, dx = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, beta=0.04)
    assert torch.equal(torch.isnan(lp), bad) and bool(torch.isnan(sums[0]))
    assert torch.equal(lp[~bad], clean[1][~bad]) and torch.equal(dx[~bad], clean[3][~bad])
    assert bool(torch.isnan(dx[bad]).any(-1).all())


@rings
def test_certain_and_impossible_tokens(T, V, dtype):
    """p of the chosen token next to 1 and next to 0, by gaps to 120 nats, and logits of -inf for the chosen one."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(T, V, generator=g, device="cuda") * 0.5).to(dtype)
    ids = torch.randint(1, V, (T,), generator=g, device="cuda")
    rows = torch.arange(T, device="cuda")
    gap = torch.linspace(5, 120, T, device="cuda").to(dtype)
    x[rows, torch.where(rows % 2 == 0, ids, 0)] = gap
    lp = torch.log_softmax(x.double(), -1)[rows, ids]
    adv = torch.where(rows % 3 == 0, -1.5, 1.0)
    w = torch.full((T,), 1.0 / T, device="cuda")
    with ring():
        pl.check(x, ids, lp.float(), (lp + 0.2).float(), adv, w)
    never = rows % 4 == 1
    x[rows[never], ids[never]] = -INF
    with ring():
        lp2, ent = q.qerl_token_logp(x, ids)
        sums, _, _, dx = q.qerl_policy_loss(x, ids, lp.float(), adv, w)
    assert bool((lp2[never] == -INF).all()) and bool(torch.isfinite(lp2[~never]).all()) and bool(torch.isfinite(ent).all())
    assert bool((dx[never] == 0).all()) and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(sums).all())


@rings
def test_rows_that_take_no_part(T, V, dtype):
    """Masks in long runs, ids outside the vocabulary; NaN and Inf there reach nothing."""
    x, ids, old, ref, adv, w = pl.make(T, V, dtype, 44, masked=0.2)
    w[10:T // 2] = 0.0
    ids[-3:] = torch.tensor([-100, V, -1], device="cuda")
    w[-3:] = 1.0 / T
    out = (w == 0) | (ids < 0) | (ids >= V)
    with ring():
        clean = pl.check(x, ids, old, ref, adv, w)
    for junk in (NAN, INF, -INF):
        x[out], old[out], adv[out] = junk, junk, junk
        got = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, clip_low=0.2, clip_high=0.28, beta=0.04)
        assert all(torch.equal(a, b) for a, b in zip(got, clean))
    assert bool((clean[3][out] == 0).all()) and bool((clean[1][out] == 0).all())
    with ring():
        sums, *_ = q.qerl_policy_loss(x, ids, old, adv, torch.zeros_like(w))
    assert sums.tolist() == [0.0] * 4


@rings
def test_ring_repeats_on_another_stream_and_in_a_graph(T, V, dtype):
    """The same bits, second attempts among the rows."""
    x, ids, old, ref, adv, w = pl.make(T, V, dtype, 45)
    x[::7, 3] = 60.0  # (at 90 and more e^(ref - logp) overflows)
    x[::11] = -INF
    kw = dict(ref_logp=ref, beta=0.04, dlogits=torch.empty_like(x), logp=torch.empty_like(old), entropy=torch.empty_like(old),
              sums=torch.empty(4, device="cuda"), ws=q.workspace(q.OP_POLICY_LOSS, T, V, 0, 0))
    with ring():
        want = [t.clone() for t in q.qerl_policy_loss(x, ids, old, adv, w, **kw)]
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(q.qerl_policy_loss(x, ids, old, adv, w, **kw), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = q.qerl_policy_loss(x, ids, old, adv, w, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with ring(), torch.cuda.graph(g):
        got = q.qerl_policy_loss(x, ids, old, adv, w, **kw)
    for t in got:
        t.fill_(NAN)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and q.get_error() == 0


@pytest.mark.parametrize("shape,kernels", [((5, 1, 3, 8, 2, 128, 40, 90), (q.KERNEL_ATTN_ROWS16,)), ((2, 2, 33, 8, 2, 64, 100, 300), (q.KERNEL_ATTN_ROWS16,))]
                         + [SHAPES[k] for k in (0, 1, 2, 5)])
@pytest.mark.parametrize("junk", [NAN, INF, -INF])
def test_values_that_a_new_token_does_not_see(shape, kernels, junk):
    """A value of a later new token that is not finite reaches no earlier row, and no other column of the rows that see it;
    those get the formula's Inf or NaN."""
    B, n, Lq, Hq, Hkv, D, P, S = shape
    x = at.inputs(*shape, 46)
    pn = at.spread(n, P // 2, P)
    sn = [S - (k * 29) % (S - Lq) for k in range(B)]
    with takes(*kernels):
        _, wl = at.check(*x, pn, sn)
    want, _, tol, _ = at.reference(*x, pn, sn, D ** -0.5)
    seen = torch.zeros(B, Lq, Hq, D, dtype=torch.bool, device="cuda")
    for b in range(B):
        for i, j in enumerate(sorted({Lq - 1, Lq // 2, 1, (b * 37) % Lq})):  # new token j, one kv head, every few columns
            hk, cols = (b + i) % Hkv, slice(i, D, 24)
            x[4][b, sn[b] - Lq + j, hk, cols] = junk
            seen[b, j:, hk * (Hq // Hkv):(hk + 1) * (Hq // Hkv), cols] = True
    with takes(*kernels):
        got, lse = torch.full_like(x[0], NAN), torch.full_like(wl, NAN)
        q.PrefixAttention(*x[1:], Hq, Lq).run(x[0], at.i32(sn), at.i32(pn), out=got, lse=lse)
    assert torch.equal(lse, wl)
    assert bool(((got.double() - want).abs() <= tol)[~seen].all())
    there = got[seen].float()
    assert bool((torch.isnan(there) if math.isnan(junk) else there == junk).all())
    assert q.get_error() == 0
