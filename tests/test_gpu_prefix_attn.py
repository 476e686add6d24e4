"""GPU parity of the attention over shared prefixes against the definition in 64 bits.

Tolerance, per output with A = sum_k p_k |v_k| (first order, times 1.02 for the rest):
  - the output's rounding to bf16: 2^-8 |ref|;
  - each probability's rounding to bf16: 2^-8 p, together 2^-8 A;
  - the logit's FP32 sum over D products and its scaling: an error of e = (D + 4) 2^-24 scale sum|q||k| (the largest over
    the keys) changes a probability by e, numerator and denominator: 2 e A; ex2 (2^-22) and the FP32 sums over n keys,
    whose partial sums are joined by chunks: (2^-21 + 128 2^-24) A.
lse: e + 2^-21 + 128 2^-24 + 2^-22 |lse|."""
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

pytestmark = pytest.mark.gpu
NAN = float("nan")


def reference(qq, kp, vp, ks, vs, pl, sl, scale):
    """(out, lse, out tolerance, lse tolerance) in float64."""
    B, Lq, Hq, D = qq.shape
    n, P, Hkv, _ = kp.shape
    gs, G = Hq // Hkv, B // n
    out = torch.zeros(B, Lq, Hq, D, dtype=torch.float64, device=qq.device)
    lse = torch.full((B, Lq, Hq), -torch.inf, dtype=torch.float64, device=qq.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        p_n, s_n = min(max(pl[b // G], 0), P), min(max(sl[b], 0), ks.shape[1])
        for h in range(Hkv):
            hs = slice(h * gs, (h + 1) * gs)
            k = torch.cat([kp[b // G, :p_n, h], ks[b, :s_n, h]]).double()
            v = torch.cat([vp[b // G, :p_n, h], vs[b, :s_n, h]]).double()
            for l in range(Lq):
                see = p_n + max(0, s_n - Lq + 1 + l)
                if see == 0:
                    continue
                x = qq[b, l, hs].double()
                a = scale * (x @ k[:see].T)
                e = ((D + 4) * 2.0 ** -24 * scale * (x.abs() @ k[:see].abs().T)).amax(1)
                lse[b, l, hs] = torch.logsumexp(a, 1)
                p = torch.exp(a - lse[b, l, hs, None])
                out[b, l, hs] = p @ v[:see]
                A = p @ v[:see].abs()
                sums = 2.0 ** -21 + 128 * 2.0 ** -24
                tol[b, l, hs] = 1.02 * (2.0 ** -8 * out[b, l, hs].abs() + (2.0 ** -8 + 2 * e[:, None] + sums) * A) + 1e-30
                ltol[b, l, hs] = 1.02 * (e + sums + 2.0 ** -22 * lse[b, l, hs].abs())
    return out, lse, tol, ltol


def inputs(B, n, Lq, Hq, Hkv, D, P, S, seed, qscale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    return r(B, Lq, Hq, D) * qscale, r(n, P, Hkv, D), r(n, P, Hkv, D), r(B, S, Hkv, D), r(B, S, Hkv, D)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(qq, kp, vp, ks, vs, pl, sl, scale=None, plan=None, **kw):
    scale = qq.shape[-1] ** -0.5 if scale is None else scale
    lse = torch.full(qq.shape[:3], NAN, device="cuda")
    out = torch.full_like(qq, NAN).contiguous()
    if plan is None:
        plan = q.PrefixAttention(kp, vp, ks, vs, qq.shape[2], qq.shape[1], scale)
        plan.ws.fill_(0xFF)  # NaN everywhere: nothing of it may be read before it is written
    plan.run(qq, i32(sl), None if pl is None else i32(pl), out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert q.get_error() == 0
    pl = [kp.shape[1]] * kp.shape[0] if pl is None else pl
    ref, rl, tol, ltol = reference(qq, kp, vp, ks, vs, pl, sl, scale)
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and bool((out[empty] == 0).all())
    assert bool((~torch.isnan(out)).all())
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    lerr = (lse.double() - rl).abs()[~empty]
    assert bool((lerr <= ltol[~empty]).all()), float((lerr / ltol[~empty]).max())
    return out, lse


def spread(n, lo, hi):
    return [lo + (k * 2654435761 + 97) % (1 << 32) * (hi - lo + 1) // (1 << 32) for k in range(n)]


# (B, n_prefix, Lq, Hq, Hkv, D, P, S): one token of one sequence; odd sizes; every head layout; many rows on one prefix
@pytest.mark.parametrize("B,n,Lq,Hq,Hkv,D,P,S", [
    (1, 1, 1, 1, 1, 128, 1, 1), (1, 1, 1, 28, 4, 128, 512, 1), (3, 1, 1, 28, 4, 128, 129, 65), (8, 8, 1, 16, 2, 128, 100, 77),
    (6, 3, 1, 40, 8, 128, 333, 200), (5, 1, 1, 8, 8, 64, 63, 17), (4, 2, 1, 20, 1, 64, 70, 130), (64, 1, 1, 28, 4, 128, 1000, 40),
    (64, 1, 1, 16, 2, 64, 2500, 9), (40, 2, 1, 40, 8, 128, 700, 300), (2, 1, 1, 17, 1, 128, 300, 300)])
def test_single_tokens(B, n, Lq, Hq, Hkv, D, P, S):
    check(*inputs(B, n, Lq, Hq, Hkv, D, P, S, B + P), spread(n, (P + 1) // 2, P), spread(B, 1, S))


@pytest.mark.parametrize("B,n,Lq,Hq,Hkv,D,P,S", [
    (2, 1, 2, 28, 4, 128, 65, 7), (3, 1, 5, 16, 2, 128, 257, 64), (2, 2, 33, 8, 2, 64, 100, 90), (4, 2, 130, 8, 2, 128, 400, 131),
    (1, 1, 300, 8, 8, 128, 0, 300), (2, 1, 67, 28, 4, 64, 1023, 200)])
def test_several_tokens_are_causal(B, n, Lq, Hq, Hkv, D, P, S):
    check(*inputs(B, n, Lq, Hq, Hkv, D, P, S, B + S), spread(n, P // 2, P), spread(B, Lq, S))


def test_rows_that_see_nothing():
    """No prefix and no suffix: zeros and -inf; fewer tokens in the cache than new ones: the first rows see only the prefix."""
    x = inputs(4, 2, 3, 8, 2, 128, 50, 20, 1)
    out, lse = check(*x, [0, 30], [0, 2, 0, 1])
    assert bool(torch.isinf(lse[0]).all()) and not bool(torch.isinf(lse[2:]).any())
    x = inputs(40, 1, 1, 28, 4, 128, 200, 20, 2)
    check(*x, [0], [0] * 20 + [20] * 20)
    check(*x, [200], [0] * 40)
    # capacities of zero
    x = inputs(4, 2, 1, 8, 2, 64, 0, 20, 3)
    check(*x, None, [0, 1, 16, 20])
    x = inputs(4, 2, 1, 8, 2, 64, 40, 0, 4)
    check(*x, [40, 0], [0, 0, 0, 0])
    x = inputs(2, 2, 1, 8, 2, 64, 0, 0, 5)
    check(*x, None, [0, 0])


@pytest.mark.parametrize("B,n,Lq,P,S", [(6, 2, 1, 200, 130), (64, 1, 1, 500, 33), (2, 1, 70, 300, 150)])
@pytest.mark.parametrize("junk", [NAN, float("inf"), 3e38])
def test_what_lies_beyond_the_lengths_is_not_used(B, n, Lq, P, S, junk):
    x = inputs(B, n, Lq, 28, 4, 128, P, S, 7)
    pl, sl = spread(n, P // 3, P - 1), spread(B, Lq, S - 1)
    want, wl = check(*x, pl, sl)
    for t, lens in ((x[1], pl), (x[2], pl), (x[3], sl), (x[4], sl)):
        for i, m in enumerate(lens):
            t[i, m:] = junk
    got, gl = check(*x, pl, sl)
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_lengths_are_taken_into_the_capacity():
    x = inputs(4, 2, 1, 8, 2, 128, 40, 30, 8)
    want, _ = check(*x, [40, 0], [30, 0, 30, 7])
    got, _ = check(*x, [1 << 30, -5], [31, -1, 2147483647, 7])
    assert torch.equal(got, want)


@pytest.mark.parametrize("qscale", [0.0, 30.0, 1000.0])
def test_flat_and_peaked(qscale):
    """Uniform weights; one key that takes all, in whichever segment it lies."""
    x = inputs(40, 1, 1, 28, 4, 128, 700, 300, 9, qscale)
    check(*x, [700], spread(40, 1, 300))


def test_growing_logits():
    """Each tile's largest logit exceeds all before it, and the reverse: every rescaling happens."""
    B, P, S = 40, 1024, 256
    qq, kp, vp, ks, vs = inputs(B, 1, 1, 8, 2, 128, P, S, 10)
    qq.fill_(1.0)
    for sign in (1, -1):
        ramp = lambda n: (sign * torch.linspace(-4, 4, n, device="cuda")).view(1, n, 1, 1).to(torch.bfloat16)  # noqa: E731
        kp.copy_(ramp(P).expand_as(kp))
        ks.copy_(ramp(S).expand_as(ks))
        check(qq, kp, vp, ks, vs, [P], [S] * B)


def test_layouts():
    """Queries inside a fused q|k|v row, caches laid out head first, an output with its own strides."""
    B, n, Hq, Hkv, D, P, S = 40, 1, 28, 4, 128, 260, 70
    _, kp, vp, ks, vs = inputs(B, n, 1, Hq, Hkv, D, P, S, 11)
    g = torch.Generator(device="cuda").manual_seed(12)
    qkv = torch.randn(B, 1, Hq + 2 * Hkv, D, generator=g, device="cuda", dtype=torch.bfloat16)
    head_first = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    want, _ = check(qkv[:, :, :Hq].contiguous(), kp, vp, ks, vs, [P], [S] * B)
    got, _ = check(qkv[:, :, :Hq], head_first(kp), head_first(vp), head_first(ks), vs, [P], [S] * B)
    assert torch.equal(got, want)
    wide = torch.full((B, 1, 2 * Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    q.qerl_prefix_attention(qkv[:, :, :Hq], kp, vp, ks, vs, i32([S] * B), out=wide[:, :, :Hq])
    assert torch.equal(wide[:, :, :Hq], want) and bool((wide[:, :, Hq:] == 7.0).all())


def test_one_cache_tensor_shared_by_every_sequence():
    """Stride 0: the same suffix for every sequence."""
    x = list(inputs(6, 1, 1, 8, 2, 128, 100, 90, 13))
    one = x[3][:1].clone()
    x[3] = one.expand(6, -1, -1, -1)
    check(*x, [100], spread(6, 1, 90))


def test_offsets_past_32_bits():
    """Sequences 2^31 elements apart in the cache, and a prefix whose last keys lie past 2^31 elements."""
    B, Hq, Hkv, D, S = 3, 8, 2, 128, 40
    far = torch.zeros((1 << 31) * 2 + (1 << 20), dtype=torch.bfloat16, device="cuda")
    qq, _, _, k0, v0 = inputs(B, 1, 1, Hq, Hkv, D, 1, S, 14)
    ks = far.as_strided((B, S, Hkv, D), ((1 << 31) - 8, Hkv * D, D, 1))
    vs = far.as_strided((B, S, Hkv, D), ((1 << 31) - 8, Hkv * D, D, 1), 1 << 16)
    ks.copy_(k0), vs.copy_(v0)
    P = 70
    kp = far.as_strided((1, P, Hkv, D), (0, 1 << 25, D, 1), 1 << 17)
    vp = far.as_strided((1, P, Hkv, D), (0, 1 << 25, D, 1), 1 << 18)
    kp.normal_(), vp.normal_()
    check(qq, kp, vp, ks, vs, [P], [S, 1, S - 3])
    del far


def test_long_prefix():
    """40 000 keys for one and for 48 sequences."""
    for B in (1, 48):
        check(*inputs(B, 1, 1, 4, 1, 128, 40000, 10, 15), [39999], [10] * B)


def test_other_stream_repeats_and_graph():
    """The same bits on every run, on another stream, and from a captured graph whose lengths move on."""
    x = inputs(40, 1, 1, 28, 4, 128, 900, 200, 16)
    sl = spread(40, 1, 200)
    want, wl = check(*x, [900], sl)
    for _ in range(3):
        got, gl = check(*x, [900], sl)
        assert torch.equal(got, want) and torch.equal(gl, wl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = check(*x, [900], sl)
    assert torch.equal(got, want)
    plan = q.PrefixAttention(*x[1:], 28)
    lens, out = i32(sl), torch.empty_like(x[0])
    plan.run(x[0], lens, out=out)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        plan.run(x[0], lens, out=out)
    for step in (0, 1):
        lens.copy_(i32([max(1, n - step) for n in sl]))
        out.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        fresh = q.qerl_prefix_attention(*x, i32([max(1, n - step) for n in sl]))
        assert torch.equal(out, fresh)


@pytest.mark.parametrize("D", [64, 128])
def test_many_short_units(D):
    """More row and key tiles than there are SMs, of every length: tiles in pairs and alone, halves that end a tile apart."""
    B, Lq, Hq, Hkv, P, S = 8, 129, 16, 2, 1000, 700
    qq, kp, vp, ks, vs = inputs(B, 2, Lq, Hq, Hkv, D, P, S, 21)
    sl = [129, 700, 0, 257, 640, 300, 513, 384]
    pl = [1000, 130]
    plan = q.PrefixAttention(kp, vp, ks, vs, Hq, Lq, D ** -0.5)
    first, lse = check(qq, kp, vp, ks, vs, pl, sl, plan=plan)
    for _ in range(300):
        out, again = torch.full_like(first, NAN), torch.full_like(lse, NAN)
        plan.run(qq, i32(sl), i32(pl), out=out, lse=again)
        assert torch.equal(out, first) and torch.equal(again, lse)
    assert q.get_error() == 0
