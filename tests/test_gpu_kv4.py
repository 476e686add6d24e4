"""GPU parity of the 4-bit cache: its quantiser against the definition in 64 bits, its attention against the definition
over the values it holds.

The quantiser's codes are exact where the factor is a power of two: amax / 6 and w / (s f) are then quotients of numbers of
at most 8 and 6 significant bits, which single precision rounds to the same side of every border as the exact ones.

Attention, per output with A = sum_k p_k |v_k| (first order, times 1.02 for the rest):
  - the output's rounding to bf16: 2^-8 |ref|;
  - each probability's rounding to fp16 and that of its product with the value's scale: 2 * 2^-11 A; below fp16's normal
    numbers 2^-25 each, (1 + s) 2^-25 6 v_scale a key, relative to a row's sum of at least 2^4 (its maximum lies 4 octaves
    above the reference at least);
  - the logit's FP32 sum over D products and its scaling: an error of e = (D + 4) 2^-24 scale sum|q||k| (the largest over
    the keys) changes a probability by e, numerator and denominator: 2 e A; ex2 (2^-22) and the FP32 sums over n keys,
    whose partial sums are joined by parts: (2^-21 + 128 2^-24) A.
lse: e + 2^-21 + 128 2^-24 + 2^-22 |lse|."""
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

pytestmark = pytest.mark.gpu
NAN = float("nan")
STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rnd(g, *s):
    return torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def nearest(x, f):
    """x [..., 16 n] in 64 bits on the grid of its blocks."""
    grid, table = torch.tensor(STEPS, dtype=torch.float64, device=x.device), torch.tensor(E4M3, dtype=torch.float64, device=x.device)
    w = x.double().reshape(-1, 16)
    want = w.abs().amax(1, keepdim=True) / (6 * f)
    s = torch.where(table >= want, table, torch.inf).amin(1, keepdim=True).clamp(max=448.0) * f
    d = (w.abs().unsqueeze(-1) / torch.where(s > 0, s, 1.0).unsqueeze(-1) - grid).abs()
    even = torch.arange(8, device=x.device) % 2 == 1
    best = d.amin(-1, keepdim=True)
    at = torch.where(d == best, even.double(), 9.0).argmin(-1)  # of two as near, the even code
    return (grid[at] * s * torch.sign(w)).reshape(x.shape)


# ------------------------------------------------------------------ the cache
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,lens,L", [(1, [1], 1), (33, [33, 1, 17], 1), (100, [100, 64, 31], 31), (100, [70, 33, 32], 32),
                                      (257, [257, 129, 40], 33), (300, [300, 299, 298], 298)])
@pytest.mark.parametrize("kf,vf", [(1.0, 1.0), (2.0 ** -6, 4.0)])
def test_append_and_read(D, T, lens, L, kf, vf):
    g, n, H = gen(T * D + L), len(lens), 3
    cache = q.Kv4Cache(n, T, H, D, kf, vf)
    cache.data.fill_(0xFF)
    k, v = rnd(g, n, L, H, D) * 3, rnd(g, n, L, H, D)
    k[0, 0, 0, :16] = 0  # a block of zeros
    k[0, 0, 1, :16] = torch.tensor([1e30, -1e30] + [5.0] * 14, device="cuda")  # saturates
    cache.append(k, v, i32(lens))
    gk, gv = cache.read(i32(lens), L)
    torch.cuda.synchronize()
    assert q.get_error() == 0
    wk, wv = nearest(k, kf), nearest(v, vf)
    wk[0, 0, 1, :2] = torch.tensor([1.0, -1.0], device="cuda", dtype=torch.float64) * 2688 * kf
    wk[0, 0, 1, 2:16] = nearest(torch.tensor([[2688 * kf] + [5.0] * 15], device="cuda"), kf)[0, 2:]
    for b in range(n):
        from_ = max(0, L - lens[b])  # tokens before position 0 are left out
        assert torch.equal(gk[b, from_:].double(), wk[b, from_:]) and torch.equal(gv[b, from_:].double(), wv[b, from_:])
        assert not gk[b, :from_].any() and not gv[b, :from_].any()


def test_append_keeps_what_was_there():
    """Token by token, in chunks, and at once: the same cache; what lies outside the new tokens keeps its bits."""
    g, T = gen(1), 150
    k, v = rnd(g, 2, T, 2, 128), rnd(g, 2, T, 2, 128)
    whole, steps, chunks = (q.Kv4Cache(2, T, 2, 128) for _ in range(3))
    for c in (whole, steps, chunks):
        c.data.fill_(0x5A)
    whole.append(k, v, i32([T, T]))
    for t in range(T):
        steps.append(k[:, t:t + 1], v[:, t:t + 1], i32([t + 1, t + 1]))
    for a, b in ((0, 7), (7, 40), (40, 41), (41, 150)):
        chunks.append(k[:, a:b], v[:, a:b], i32([b, b]))
    torch.cuda.synchronize()
    assert torch.equal(whole.data, steps.data) and torch.equal(whole.data, chunks.data)
    before = whole.data.clone()
    whole.append(k[:, :1] * 2, v[:, :1] * 2, i32([0, 1]))  # no token; position 0
    torch.cuda.synchronize()
    assert torch.equal(whole.data[0], before[0]) and not torch.equal(whole.data[1], before[1])
    whole.append(k[:, :1], v[:, :1], i32([-5, 1]))
    torch.cuda.synchronize()
    assert torch.equal(whole.data, before)


def test_append_counts_lengths_and_strides():
    g, T, L, H, D = gen(2), 90, 40, 2, 64
    wide_k, wide_v = rnd(g, 3, L, H + 1, D + 8), rnd(g, 3, H, L, D)
    k, v = wide_k[:, :, :H, :D], wide_v.transpose(1, 2)
    store = torch.full((3, 5, H, 36 * D + 16), 0x33, dtype=torch.uint8, device="cuda")
    data = store.permute(0, 2, 1, 3)[:, :, :3, :36 * D]
    cache = q.Kv4Cache(3, T, H, D, data=data)
    counts = i32([40, 0, 13])
    cache.append(k, v, i32([1000, 50, 20]), counts=counts)  # 1000 counts as 90
    gk, gv = cache.read(i32([90, 50, 20]), 13)
    torch.cuda.synchronize()
    assert torch.equal(gk[0].double(), nearest(k[0, 27:40], 1.0)) and torch.equal(gv[0].double(), nearest(v[0, 27:40], 1.0))
    assert torch.equal(gk[2].double(), nearest(k[2, :13], 1.0)) and torch.equal(gv[2].double(), nearest(v[2, :13], 1.0))
    assert bool((data[1] == 0x33).all()) and bool((store[:, 3:] == 0x33).all()) and bool((store[..., 36 * D:] == 0x33).all())
    cache.append(k[:, :0], v[:, :0], i32([5, 5, 5]))  # nothing


def test_read_rounds_other_factors_once():
    g = gen(3)
    k = rnd(g, 1, 40, 1, 128)
    cache = q.Kv4Cache(1, 40, 1, 128, 0.3, 0.7)
    one = q.Kv4Cache(1, 40, 1, 128, data=cache.data)
    cache.append(k, k, i32([40]))
    a, b = cache.read(i32([40]), 40), one.read(i32([40]), 40)
    for x, y, f in zip(a, b, (0.3, 0.7)):
        assert bool(((x.double() - y.double() * f).abs() <= (2.0 ** -8 + 2.0 ** -22) * (y.double() * f).abs()).all())


def test_append_non_finite():
    g = gen(4)
    k, v = rnd(g, 1, 3, 1, 64), rnd(g, 1, 3, 1, 64)
    k[0, 0, 0, 3], k[0, 1, 0, 20], v[0, 2, 0, 63] = NAN, float("inf"), -float("inf")
    cache = q.Kv4Cache(1, 3, 1, 64)
    cache.append(k, v, i32([3]))
    assert q.get_error() == 4 and q.get_error() == 0
    gk, gv = cache.read(i32([3]), 3)
    assert bool(torch.isfinite(gk).all()) and bool(torch.isfinite(gv).all())
    assert gk[0, 0, 0, 3] == 0 and gk[0, 1, 0, 20] == 2688 and gv[0, 2, 0, 63] == -2688
    clean = k.clone()
    clean[0, 0, 0, 3] = 0
    assert torch.equal(gk[0, 0].double(), nearest(clean[0, 0], 1.0))  # a NaN spoils no neighbour


# ------------------------------------------------------------------ attention
def reference(qq, pre, suf, pl, sl, scale, smax):
    """(out, lse, out tolerance, lse tolerance) in float64; pre, suf: (k, v) values or None; smax: the largest scale times factor."""
    B, Lq, Hq, D = qq.shape
    Hkv = (suf or pre)[0].shape[2]
    gs = Hq // Hkv
    out = torch.zeros(B, Lq, Hq, D, dtype=torch.float64, device=qq.device)
    lse = torch.full((B, Lq, Hq), -torch.inf, dtype=torch.float64, device=qq.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        g = b // (B // len(pl)) if pre else 0
        p_n = min(max(pl[g], 0), pre[0].shape[1]) if pre else 0
        s_n = min(max(sl[b], 0), suf[0].shape[1]) if suf else 0
        for h in range(Hkv):
            hs = slice(h * gs, (h + 1) * gs)
            k, v = (torch.cat(([pre[t][g, :p_n, h]] if pre else []) + ([suf[t][b, :s_n, h]] if suf else [])).double() for t in range(2))
            for l in range(Lq):
                see = p_n + max(0, s_n - Lq + 1 + l) if suf else p_n
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
                tol[b, l, hs] = 1.02 * (2.0 ** -8 * out[b, l, hs].abs() + (2.0 ** -10 + 2 * e[:, None] + sums) * A + see * 6 * 2.0 ** -29 * smax)
                ltol[b, l, hs] = 1.02 * (e + sums + 2.0 ** -22 * lse[b, l, hs].abs())
    return out, lse, tol, ltol


def filled(g, n, T, H, D, kf=1.0, vf=0.5):
    """A cache full of tokens, and the values it holds."""
    c = q.Kv4Cache(n, T, H, D, kf, vf)
    full = i32([T] * n)
    c.append(rnd(g, n, T, H, D), rnd(g, n, T, H, D), full)
    return c, c.read(full, T)


def check(qq, pre, suf, pl, sl, scale=None, plan=None, out=None, **kw):
    scale = qq.shape[-1] ** -0.5 if scale is None else scale
    lse = torch.full(qq.shape[:3], NAN, device="cuda")
    out = torch.full_like(qq, NAN).contiguous() if out is None else out
    pc, sc = (None if c is None else c[0] for c in (pre, suf))
    if plan is None:
        plan = q.Kv4Attention(sc, qq.shape[2], qq.shape[1], prefix=pc, scale=scale, batch=qq.shape[0])
        plan.ws.fill_(0xFF)  # NaN everywhere: nothing of it may be read before it is written
    plan.run(qq, None if suf is None else i32(sl), None if pre is None or pl is None else i32(pl), out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert q.get_error() == 0
    if pre is not None and pl is None:
        pl = [pc.T] * pc.n
    smax = max(c._c.v_scale * (1 + 448.0 / 64) for c in (pc, sc) if c is not None)  # scales of unit normal values stay below 7
    ref, rl, tol, ltol = reference(qq, *(None if c is None else c[1] for c in (pre, suf)), pl, sl, scale, smax)
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and bool((out[empty] == 0).all())
    assert bool((~torch.isnan(out)).all())
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).nan_to_num().max())
    lerr = (lse.double() - rl).abs()[~empty]
    assert bool((lerr <= ltol[~empty]).all()), float((lerr / ltol[~empty]).max())
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (7, 7), (28, 4), (15, 1)])
@pytest.mark.parametrize("n,P,pl,S,sl,Lq", [
    (0, 0, None, 1, [1], 1),
    (0, 0, None, 33, [33, 32, 31, 1, 0], 1),
    (1, 31, None, 40, [40, 3], 1),
    (2, 65, [65, 0], 130, [130, 97, 0, 64], 1),
    (2, 100, [33, 99], 70, [5, 70, 32, 4], 4),
    (1, 1, [1], 200, [200, 7, 3], 19),
])
def test_attention(D, Hq, Hkv, n, P, pl, S, sl, Lq):
    g = gen(D + Hq + S)
    pre = filled(g, n, P, Hkv, D, 0.5, 1.0) if n else None
    check(rnd(g, len(sl), Lq, Hq, D) * 1.5, pre, filled(g, len(sl), S, Hkv, D), pl, sl)


@pytest.mark.parametrize("B,n,Hq,Hkv,P,S,Lq,lo", [(24, 3, 28, 4, 700, 900, 1, 1), (2, 1, 40, 8, 3000, 2500, 1, 2000), (70, 1, 16, 2, 40, 33, 1, 0),
                                                 (4, 2, 16, 2, 130, 260, 129, 129), (8, 1, 14, 2, 515, 64, 40, 40)])
def test_attention_over_many_ctas(B, n, Hq, Hkv, P, S, Lq, lo):
    g = gen(B + P)
    pl, sl = ([int(x) for x in torch.randint(a, b + 1, (m,), generator=torch.Generator().manual_seed(B))] for a, b, m in ((P // 2, P, n), (lo, S, B)))
    check(rnd(g, B, Lq, Hq, 128) * 1.5, filled(g, n, P, Hkv, 128), filled(g, B, S, Hkv, 128), pl, sl)


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("n,P,pl,S,sl,Lq,Hq,Hkv", [
    (1, 3000, [2999], 64, [64, 41, 40, 50, 63, 45, 60, 42], 40, 16, 2),  # the prefix there, the own tokens not
    (0, 0, None, 1100, [1100, 129, 600, 1001], 129, 16, 2),  # own tokens, causal
    (2, 1500, [1, 1500], 900, [900, 161, 100, 0], 160, 28, 4),  # both; sequences shorter than their new tokens
    (3, 2000, [2000, 0, 65], 40, [40, 33, 7, 40, 1, 20, 38, 39, 40], 33, 40, 8),
])
def test_attention_of_many_rows(D, n, P, pl, S, sl, Lq, Hq, Hkv):
    """Sizes that take the tcgen05 kernel."""
    g = gen(P + S + D)
    pre = filled(g, n, P, Hkv, D, 0.5, 1.0) if n else None
    before = q.kernel_launch_count(q.KERNEL_KV4_ROWS128)
    check(rnd(g, len(sl), Lq, Hq, D) * 1.5, pre, filled(g, len(sl), S, Hkv, D), pl, sl)
    assert q.kernel_launch_count(q.KERNEL_KV4_ROWS128) == before + 1


@pytest.mark.parametrize("fill", [0xFF, 0x7F])
def test_many_rows_use_nothing_beyond_the_lengths(fill):
    g = gen(21)
    B, S, H, D, sl, Lq = 4, 1000, 2, 128, [999, 700, 641, 130], 129
    k, v = rnd(g, B, S, H, D), rnd(g, B, S, H, D)
    cache = q.Kv4Cache(B, S, H, D)
    cache.data.fill_(fill)
    cache.append(k, v, i32(sl), counts=i32(sl))
    held = tuple(torch.nan_to_num(x) for x in cache.read(i32([S] * B), S))
    before = q.kernel_launch_count(q.KERNEL_KV4_ROWS128)
    qq = rnd(g, B, Lq, 16, D)
    check(qq, None, (cache, held), None, sl)
    assert q.kernel_launch_count(q.KERNEL_KV4_ROWS128) == before + 1
    # a query that is not finite stays in its row; large logits
    plan = q.Kv4Attention(cache, 16, Lq)
    clean = plan.run(qq, i32(sl)).clone()
    bad = qq.clone()
    bad[1, 7, 3, 5], bad[2, 128, 15, 0] = NAN, float("inf")
    got = plan.run(bad, i32(sl))
    same = torch.ones(B, Lq, 16, dtype=torch.bool, device="cuda")
    same[1, 7, 3] = same[2, 128, 15] = False
    assert torch.equal(got[same], clean[same]) and bool(torch.isnan(got[~same]).all())
    check(qq * 60, None, (cache, held), None, sl, plan=plan)


def test_prefix_alone_and_scale():
    g = gen(7)
    pre = filled(g, 2, 90, 2, 128)
    check(rnd(g, 6, 2, 8, 128), pre, None, [90, 41], None, scale=0.3)
    check(rnd(g, 6, 2, 8, 128), pre, None, None, None, scale=1e-3)


def test_large_logits():
    """Rows whose weights sit on one key, and maxima that grow from tile to tile."""
    g = gen(8)
    suf = filled(g, 2, 300, 2, 128)
    check(rnd(g, 2, 1, 8, 128) * 60, None, suf, None, [300, 177])
    k = rnd(g, 2, 300, 2, 128) * (1 + torch.arange(300, device="cuda").view(1, 300, 1, 1) / 10).to(torch.bfloat16)
    suf[0].append(k, rnd(g, 2, 300, 2, 128), i32([300, 300]))
    check(rnd(g, 2, 1, 8, 128) * 2, None, (suf[0], suf[0].read(i32([300, 300]), 300)), None, [300, 255])


@pytest.mark.parametrize("fill", [0xFF, 0x7F, 0x00])
def test_what_lies_beyond_the_lengths_is_not_used(fill):
    g = gen(9)
    B, S, H, D, sl = 3, 100, 2, 128, [37, 64, 1]
    k, v = rnd(g, B, S, H, D), rnd(g, B, S, H, D)
    cache = q.Kv4Cache(B, S, H, D)
    cache.data.fill_(fill)
    cache.append(k, v, i32(sl), counts=i32(sl))
    held = cache.read(i32([S] * B), S)
    held = tuple(torch.nan_to_num(x) for x in held)
    for Lq in (1, 3):
        check(rnd(g, B, Lq, 8, D), None, (cache, held), None, sl)


def test_strides_and_untouched_rows():
    g = gen(10)
    suf = filled(g, 2, 80, 2, 64)
    wide = rnd(g, 3, 2, 10, 96)
    big = torch.full((2, 3, 9, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[:, 1:, :8, :64]
    check(wide[:2, :, :8, :64], None, suf, None, [80, 33], out=out)
    assert bool((big[:, 0] == 7).all()) and bool((big[:, :, 8] == 7).all()) and bool((big[..., 64:] == 7).all())


def test_a_query_that_is_not_finite_stays_in_its_row():
    g = gen(11)
    suf = filled(g, 1, 70, 1, 128)
    qq = rnd(g, 1, 1, 8, 128)
    clean, _ = check(qq, None, suf, None, [70])
    qq[0, 0, 3, 5], qq[0, 0, 6, 0] = NAN, float("inf")
    plan = q.Kv4Attention(suf[0], 8)
    out = plan.run(qq, i32([70]))
    bad = torch.tensor([3, 6], device="cuda")
    good = torch.tensor([0, 1, 2, 4, 5, 7], device="cuda")
    assert torch.equal(out[0, 0, good], clean[0, 0, good]) and bool(torch.isnan(out[0, 0, bad]).all())


def test_repeats_and_graph_and_stream():
    g = gen(12)
    pre, suf = filled(g, 2, 500, 4, 128), filled(g, 16, 300, 4, 128)
    qq, sl, pl = rnd(g, 16, 1, 28, 128), i32([300 - 11 * i for i in range(16)]), i32([500, 413])
    plan = q.Kv4Attention(suf[0], 28, prefix=pre[0])
    out, lse = torch.empty_like(qq), torch.empty(16, 1, 28, device="cuda")
    plan.run(qq, sl, pl, out=out, lse=lse)
    first, first_lse = out.clone(), lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            plan.run(qq, sl, pl, out=out, lse=lse)
            assert torch.equal(out, first) and torch.equal(lse, first_lse)
        k = torch.zeros(16, 1, 4, 128, dtype=torch.bfloat16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):  # append and attention of one step, lengths on the device
            suf[0].append(k, k, sl)
            plan.run(qq, sl, pl, out=out, lse=lse)
    torch.cuda.synchronize()
    new = suf[0].read(i32([300] * 16), 300)
    for step in range(3):
        sl.add_(-7)
        k.copy_(rnd(g, 16, 1, 4, 128))
        graph.replay()
        torch.cuda.synchronize()
        new = suf[0].read(i32([300] * 16), 300)
        ref, rl, tol, _ = reference(qq, pre[1], new, [500, 413], sl.tolist(), 128 ** -0.5, 4.0)
        assert bool(((out.double() - ref).abs() <= tol).all())
    q.set_launch_chaining(False)
    try:
        plan.run(qq, sl, pl, out=first, lse=first_lse)
    finally:
        q.set_launch_chaining(True)
    assert torch.equal(out, first) and torch.equal(lse, first_lse)
    late = plan.run(qq, sl, pl, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(late, first)


def test_offsets_past_32_bits():
    """Sequences, heads and tiles that lie more than 4 GB into the cache."""
    g = gen(13)
    D, T, H = 128, 70, 2
    base = torch.zeros(9 << 30, dtype=torch.uint8, device="cuda")
    for strides in ((4 << 30, 36 * D * 4, 36 * D), (36 * D * 4, 4 << 30, 36 * D), (36 * D * 4, 36 * D * 16, 2 << 30)):
        data = torch.as_strided(base, (2, H, 3, 36 * D), strides + (1,))
        c = q.Kv4Cache(2, T, H, D, data=data)
        c.append(rnd(g, 2, T, H, D), rnd(g, 2, T, H, D), i32([T, T]))
        check(rnd(g, 2, 1, 8, D), None, (c, c.read(i32([T, T]), T)), None, [70, 66])


def test_one_call_of_a_step():
    """A step of a rollout: the linears' keys and values into the cache, attention over prompt and answer."""
    g = gen(14)
    pre = q.Kv4Cache(2, 64, 2, 128)
    own = q.Kv4Cache(8, 40, 2, 128)
    pk, pv = rnd(g, 2, 64, 2, 128), rnd(g, 2, 64, 2, 128)
    pl = [64, 21]
    pre.append(pk, pv, i32(pl), counts=i32(pl))
    plan = q.Kv4Attention(own, 14, prefix=pre)
    for t in range(1, 36, 7):
        own.append(rnd(g, 8, 1 if t == 1 else 7, 2, 128), rnd(g, 8, 1 if t == 1 else 7, 2, 128), i32([t] * 8))
        qq = rnd(g, 8, 1, 14, 128)
        check(qq, (pre, pre.read(i32([64, 64]), 64)), (own, own.read(i32([40] * 8), 40)), pl, [t] * 8, plan=plan)
