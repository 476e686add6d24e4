"""GPU parity of the multi-tensor AdamW step.

FP32 states against float64, u = 2^-24: m is two products and a sum of rounded terms (3 u (|b1 m| + |c1 g|)), v likewise with
one more product (4 u v), the step s = lr / bc1 m / (sqrt(v) rs2 + eps) adds at most 12 u |s| (division to 2 units, root,
product and sum) to what m and v bring, 4 u |s| (1 + (|b1 m| + |c1 g|) / |m|), and p (1 - lr wd) - s rounds thrice: 3 u (|p| + |s|).
The clip's factor is right to one unit: every g is off by 2 u more.  A bf16 param is its master, rounded.

8-bit states: the kernel rounds every product, quotient and root by itself, so numpy in float32 must give the same codes and
scales bit for bit; Philox and the codes are written here from their definitions."""
import numpy as np
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
B1, B2, EPS = 0.9, 0.999, 1e-8
F = np.float32


def philox(n, tensor, step, seed):
    """Philox4x32-10: the word of each of n elements."""
    g = np.arange((n + 3) // 4, dtype=np.uint64)
    m = np.uint64(0xFFFFFFFF)
    c = [g & m, g >> np.uint64(32), np.full_like(g, tensor), np.full_like(g, step)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & m, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).reshape(-1)[:n]


def value(code, bits):
    e, f = code >> bits, (code & ((1 << bits) - 1)) / (1 << bits)
    return np.where(e > 0, (1 + f) * 2.0 ** (e - 7.0), f * 2.0 ** -6)


def decode_m(code, scale):
    """float32 values, the block's scale times the code's value in one rounding."""
    s = np.repeat(scale, 256)[:code.size]
    return np.where(code > 127, F(-1), F(1)) * (value(code & 127, 4).astype(F) * s)


def decode_s(code, scale):
    return value(code.astype(np.int64), 5).astype(F) * np.repeat(scale, 256)[:code.size]


def encode(x, rnd, bits, top):
    """(codes, scales) of float32 magnitudes, float32 throughout; the code from a floor on the code's own grid."""
    n, nb = x.size, -(-x.size // 256)
    pad = np.zeros(nb * 256, F)
    pad[:n] = x
    amax = pad.reshape(nb, 256).max(1)
    ok = amax >= F(2.0 ** -100)
    scale = np.where(ok, amax / F(top), F(0)).astype(F)
    inv = np.where(ok, F(top) / np.where(ok, amax, F(1)), F(0)).astype(F)
    y = (x * np.repeat(inv, 256)[:n]).astype(F)
    # below 2^-6 (the subnormal grid) the value is held to 2^-29, as FP32's own subnormals 2^-120 further down hold it
    y = np.where(y < 2.0 ** -6, np.round(y.astype(np.float64) * 2.0 ** 29) / 2.0 ** 29, y.astype(np.float64))
    e = np.clip(np.floor(np.log2(np.maximum(y, 2.0 ** -60))), -6, 0)
    grid = 2.0 ** (e - bits)
    k = np.floor(y / grid + (rnd + 0.5) / 65536).astype(np.int64)  # in units of the grid: from 2^bits up where e > -6
    code = np.where(e > -6, (e + 6).astype(np.int64) * (1 << bits) + k, k)
    return np.minimum(code, (8 << bits) - 1), scale, np.repeat(ok, 256)[:n]


def host_step(p, g, m, v, coef, lr, wd, step, t, seed, state8):
    """One tensor in float32, each operation rounded by itself."""
    c1, c2 = F(1 - B1), F(1 - B2)
    ss, decay = F(lr / (1 - B1 ** step)), F(1 - lr * wd)
    if coef is not None:
        g = g * F(coef)
    m = m * F(B1) + g * c1
    v = v * F(B2) + (g * g) * c2
    root = np.sqrt(v)
    p = p * decay - ss * (m / (root * F(1 / np.sqrt(1 - B2 ** step)) + F(EPS)))
    if not state8:
        return p, m, v
    w = philox(p.size, t, step, seed)
    cm, sm, _ = encode(np.abs(m), (w & np.uint64(0xFFFF)).astype(np.int64), 4, 1.9375)
    cs, sv, ok = encode(root, (w >> np.uint64(16)).astype(np.int64), 5, 1.96875)
    cs = np.where(ok & (root > 0) & (cs == 0), 1, cs)
    return p, (cm + 128 * ((m < 0) & (cm > 0)), sm), (cs, sv)


SIZES = [1, 7, 255, 256, 257, 2048, 8191, 8192, 8193, 40000, 0, 3]


def make(sizes, pdt, gdt, seed, dev="cuda", std=1e-2):
    r = np.random.RandomState(seed)
    ps = [torch.tensor(r.randn(n) * 0.05, dtype=torch.float32, device=dev) for n in sizes]
    gs = [torch.tensor(r.randn(n) * std * np.exp(r.randn(n)), dtype=gdt, device=dev) for n in sizes]
    masters = None
    if pdt == torch.bfloat16:
        masters, ps = ps, [p.to(torch.bfloat16) for p in ps]
    return ps, gs, masters


@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("clip", [0.0, 0.5, 1e6])
def test_fp32_states(pdt, gdt, clip):
    """Three steps; sizes around the block, the vector and the chunk; a learning rate and a decay per tensor."""
    ps, gs, masters = make(SIZES, pdt, gdt, 1)
    lrs, wds = [1.0 + 0.5 * i for i in range(len(SIZES))], [0.01 * i for i in range(len(SIZES))]
    opt = q.AdamW(ps, gs, masters=masters, lr_scale=lrs, weight_decay=wds, betas=(B1, B2), eps=EPS)
    norm = torch.full((1,), float("nan"), device="cuda")
    w = [t.double() for t in (masters or ps)]
    m, v = [torch.zeros_like(t) for t in w], [torch.zeros_like(t) for t in w]
    tp, tm, tv = ([torch.zeros_like(t) for t in w] for _ in range(3))
    for step in (1, 2, 3):
        opt.step(1e-3, step, max_grad_norm=clip, grad_norm=norm if clip else None)
        true = torch.sqrt(sum((g.double() ** 2).sum() for g in gs))
        coef = float(min(1.0, clip / true)) if clip else 1.0
        torch.cuda.synchronize()
        assert q.get_error() == 0
        if clip:
            assert abs(float(norm) - float(true)) <= U * float(true)
        for i in range(len(w)):
            g, lr = gs[i].double() * coef, 1e-3 * lrs[i]
            am = B1 * m[i].abs() + (1 - B1) * g.abs()
            m[i] = B1 * m[i] + (1 - B1) * g
            v[i] = B2 * v[i] + (1 - B2) * g * g
            tm[i], tv[i] = B1 * tm[i] + 5 * U * am, B2 * tv[i] + 8 * U * v[i]
            den = (v[i] / (1 - B2 ** step)).sqrt() + EPS
            s = lr / (1 - B1 ** step) * m[i] / den
            ds = 16 * U * s.abs() + lr / (1 - B1 ** step) * tm[i] / den + s.abs() * tv[i] / v[i].clamp(min=1e-300)
            w[i] = w[i] * (1 - lr * wds[i]) - s
            tp[i] = tp[i] + ds + 4 * U * (w[i].abs() + s.abs())
            assert bool(((opt.m[i].double() - m[i]).abs() <= tm[i] + 1e-38).all())
            assert bool(((opt.v[i].double() - v[i]).abs() <= tv[i] + 1e-38).all())
            got = (masters or ps)[i]
            assert bool(((got.double() - w[i]).abs() <= tp[i]).all())
            if masters:
                assert torch.equal(ps[i], got.to(torch.bfloat16))


@pytest.mark.parametrize("pdt,gdt", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("clip", [0.0, 0.3])
def test_8bit_states_bit_for_bit(pdt, gdt, clip):
    """Four steps from zero: every code, scale and weight against float32 on the host."""
    seed = 0x123456789ABCDEF
    ps, gs, masters = make(SIZES, pdt, gdt, 2)
    gs[5][100:1900] *= 1e-4  # blocks whose values span the codes' whole range
    gs[5][600:612] = 0.0
    opt = q.AdamW(ps, gs, masters=masters, state_bits=8, weight_decay=0.02, betas=(B1, B2), eps=EPS)
    cpu = lambda t: t.float().cpu().numpy().astype(F)  # noqa: E731
    w = [cpu(t) for t in (masters or ps)]
    g = [cpu(t) for t in gs]
    for step in (1, 2, 3, 4):
        before = [(opt.m[i].cpu().numpy().astype(np.int64), opt.m_scale[i].cpu().numpy(), opt.v[i].cpu().numpy(), opt.v_scale[i].cpu().numpy())
                  for i in range(len(w))]
        opt.step(1e-3, step, seed=seed, max_grad_norm=clip)
        torch.cuda.synchronize()
        assert q.get_error() == 0
        norm = np.sqrt(sum((x.astype(np.float64) ** 2).sum() for x in g))
        coef = min(1.0, clip / norm) if clip else None
        for i in range(len(w)):
            if w[i].size == 0:
                continue
            cm, sm, cv, sv = before[i]
            s = decode_s(cv, sv)
            p, (em, esm), (ev, esv) = host_step(w[i], g[i], decode_m(cm, sm), s * s, coef, 1e-3, 0.02, step, i, seed, True)
            assert np.array_equal(opt.m_scale[i].cpu().numpy(), esm) and np.array_equal(opt.v_scale[i].cpu().numpy(), esv)
            assert np.array_equal(opt.m[i].cpu().numpy(), em) and np.array_equal(opt.v[i].cpu().numpy(), ev)
            got = cpu((masters or ps)[i])
            assert np.all(np.abs(got - p) <= 4 * U * (np.abs(p) + np.abs(p - w[i])))  # the quotient: two units
            w[i] = got


def test_read_state():
    ps, gs, _ = make([300, 0, 513, 256, 5], torch.float32, torch.float32, 3)
    opt = q.AdamW(ps, gs, state_bits=8)
    opt.step(1e-3, 1, seed=5)
    opt.step(1e-3, 2, seed=5)
    starts, total = [0, 512, 512, 1280, 1536], 1541
    for dt in (torch.float32, torch.bfloat16):
        mo, vo = (torch.full((total,), 9.0, dtype=dt, device="cuda") for _ in range(2))
        opt.read_state(mo, vo)
        filled = torch.zeros(total, dtype=torch.bool)
        for i, (a, p) in enumerate(zip(starts, ps)):
            n = p.numel()
            m = decode_m(opt.m[i].cpu().numpy().astype(np.int64), opt.m_scale[i].cpu().numpy())
            s = decode_s(opt.v[i].cpu().numpy(), opt.v_scale[i].cpu().numpy())
            assert torch.equal(mo[a:a + n].cpu(), torch.from_numpy(m).to(dt)) and torch.equal(vo[a:a + n].cpu(), torch.from_numpy(s * s).to(dt))
            filled[a:a + n] = True
        assert bool((mo.cpu()[~filled] == 9.0).all())


def test_rounding_is_unbiased_and_does_not_stick():
    """A constant second moment from zero: after 3000 steps of b2 = 0.999 (95 % of the way) the mean of sqrt(v) over 65536
    elements follows the 64-bit average; rounding to nearest would have stopped below a tenth of v.  The mean's own spread:
    a step's drift d moves sqrt(v) by one code with a probability, so an element's variance is about d x code step / (2 x
    0.0005), under (0.2)^2 of its square: 0.2 / 256 of the mean; v = sqrt(v)^2 then lies up to 4 % high.  1 % and 5 %."""
    n = 1 << 16
    r = np.random.RandomState(4)
    mag = torch.tensor(np.exp(r.uniform(-2, 0, n)), dtype=torch.float32, device="cuda")
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, device="cuda")
    opt = q.AdamW([p], [g], state_bits=8, weight_decay=0.0)
    sign = torch.tensor(r.choice([-1.0, 1.0], n), dtype=torch.float32, device="cuda")
    for step in range(1, 3001):
        g.copy_(mag * (sign if step % 2 else -sign))
        opt.step(1e-5, step, seed=77)
    m, v = (torch.empty(n, device="cuda") for _ in range(2))
    opt.read_state(m, v)
    want = mag.double() ** 2 * (1 - 0.999 ** 3000)
    assert abs(float((v.double().sqrt() / want.sqrt()).mean()) - 1) < 0.01
    assert abs(float((v.double() / want).mean()) - 1) < 0.05
    # m alternates between +- (1 - b1) / (1 + b1) of the magnitude: its mean has the last gradient's sign (step 3000: -sign)
    ratio = (m.double() / (-sign * mag).double()).mean()
    assert abs(float(ratio) - 0.1 / 1.9) < 0.01 * 0.1 / 1.9 + 3 * 0.05 / 256


def test_a_norm_that_is_not_finite_leaves_everything():
    for bad in (float("inf"), float("nan"), 3e38):
        for bits in (32, 8):
            ps, gs, masters = make([1000, 300], torch.bfloat16, torch.float32, 5)
            opt = q.AdamW(ps, gs, masters=masters, state_bits=bits)
            opt.step(1e-3, 1, seed=1, max_grad_norm=1.0)
            keep = [t.clone() for t in (*ps, *masters, *opt.m, *opt.v)]
            gs[1][7] = bad
            norm = torch.zeros(1, device="cuda")
            opt.step(1e-3, 2, seed=1, max_grad_norm=1.0, grad_norm=norm)
            assert not bool(torch.isfinite(norm))
            assert all(torch.equal(a, b) for a, b in zip(keep, (*ps, *masters, *opt.m, *opt.v)))
            gs[1][7] = 0.0
            opt.step(1e-3, 2, seed=1, max_grad_norm=1.0, grad_norm=norm)  # and the next step is a whole one
            assert bool(torch.isfinite(norm)) and not torch.equal(keep[2], masters[0])


def test_nan_without_the_clip_stays_in_its_element():
    ps, gs, _ = make([600], torch.float32, torch.float32, 6)
    gs[0][300] = float("nan")
    opt = q.AdamW(ps, gs)
    opt.step(1e-3, 1)
    assert torch.isnan(ps[0]).nonzero().flatten().tolist() == [300]


def test_zero_gradients_and_tiny_blocks():
    """States of zero stay zero (no division by a zero scale); a block below 2^-100 is stored as zero."""
    ps = [torch.ones(512, device="cuda")]
    gs = [torch.zeros(512, device="cuda")]
    opt = q.AdamW(ps, gs, state_bits=8, weight_decay=0.1)
    opt.step(1e-2, 1, seed=3)
    assert bool((opt.m[0] == 0).all()) and bool((opt.v_scale[0] == 0).all()) and bool((ps[0] == 1 - 1e-3).all())
    gs[0][:256] = 1e-37
    opt.step(1e-2, 2, seed=3)
    assert bool((opt.m[0] == 0).all()) and bool(torch.isfinite(ps[0]).all())


def test_repeats_streams_and_graph():
    """The same bits from the same inputs, eagerly, on another stream and from a graph, norm included."""
    def fresh():
        ps, gs, ms = make([5000, 70000, 33], torch.bfloat16, torch.float32, 7)
        return q.AdamW(ps, gs, masters=ms, state_bits=8), ps, ms

    def end(opt, ps, ms):
        torch.cuda.synchronize()
        return [t.clone() for t in (*ps, *ms, *opt.m, *opt.v, *opt.m_scale, *opt.v_scale)]
    a = fresh()
    a[0].step(1e-3, 1, seed=9, max_grad_norm=0.1)
    want = end(*a)
    b = fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b[0].step(1e-3, 1, seed=9, max_grad_norm=0.1)
    assert all(torch.equal(x, y) for x, y in zip(want, end(*b)))
    c = fresh()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c[0].step(1e-3, 1, seed=9, max_grad_norm=0.1)
    g.replay()
    assert all(torch.equal(x, y) for x, y in zip(want, end(*c)))
    d = fresh()
    d[0].step(1e-3, 1, seed=10, max_grad_norm=0.1)
    assert not torch.equal(want[6], end(*d)[6])  # another seed rounds otherwise


def test_only_empty_tensors():
    e = torch.empty(0, device="cuda")
    opt = q.AdamW([e], [e])
    norm = torch.full((1,), 5.0, device="cuda")
    opt.step(1e-3, 1, max_grad_norm=1.0, grad_norm=norm)
    opt.step(1e-3, 2)
    assert float(norm) == 0.0


def test_step_refusals():
    ps, gs, _ = make([10], torch.float32, torch.float32, 8)
    opt = q.AdamW(ps, gs)
    norm = torch.zeros(2, device="cuda")
    for kw in (dict(step=0), dict(step=1 << 32), dict(lr=float("nan")), dict(max_grad_norm=-1.0), dict(grad_norm=norm)):
        with pytest.raises(q.QerlError):
            opt.step(**{"lr": 1e-3, "step": 1, **kw})
    with pytest.raises(q.QerlError):  # FP32 states have no codes to read
        opt.read_state(torch.empty(10, device="cuda"), torch.empty(10, device="cuda"))
    assert q.get_error() == 0


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-300, 1e-39, 1e-30, 1e30, 1e39])
def test_any_eps(bits, eps):
    """An eps beyond FP32's normal range: weights without a gradient stay, and the others take the step of the formula
    (none where eps is beyond FP32's largest)."""
    p = torch.full((600,), 0.5, device="cuda")
    g = torch.zeros(600, device="cuda")
    g[300:] = 2.0
    opt = q.AdamW([p], [g], state_bits=bits, weight_decay=0.0, eps=eps)
    opt.step(1e-2, 1, seed=1)
    if eps > 1e-50:  # else 0 / 0, as the formula has it in FP32
        assert bool((p[:300] == 0.5).all())
    want = 0.5 - 1e-2 * 2.0 / (2.0 + eps)
    assert bool(((p[300:].double() - want).abs() <= 16 * U).all())


def test_plan_on_a_busy_stream():
    """A plan made while its stream still writes to the memory that the allocator hands out for its table."""
    ps, gs, _ = make([5000, 300, 70000], torch.float32, torch.float32, 9)
    want = [p.clone() for p in ps]
    ref = q.AdamW(want, gs)
    ref.step(1e-3, 1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        opt0 = q.AdamW([p.clone() for p in ps], gs)
        size = opt0.ws.numel()
        del opt0
        m, v = ([torch.zeros_like(p) for p in ps] for _ in range(2))
        for _ in range(20):
            big = torch.empty(1 << 28, device="cuda").normal_()  # some ms each
        junk = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xAB)
        at = junk.data_ptr()
        del junk, big
        opt = q.AdamW(ps, gs, m=m, v=v)
        opt.step(1e-3, 1)
    torch.cuda.synchronize()
    assert opt.ws.data_ptr() == at  # the block that the stream had still to fill
    assert q.get_error() == 0 and all(torch.equal(a, b) for a, b in zip(ps, want))


def test_plan_keeps_every_tensor():
    """The lists that were given may change afterwards; the plan's tensors stay."""
    import gc
    import weakref
    ps, gs, masters = make([100, 300], torch.bfloat16, torch.float32, 10)
    opt = q.AdamW(ps, gs, masters=masters, state_bits=8)
    kept = [weakref.ref(t) for t in (*ps, *gs, *masters)]
    ps.clear(), gs.clear(), masters.clear()
    gc.collect()
    assert all(r() is not None for r in kept)
    opt.step(1e-3, 1)
    torch.cuda.synchronize()
    assert q.get_error() == 0


def test_roots_are_correctly_rounded():
    """sqrt(v) against numpy's over v's whole range, by the scale it leaves (the block's largest root over the largest code):
    a block per value, one element of it not zero, no gradient."""
    nb = 1 << 16
    r = np.random.RandomState(11)
    code = r.randint(1, 256, nb).astype(np.uint8)
    at = r.randint(0, 256, nb)
    want_s = np.exp(r.uniform(np.log(1e-18), np.log(1e17), nb))
    want_s[::4] = np.exp(r.uniform(np.log(1e-6), np.log(1e-1), len(want_s[::4])))  # where gradients' roots lie
    scale = (want_s / value(code.astype(np.int64), 5)).astype(F)
    codes = np.zeros((nb, 256), np.uint8)
    codes[np.arange(nb), at] = code
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    n = nb * 256
    p, g = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    opt = q.AdamW([p], [g], m=[torch.zeros(n, dtype=torch.uint8, device="cuda")], v=[dev(codes.reshape(-1))],
                  m_scale=[torch.zeros(nb, device="cuda")], v_scale=[dev(scale)], betas=(B1, B2), weight_decay=0.0)
    opt.step(1e-3, 3, seed=1)
    s = value(code.astype(np.int64), 5).astype(F) * scale
    v = (s * s) * F(B2)
    assert np.array_equal(opt.v_scale[0].cpu().numpy(), np.sqrt(v) / F(1.96875))
    assert bool((p == 1.0).all()) and q.get_error() == 0
