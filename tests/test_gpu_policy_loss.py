"""GPU parity of the token log-probabilities, the policy loss and its gradient against the definition in 64 bits.

Tolerances, from FP32 arithmetic (u = 2^-24), with y = (x - max) / tau in log2 units:
  - y: two products and a difference, 3 u |y|; e^y: 2^-22 more; a sum over a row: at most 64 terms one after another in a
    thread (more where rows exceed the registers: then 64 + V / 4096), then a tree of at most 16: s = (80 + V / 4096) u + 2^-22;
  - logp = y_id ln 2 - ln Z: d = s + 4 u |y_id| + 2 u |ln Z| + 4 u;
  - entropy = ln Z - sum e y / Z: d_H = 3 s (1 + sum |p y|) + 4 u |ln Z| (weights that are off by 3 u |y| with y to 40: s covers);
  - p_j: relative r = 2 s + 3 u |y_j| + 4 u;
  - loss terms: amp = w (rho |A| + beta (e^d' + 1)), error amp (2 d + 16 u); the sum's own rounding u;
  - dlogits: the rounding to its type (eps / 2 |ref|) + (amp / tau) (2 d + r + 16 u) p_j, and at the chosen token also
    (amp / tau) d for 1 - p; 1e-37 for what underflows."""
import math

import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

pytestmark = pytest.mark.gpu
NAN, INF, U = float("nan"), float("inf"), 2.0 ** -24


def make(T, V, dtype, seed, std=2.5, tau=1.0, masked=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(T, V, generator=g, device="cuda") * std).to(dtype)
    ids = torch.randint(V, (T,), generator=g, device="cuda")
    at = torch.arange(T, device="cuda")
    x[at, ids] += (6 * torch.rand(T, generator=g, device="cuda")).to(dtype)
    lp = torch.log_softmax(x.double() / tau, -1)[at, ids]
    # ratios inside, outside and far from the clip, none at its edges
    r = torch.tensor([0.3, 0.79, 0.82, 1.0, 1.19, 1.26, 1.31, 2.5], device="cuda", dtype=torch.float64)[at % 8]
    old = (lp - r.log()).float()
    ref = (lp + 0.5 * torch.randn(T, generator=g, device="cuda")).float()
    adv = torch.randn(T, generator=g, device="cuda")
    w = torch.rand(T, generator=g, device="cuda") / T
    w[torch.rand(T, generator=g, device="cuda") < masked] = 0.0
    return x, ids, old, ref, adv, w


def reference(x, ids, old, ref, adv, w, lo, hi, beta, tau, scale):
    """Every result and its tolerance in float64."""
    T, V = x.shape
    at = torch.arange(T, device=x.device)
    takes = (w != 0) & (ids >= 0) & (ids < V)
    ids = ids.clamp(0, V - 1).long()
    lse = torch.logsumexp(x.double() / tau, -1)
    p = torch.exp(x.double() / tau - lse[:, None])
    top = x.double().amax(-1)
    yabs = (top[:, None] - x.double()) / tau / math.log(2)
    py = torch.where(p > 0, p * yabs, 0.0)  # a masked logit (-inf) has no weight
    lnz = lse - top / tau
    s = (80 + V / 4096) * U + 2.0 ** -22
    y_id = yabs[at, ids].nan_to_num(posinf=0.0)
    logp, ent = x.double()[at, ids] / tau - lse, lnz + py.sum(-1) * math.log(2)
    d = s + 4 * U * y_id + 2 * U * lnz.abs() + 4 * U
    dH = 3 * s * (1 + py.sum(-1)) + 4 * U * lnz.abs()
    out = dict(logp=(logp, d), entropy=(ent, dH))
    if old is not None:
        lo, hi = 1 - lo, 1 + hi
        A, wd = adv.double(), w.double()
        rho = torch.exp(logp - old.double())
        u = ref.double() - logp if ref is not None else torch.zeros_like(logp)
        keeps = torch.where(A >= 0, rho <= hi, rho >= lo)
        pol = -torch.minimum(rho * A, rho.clamp(lo, hi) * A)
        kl = torch.exp(u) - u - 1
        c = torch.where(takes, wd * (beta * (1 - torch.exp(u)) - torch.where(keeps, rho * A, 0.0)), 0.0) * scale / tau
        amp = torch.where(takes, wd * (rho * A.abs() + beta * (torch.exp(u) + 1) + torch.exp(u) + u.abs() + 1), 0.0)
        add = lambda t: torch.where(takes, wd * t, 0.0).sum()  # noqa: E731
        sums = torch.stack([add(pol + beta * kl), add(pol), add(kl), add((~keeps).double())])
        out["sums"] = (sums, (amp * (2 * d + 16 * U)).sum() + 2 * U * amp.sum())
        g = -c[:, None] * p
        g[at, ids] += c
        r = 2 * s + 3 * U * yabs.nan_to_num(posinf=0.0) + 4 * U
        tol = torch.finfo(x.dtype).eps / 2 * g.abs() + (abs(scale) * amp / tau)[:, None] * (2 * d[:, None] + r + 16 * U) * p + 1e-37
        tol[at, ids] += abs(scale) * amp / tau * (3 * d + 16 * U)
        out["dlogits"] = (g, tol)
    for k in ("logp", "entropy"):
        v, t = out[k]
        out[k] = (torch.where(takes, v, 0.0), t)
    return out


def close(name, got, want):
    ref, tol = want
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (name, int(bad.sum()), float(((got - ref).abs() / tol).nan_to_num(0.0).max()))


def check(x, ids, old, ref, adv, w, lo=0.2, hi=0.28, beta=0.04, tau=1.0, scale=1.0, dlogits=None):
    T = x.shape[0]
    want = reference(x, ids, old, ref, adv, w, lo, hi, beta, tau, scale)
    nan = lambda *s: torch.full(s, NAN, device="cuda")  # noqa: E731
    if dlogits is None:
        dlogits = torch.full_like(x, NAN)
    ws = q.workspace(q.OP_POLICY_LOSS, T, x.shape[1], 0, 0).fill_(0xFF)
    got = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, clip_low=lo, clip_high=hi, beta=beta, temperature=tau,
                             grad_scale=scale, dlogits=dlogits, logp=nan(T), entropy=nan(T), sums=nan(4), ws=ws)
    torch.cuda.synchronize()
    assert q.get_error() == 0
    for k, v in zip(("sums", "logp", "entropy", "dlogits"), got):
        close(k, v, want[k])
    return got


# rows shorter than a vector; one thread block, every cluster size; odd rows at every alignment; rows past the registers
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (5, 7), (40, 33), (300, 1000), (7, 8191), (200, 8200), (33, 16001), (2, 32768),
                                 (160, 40001), (9, 100003), (170, 131072), (3, 151937), (2, 262144), (3, 300007)])
def test_loss_and_gradient(T, V, dtype):
    x, ids, old, ref, adv, w = make(T, V, dtype, T + V)
    if T == 1:
        w.fill_(0.7)
    check(x, ids, old, ref, adv, w)


@pytest.mark.parametrize("tau,beta,scale", [(0.7, 0.0, 1.0), (1.5, 0.2, -3.0), (1.0, 0.04, 1024.0)])
def test_options(tau, beta, scale):
    x, ids, old, ref, adv, w = make(64, 5003, torch.bfloat16, 5, tau=tau)
    check(x, ids.int(), old, ref if beta else None, adv, w, 0.1, 0.3, beta, tau, scale)


def test_log_probabilities_alone():
    for T, V, dt in ((1, 9, torch.float32), (64, 32768, torch.bfloat16), (5, 131072, torch.bfloat16), (300, 50001, torch.float32)):
        x, ids, *_, w = make(T, V, dt, V, tau=0.9)
        for weights in (None, w):
            lp, ent = q.qerl_token_logp(x, ids, weights=weights, temperature=0.9)
            want = reference(x, ids, None, None, None, torch.ones_like(w) if weights is None else w, 0, 0, 0, 0.9, 1)
            close("logp", lp, want["logp"])
            close("entropy", ent, want["entropy"])


def test_no_gradient_wanted():
    x, ids, old, ref, adv, w = make(50, 3001, torch.bfloat16, 6)
    with_g = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, beta=0.1)
    sums, lp, ent, none = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, beta=0.1, want_grad=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip((sums, lp, ent), with_g))
    no_w = q.qerl_policy_loss(x, ids, old, adv, None, ref_logp=ref, beta=0.1)
    ones = q.qerl_policy_loss(x, ids, old, adv, torch.ones_like(w), ref_logp=ref, beta=0.1)
    assert all(torch.equal(a, b) for a, b in zip(no_w, ones))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(20, 1003), (160, 40001), (3, 300007)])
def test_in_place_and_strides(T, V, dtype):
    """dlogits over the logits; logits and dlogits inside wider rows that keep their margins, at unlike alignments."""
    x, ids, old, ref, adv, w = make(T, V, dtype, 7)
    want = check(x, ids, old, ref, adv, w)
    y = x.clone()
    got = q.qerl_policy_loss(y, ids, old, adv, w, ref_logp=ref, clip_low=0.2, clip_high=0.28, beta=0.04, dlogits=y)
    assert got[3] is y and all(torch.equal(a, b) for a, b in zip(got, want))
    wide = torch.full((T, V + 13), 5.0, dtype=dtype, device="cuda")
    wide[:, 3:V + 3] = x
    other = torch.full((T, V + 30), 9.0, dtype=dtype, device="cuda")
    # rows at another alignment are summed in another order: within the tolerances, not bit for bit
    check(wide[:, 3:V + 3], ids, old, ref, adv, w, dlogits=other[:, 6:V + 6])
    assert bool((other[:, :6] == 9.0).all()) and bool((other[:, V + 6:] == 9.0).all()) and bool((wide[:, V + 3:] == 5.0).all())


def test_rows_that_take_no_part():
    """Weight 0 or an id outside the vocabulary: NaN and Inf there reach nothing."""
    x, ids, old, ref, adv, w = make(64, 2003, torch.bfloat16, 8, masked=0.3)
    ids[:3] = torch.tensor([-100, 2003, -1], device="cuda")
    out = (w == 0) | (ids < 0) | (ids >= 2003)
    clean = check(x, ids, old, ref, adv, w)
    for junk in (NAN, INF, -INF):
        x[out], old[out], adv[out] = junk, junk, junk
        got = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, clip_low=0.2, clip_high=0.28, beta=0.04)
        assert all(torch.equal(a, b) for a, b in zip(got, clean))
        assert bool((got[3][out] == 0).all()) and bool((got[1][out] == 0).all())
    sums, *_ = q.qerl_policy_loss(x, ids, old, adv, torch.zeros_like(w))
    assert sums.tolist() == [0.0] * 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_vocabulary(dtype):
    """Logits at -inf and at the type's lowest value: no weight, no gradient, no NaN; a row of lowest values is uniform;
    a row that is all -inf adds nothing."""
    T, V = 12, 9000
    x, ids, old, ref, adv, w = make(T, V, dtype, 9, masked=0.0)
    keep = torch.zeros(T, V, dtype=torch.bool, device="cuda")
    keep[:, ::3] = True
    keep[torch.arange(T), ids] = True
    for junk in (-INF, torch.finfo(dtype).min):
        y = torch.where(keep, x, torch.full_like(x, junk))
        lp = torch.log_softmax(y.double(), -1)[torch.arange(T), ids]
        got = check(y, ids, (lp - 0.05).float(), (lp + 0.1).float(), adv, w)
        assert bool((got[3][~keep] == 0).all())
    y = torch.full_like(x, torch.finfo(dtype).min)
    lp, ent = q.qerl_token_logp(y, ids)
    assert bool(((lp + math.log(V)).abs() < 1e-5).all()) and bool(((ent - math.log(V)).abs() < 1e-4).all())
    x[4] = -INF
    lp, ent = q.qerl_token_logp(x, ids)
    assert lp[4] == -INF and ent[4] == 0
    got = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, beta=0.04)
    w2 = w.clone()
    w2[4] = 0
    rest = q.qerl_policy_loss(x, ids, old, adv, w2, ref_logp=ref, beta=0.04)
    assert torch.equal(got[0], rest[0]) and torch.equal(got[3], rest[3])


def test_nan_shows_in_its_row_only():
    x, ids, old, ref, adv, w = make(8, 5000, torch.float32, 10, masked=0.0)
    x[2, 77] = NAN
    x[5, 78] = INF
    sums, lp, ent, dx = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, beta=0.04)
    bad = torch.isnan(lp)
    assert bad.tolist() == [i in (2, 5) for i in range(8)] and bool(torch.isnan(sums[0]))
    assert bool(torch.isfinite(dx[~bad]).all()) and bool(torch.isnan(dx[2]).any())


def test_certain_and_impossible_tokens():
    """p of the chosen token next to 1 (1 - p without cancellation) and next to 0."""
    x = torch.zeros(4, 4096, device="cuda")
    ids = torch.tensor([5, 5, 9, 9], device="cuda")
    x[0, 5], x[1, 5], x[2, 5], x[3, 5] = 30.0, 60.0, 30.0, 80.0
    lp = torch.log_softmax(x.double(), -1)[torch.arange(4), ids]
    adv = torch.tensor([1.0, -1.0, 2.0, -2.0], device="cuda")
    check(x, ids, lp.float(), (lp + 0.2).float(), adv, torch.full((4,), 0.25, device="cuda"))


def test_gradient_against_differences():
    """Central differences of the loss in 64 bits, at the chosen token and elsewhere: h^2 max|L'''| / 6 with |L'''| <= 8 amp."""
    T, V, h = 6, 50, 2.0 ** -8
    x, ids, old, ref, adv, w = make(T, V, torch.float32, 11, std=1.0, masked=0.0)
    dx = q.qerl_policy_loss(x, ids, old, adv, w, ref_logp=ref, clip_low=0.2, clip_high=0.28, beta=0.04)[3].double()
    L = lambda y: reference(y, ids, old, ref, adv, w, 0.2, 0.28, 0.04, 1.0, 1.0)["sums"][0][0]  # noqa: E731
    amp = float((w.double() * (3 * adv.double().abs() + 4)).max())
    for t in range(T):
        for j in (int(ids[t]), (int(ids[t]) + 1) % V, 17):
            e = torch.zeros_like(x, dtype=torch.float64)
            e[t, j] = h
            diff = float(L(x.double() + e) - L(x.double() - e)) / (2 * h)
            assert abs(diff - float(dx[t, j])) <= 8 * amp * h * h / 6 + 1e-6 * amp


def test_empty_repeat_and_other_stream():
    e = torch.empty(0, device="cuda")
    sums, lp, ent, dx = q.qerl_policy_loss(torch.empty(0, 7, device="cuda"), e.long(), e, e)
    assert sums.tolist() == [0.0] * 4 and lp.numel() == 0
    x, ids, old, ref, adv, w = make(700, 3000 + 5, torch.bfloat16, 12)
    want = check(x, ids, old, ref, adv, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = check(x, ids, old, ref, adv, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(1, 501), (5, 9000), (3, 300007), (400, 40001)])
@pytest.mark.parametrize("gap", [9.0, 24.0, 60.0])
def test_nearly_certain_tokens_keep_their_digits(dtype, T, V, gap):
    """log p = -log(1 + r) and the entropy of tokens with r, the others' sum over the token's own e^x, far below 1: errors
    relative to the values.  r: s = (80 + V / 4096) u + 2^-22 as above, 2^-22 for the change of its unit, and 3 u |y| of
    exponents y, taken twice; twice that for the entropy, whose two terms have one sign; log1p and the products: 16 u."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(T, V, generator=g, device="cuda") * 2).to(dtype)
    ids, at = torch.randint(V, (T,), generator=g, device="cuda"), torch.arange(T, device="cuda")
    x[at, ids] = math.log(V) + 2.0 + gap
    nan = lambda: torch.full((T,), NAN, device="cuda")  # noqa: E731
    logp, ent = q.qerl_token_logp(x, ids, logp=nan(), entropy=nan())
    d = x.double() - x.double()[at, ids][:, None]
    d[at, ids] = -INF
    e = d.exp()
    r = e.sum(-1)
    want = -torch.log1p(r)
    H = torch.log1p(r) - (e * d.clamp_min(-1e4)).sum(-1) / (1 + r)
    ymax = float(-d.clamp_min(-1e4).masked_fill(d == -INF, 0.0).min()) / math.log(2)
    rel = (80 + V / 4096) * U + 2.0 ** -21 + 6 * U * ymax
    assert bool(((logp.double() - want).abs() <= (rel + 16 * U) * want.abs()).all())
    assert bool(((ent.double() - H).abs() <= (2 * rel + 16 * U) * H).all())
    assert q.get_error() == 0


# rows that the ring's kernel takes, and a shape for one cluster per row
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(160, 40001), (8, 9000)])
@pytest.mark.parametrize("gap", [30.0, 45.0, 70.0, 80.0, 83.0, 90.0])
def test_gradient_of_improbable_tokens(dtype, T, V, gap):
    """A chosen token far below the row's maximum, at weights from 1 down to 1e-9: the likely tokens' gradient keeps its
    digits (the tolerances are relative to the loss term's amplitude)."""
    x, ids, _, _, adv, _ = make(T, V, dtype, 13, std=1.0)
    g = torch.Generator(device="cuda").manual_seed(V)
    at = torch.arange(T, device="cuda")
    for k in range(3):  # the likely tokens
        x[at, (ids + 17 + 5000 * k) % V] = gap - 10.0 + k
    x[at, ids] = -10.0
    lp = torch.log_softmax(x.double(), -1)[at, ids]
    w = 10.0 ** (-9.0 * torch.rand(T, generator=g, device="cuda"))
    check(x, ids, (lp - 0.05).float(), (lp + 0.1).float(), adv.sign() * (adv.abs() + 0.5), w)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(8, 5000), (160, 40001)])
def test_nan_shows_without_the_kl_term(dtype, T, V):
    """beta = 0 and no reference: a NaN logit, an infinite one, a NaN old log-probability and a NaN advantage reach the loss
    and their own rows' gradient, and no other row."""
    x, ids, old, _, adv, w = make(T, V, dtype, 14, masked=0.0)
    adv = adv.sign() * (adv.abs() + 0.1)
    clean = q.qerl_policy_loss(x, ids, old, adv, w)
    assert bool(torch.isfinite(clean[3]).all()) and bool(torch.isfinite(clean[0]).all())
    for row, name in ((1, "logit"), (3, "inf"), (4, "old"), (6, "adv")):
        y, o, a = x.clone(), old.clone(), adv.clone()
        if name == "logit":
            y[row, 77] = NAN
        elif name == "inf":
            y[row, 78] = INF
        else:
            (o if name == "old" else a)[row] = NAN
        sums, lp, ent, dx = q.qerl_policy_loss(y, ids, o, a, w)
        rest = torch.arange(T, device="cuda") != row
        assert bool(torch.isnan(sums[:2]).all()), name
        assert bool(torch.isnan(dx[row]).any()), name
        assert bool(torch.isnan(lp[row])) == (name in ("logit", "inf")), name
        assert torch.equal(dx[rest], clean[3][rest]) and torch.equal(lp[rest], clean[1][rest]), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(6, 9000), (160, 40001)])
def test_extreme_temperatures(dtype, T, V):
    """Every temperature that is taken, with -inf logits: at 1e30 the rest is uniform, at 1e-12 the largest takes all."""
    x, ids, *_ = make(T, V, dtype, 15)
    at = torch.arange(T, device="cuda")
    keep = torch.zeros(T, V, dtype=torch.bool, device="cuda")
    keep[:, ::3] = True
    keep[at, ids] = True
    x[at, ids] = 20.0
    x = torch.where(keep, x, torch.full_like(x, -INF))
    n = keep.sum(-1).double().log()
    lp, ent = q.qerl_token_logp(x, ids, temperature=1e30)
    tol = (80 + V / 4096) * U + 2.0 ** -22 + 4 * U * float(n.max())
    assert bool(((lp.double() + n).abs() <= tol).all()) and bool(((ent.double() - n).abs() <= 3 * tol).all())
    lp, ent = q.qerl_token_logp(x, ids, temperature=1e-12)
    assert bool((lp == 0).all()) and bool((ent == 0).all())
    sums, lp, ent, dx = q.qerl_policy_loss(x, ids, -n.float(), torch.ones(T, device="cuda"), temperature=1e30, grad_scale=1e30)
    assert bool((dx[~keep] == 0).all()) and bool(torch.isfinite(dx).all())
    assert abs(float(sums[1]) + T) < 1e-4 * T  # rho = 1
