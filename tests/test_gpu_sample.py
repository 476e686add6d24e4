"""GPU parity of token sampling against the definition in 64 bits.

The token itself has to be equal: its masses are good to 2^-40, so that only draws within some 2^-38 of a border could differ,
and none of the fixed draws here is that near (the reference checks it).  Log-probabilities: (x - max) / tau and the
sum's logarithm are taken in 64 bits and rounded once, 2^-24 relative; the sum is FP32 per chunk, off by at most 4e-6."""
import math

import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def logits_of(T, V, dtype, seed, kind="normal"):
    g = gen(seed)
    x = torch.randn(T, V, generator=g, device="cuda") * 2.5
    if kind == "peaked":
        at = torch.randint(V, (T, 1), generator=g, device="cuda") // 2 * 2 % V
        x.scatter_(1, at, 20.0)
    elif kind == "equal":
        x = torch.full((T, V), -3.25, device="cuda")
    elif kind == "few":  # a few distinct values: ties everywhere
        x = torch.round(x)
    elif kind == "far":  # beyond the first histogram's keys
        x = x * 1e-3 + 1e-4
    elif kind == "large":
        x = x * 1e4
    elif kind == "masked":
        x[torch.rand(T, V, generator=g, device="cuda") < 0.9] = -math.inf
        x[:, 0] = 1.0
    elif kind == "lowest":
        x[torch.rand(T, V, generator=g, device="cuda") < 0.5] = torch.finfo(dtype).min
    return x.to(dtype)


def reference(x, u, tau, k, p, m):
    """(id, logp, logq, how far from a border the draw is, relative) of one row, 64 bits."""
    y = x.double() / tau
    y = y - y.max()
    e = torch.exp(y)
    order = torch.sort(-y, stable=True).indices  # equal ones by index
    w = e[order]
    n = len(w) if k <= 0 else min(k, len(w))
    near = math.inf
    if p <= 0:
        n = 1
    elif p < 1:
        c = w[:n].cumsum(0)
        want = p * c[-1]
        at = int((c < want).sum())
        near = min(near, float((c - want).abs().min() / c[-1]))
        n = at + 1
    if m > 0:
        n = min(n, int((w >= min(m, 1.0)).sum()))
    kept = torch.sort(order[:n]).values
    c = e[kept].cumsum(0)
    t = min(max(u, 0.0), 0.99999994) * c[-1]
    i = int((c <= t).sum())
    near = min(near, float((c[e[kept] > 0] - t).abs().min() / c[-1]) if u > 0 else 1.0)
    return int(kept[i]), float(y[kept[i]] - e.sum().log()), float(y[kept[i]] - c[-1].log()), near


def check(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, **kw):
    T = x.shape[0]
    out = q.qerl_sample(x, u, temperature, top_k, top_p, min_p, **kw)
    torch.cuda.synchronize()
    assert q.get_error() == 0
    ids, logp, logq = (t.tolist() for t in out)
    at = lambda s, t: float(s[t]) if torch.is_tensor(s) else float(torch.tensor(s, dtype=torch.float32))  # noqa: E731
    for t in range(T):
        i, lp, lq, near = reference(x[t], float(u[t]), at(temperature, t), int(at(top_k, t)), at(top_p, t), at(min_p, t))
        # a draw of exactly a border's value is right in both; nearer than 2^-38 but not on it, the reference could not tell
        assert near == 0 or near > 2.0 ** -38, "change the case's seed"
        assert ids[t] == i, (t, ids[t], i, logp[t], lp)
        for got, want in ((logp[t], lp), (logq[t], lq)):
            assert abs(got - want) <= 4e-6 + 2.0 ** -23 * abs(want), (t, got, want)
    return out


CUTS = [dict(), dict(top_k=1), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=50, top_p=0.95, min_p=0.02), dict(top_k=1000, top_p=0.5),
        dict(top_p=0.05), dict(top_p=0.9999), dict(min_p=1.0), dict(top_k=7, min_p=1e-6)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (2, 7), (5, 129), (3, 1000), (2, 1025), (1, 16001), (33, 4099), (160, 2050), (2, 131072)])
@pytest.mark.parametrize("cut", CUTS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()) or "none")
def test_sample(dtype, T, V, cut):
    check(logits_of(T, V, dtype, T * V), torch.rand(T, generator=gen(V), device="cuda"), temperature=0.7, **cut)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["peaked", "equal", "few", "far", "large", "masked", "lowest"])
@pytest.mark.parametrize("cut", CUTS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()) or "none")
def test_kinds_of_rows(dtype, kind, cut):
    # an odd number, so that sums of equal masses meet no border of u or top_p (both dyadic multiples) but by the count
    check(logits_of(4, 5001, dtype, 11, kind), torch.tensor([0.1, 0.503, 0.77, 0.999], device="cuda"), **cut)


def test_many_rows_of_a_full_vocabulary():
    """Draws by the thousand, among them some that the fast sums cannot decide."""
    x = logits_of(400, 100003, torch.bfloat16, 5)
    u = torch.rand(400, generator=gen(6), device="cuda")
    for cut in (dict(), dict(top_p=0.95)):
        check(x, u, **cut)
    check(x[:100].float() + torch.randn(100, 100003, generator=gen(7), device="cuda") * 0.01, u[:100], top_p=0.95)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [300007, 1 << 20])
def test_the_largest_vocabularies(dtype, V):
    u = torch.rand(3, generator=gen(20), device="cuda")
    x = logits_of(3, V, dtype, 21)
    for cut in (dict(), dict(top_k=100, top_p=0.9), dict(top_p=0.7), dict(top_k=300000), dict(min_p=0.3)):
        check(x, u, **cut)
    check(torch.zeros(2, V, dtype=dtype, device="cuda"), torch.tensor([0.3, 0.999], device="cuda"), top_k=77777)


def test_tensors_of_another_device_are_refused():
    x, u = logits_of(2, 100, torch.float32, 22), torch.rand(2, device="cuda")
    for args in ((x.cpu(), u), (x, u.cpu())):
        with pytest.raises(AssertionError):
            q.qerl_sample(*args)


def test_ends_of_u():
    x = logits_of(6, 3000, torch.float32, 8)
    u = torch.tensor([0.0, 1.0, 5.0, -1.0, math.nan, 2.0 ** -149], device="cuda")
    ids, _, _ = q.qerl_sample(x, u, top_k=20)
    kept = torch.sort(torch.topk(x, 20).indices).values
    assert ids.tolist() == [int(kept[i, -1 if i in (1, 2) else 0]) for i in range(6)]
    # a token of no mass is never drawn
    x = torch.full((2, 100), -math.inf, device="cuda")
    x[:, 50:52] = 1.0
    assert q.qerl_sample(x, torch.tensor([0.0, 1.0], device="cuda"))[0].tolist() == [50, 51]


def test_exact_borders():
    """Four equal tokens: sums that meet top_p and u exactly."""
    x = torch.zeros(8, 4, device="cuda")
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.0, 0.5, 0.49, 0.99], device="cuda")
    assert q.qerl_sample(x, u)[0].tolist() == [0, 1, 2, 3, 0, 2, 1, 3]
    assert q.qerl_sample(x, u, top_p=0.5)[0].tolist() == [0, 0, 1, 1, 0, 1, 0, 1]
    assert q.qerl_sample(x, u, top_k=2)[0].tolist() == [0, 0, 1, 1, 0, 1, 0, 1]
    _, lp, lq = q.qerl_sample(x, u, top_k=1)
    assert bool((lq == 0).all()) and bool((lp == torch.tensor(0.25, device="cuda").log()).all())
    zeros = torch.tensor([[0.0, -0.0, 0.0, -0.0]], device="cuda")  # equal, whatever their sign
    assert [int(q.qerl_sample(zeros, u[i:i + 1], top_k=2)[0]) for i in range(4)] == [0, 0, 1, 1]


def test_rows_without_a_distribution():
    x = logits_of(5, 2000, torch.bfloat16, 9)
    x[0] = -math.inf
    x[1, 77] = math.nan
    x[2, 1999] = math.inf
    tau = torch.tensor([1.0, 1.0, 1.0, 0.0, math.nan], device="cuda")
    for kw in (dict(), dict(top_k=5), dict(top_p=0.5, min_p=0.1)):
        ids, lp, lq = q.qerl_sample(x, torch.full((5,), 0.5, device="cuda"), temperature=tau, **kw)
        assert ids.tolist() == [-1] * 5
        assert lp[0] == lq[0] == -math.inf and bool(torch.isnan(lp[1:]).all()) and bool(torch.isnan(lq[1:]).all())


def test_settings_of_each_row_and_their_ends():
    T = 12
    x = logits_of(T, 7003, torch.float32, 10)
    k = torch.tensor([0, 1, -3, 50, 7003, 10000, 2, 0, 0, 40, 0, 0], dtype=torch.int32, device="cuda")
    p = torch.tensor([1.0, 0.5, 0.9, 0.0, -1.0, math.nan, 2.0, 0.3, 1.0, 0.99, 1e-30, 1.0], device="cuda")
    m = torch.tensor([0.0, 0.1, -1.0, 0.0, 0.5, 0.0, math.nan, 0.0, 2.0, 0.01, 0.0, 1e-30], device="cuda")
    tau = torch.linspace(0.2, 3.0, T, device="cuda")
    plain_p, plain_m = torch.nan_to_num(p, nan=1.0), torch.nan_to_num(m, nan=0.0)
    u = torch.rand(T, generator=gen(12), device="cuda")
    want = check(x, u, tau, k, plain_p, plain_m)
    got = q.qerl_sample(x, u, tau, k, p, m)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tau", [1e-29, 1e-6, 1e6, 1e30])
def test_temperatures(tau):
    for cut in (dict(), dict(top_p=0.9), dict(top_k=5)):
        check(logits_of(3, 999, torch.float32, 13), torch.tensor([0.2, 0.55, 0.9], device="cuda"), temperature=tau, **cut)


def test_the_split_does_not_matter():
    """A row alone (a cluster of CTAs) and among many (one): the same token and log-probabilities within rounding."""
    for dtype in (torch.bfloat16, torch.float32):
        x = logits_of(200, 40001, dtype, 14)
        u = torch.rand(200, generator=gen(15), device="cuda")
        for cut in (dict(), dict(top_k=30, top_p=0.9), dict(top_p=0.9)):
            ids, lp, lq = q.qerl_sample(x, u, **cut)
            for t in range(0, 200, 23):
                i, a, b = q.qerl_sample(x[t:t + 1], u[t:t + 1], **cut)
                assert int(i) == int(ids[t]) and float(a) == float(lp[t]) and float(b) == float(lq[t])
            again = q.qerl_sample(x, u, **cut)
            assert torch.equal(again[0], ids) and torch.equal(again[1], lp) and torch.equal(again[2], lq)


def test_lists_of_a_whole_row():
    """Rows that are listed whole, from every alignment, with tokens of no mass among them and the maximum below zero."""
    for dtype in (torch.bfloat16, torch.float32):
        wide = (-1.9921875 - 0.3 * logits_of(3, 8200, torch.float32, 23).abs()).to(dtype)
        wide[1, 100:7000] = -math.inf
        wide[2] = wide[2] * 1e-3 - 7
        u = torch.tensor([0.11, 0.73, 0.998], device="cuda")
        for first in (0, 1, 3, 6):
            for V in (600, 8000, 8185):
                for cut in (dict(top_p=0.9999), dict(top_k=V - 1), dict(top_k=V // 2, top_p=0.99), dict(top_p=0.3, min_p=0.2)):
                    check(wide[:, first:first + V], u, **cut)


def test_strides_graph_and_stream():
    wide = logits_of(7, 3001, torch.bfloat16, 16)
    x, u = wide[:, 5:2998], torch.rand(7, generator=gen(17), device="cuda")
    want = check(x, u, top_k=40)
    x = x.clone()
    out = torch.empty(7, dtype=torch.int64, device="cuda"), torch.empty(7, device="cuda"), torch.empty(7, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            q.qerl_sample(x, u, top_k=40, ids=out[0], logp=out[1], logq=out[2])
    for _ in range(3):
        graph.replay()
    late = q.qerl_sample(x, u, top_k=40, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(want[0], out[0])
    for a, b, c in zip(want, out, late):
        # rows at another alignment are summed in other chunks: each of the two within 4e-6 + 2^-23 |.| of the exact value
        assert torch.equal(b, c) and bool(((a - b).abs() <= 2 * (4e-6 + 2.0 ** -23 * a.abs())).all())
    assert q.qerl_sample(x[:0], u[:0])[0].shape == (0,)


def test_logp_is_the_old_logp_of_the_policy_loss():
    """Sampled tokens go on to the policy loss: their ratio is 1."""
    x = logits_of(64, 32000, torch.bfloat16, 18)
    ids, lp, _ = q.qerl_sample(x, torch.rand(64, generator=gen(19), device="cuda"), temperature=0.8, top_p=0.9)
    again, _ = q.qerl_token_logp(x, ids, temperature=0.8)
    assert bool(((again - lp).abs() <= 4e-6 + 2.0 ** -20).all())
