"""Attention over 4-bit caches at sizes that take the kernel of many rows, alone and beside the one of few rows: repeats,
back-to-back calls on one workspace, graphs whose lengths change on the device, streams, launches that are not chained, caches
that span more than 32 bits, whole prompts.  Tolerances as in test_gpu_kv4.py."""
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q
from test_gpu_kv4 import check, filled, gen, i32, reference, rnd

pytestmark = pytest.mark.gpu

# (prefixes, their capacity and lengths, own capacity and lengths, new tokens, heads, launches of the kernels of many and few rows)
BOTH = (1, 3000, [2999], 64, [64, 41, 40, 50, 63, 45, 60, 42], 40, 16, 2, 1, 1)
MANY = (2, 1500, [701, 1500], 900, [900, 161, 400, 170], 160, 28, 4, 1, 0)
OWN = (0, 0, None, 1100, [1100, 129, 600, 1001], 129, 16, 2, 1, 0)


def counts():
    return q.kernel_launch_count(q.KERNEL_KV4_ROWS128), q.kernel_launch_count(q.KERNEL_KV4_ROWS8)


def made(form, seed, D=128):
    n, P, pl, S, sl, Lq, Hq, Hkv = form[:8]
    g = gen(seed)
    pre = filled(g, n, P, Hkv, D, 0.5, 1.0) if n else None
    suf = filled(g, len(sl), S, Hkv, D)
    plan = q.Kv4Attention(suf[0], Hq, Lq, prefix=pre[0] if n else None)
    plan.ws.fill_(0xFF)
    return g, pre, suf, plan, None if pl is None else i32(pl), i32(sl)


@pytest.mark.parametrize("form", [BOTH, MANY, OWN], ids=["both", "many", "own"])
def test_back_to_back_calls_repeat(form):
    """Other lengths and other queries in turn, nothing waited for in between: each call's bits are those that it has alone."""
    g, pre, suf, plan, pl, sl = made(form, 41)
    B, Lq, Hq = len(form[4]), form[5], form[6]
    qs = [rnd(g, B, Lq, Hq, 128) * 1.5 for _ in range(3)]
    lens = [sl, sl.flip(0), (sl - 7).clamp(min=0)]
    alone = []
    for x, n in zip(qs, lens):
        before = counts()
        lse = torch.empty(B, Lq, Hq, device="cuda")
        alone.append((plan.run(x, n, pl, lse=lse), lse))
        torch.cuda.synchronize()
        assert tuple(b - a for a, b in zip(before, counts())) == form[8:]
    for x, n, (out, lse) in zip(qs, lens, alone):
        ref, rl, tol, ltol = reference(x, pre and pre[1], suf[1], form[2], n.tolist(), 128 ** -0.5, 8.0)
        assert bool(((out.double() - ref).abs() <= tol).all())
        seen = ~torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), ~seen) and bool(((lse.double() - rl).abs()[seen] <= ltol[seen]).all())

    def turn(stream=None):
        got = []
        for _ in range(4):
            for x, n in zip(qs, lens):
                lse = torch.empty(B, Lq, Hq, device="cuda")
                got.append((plan.run(x, n, pl, lse=lse, stream=stream), lse))
        torch.cuda.synchronize()
        for k, (out, lse) in enumerate(got):
            assert torch.equal(out, alone[k % 3][0]) and torch.equal(lse, alone[k % 3][1])

    turn()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        turn()
    torch.cuda.synchronize()
    q.set_launch_chaining(False)
    try:
        turn()
    finally:
        q.set_launch_chaining(True)
    late = plan.run(qs[1], lens[1], pl, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(late, alone[1][0]) and q.get_error() == 0


@pytest.mark.parametrize("form", [BOTH, MANY, OWN], ids=["both", "many", "own"])
def test_graph_of_steps_with_lengths_on_the_device(form):
    """A kernel that changes the lengths, append, attention and again, captured once: the lengths and tokens that the calls
    see are those that the work before them left."""
    g, pre, suf, plan, pl, sl = made(form, 42)
    B, Lq, Hq, Hkv = len(form[4]), form[5], form[6], form[7]
    qq = torch.zeros(B, Lq, Hq, 128, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(B, 9, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    outs = [torch.empty_like(qq) for _ in range(2)]
    lens = sl.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            for out in outs:
                lens.sub_(5)
                suf[0].append(k, v, lens)
                plan.run(qq, lens, pl, out=out)
    torch.cuda.synchronize()
    for _ in range(3):
        for t in (k, v, qq):
            t.copy_(rnd(g, *t.shape))
        n, cache = lens.clone(), suf[0].data.clone()
        graph.replay()
        torch.cuda.synchronize()
        after = suf[0].data.clone()
        suf[0].data.copy_(cache)
        for out in outs:  # the same, call by call
            n -= 5
            suf[0].append(k, v, n)
            want = plan.run(qq, n, pl)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert torch.equal(suf[0].data, after) and torch.equal(n, lens)
        held = suf[0].read(i32([suf[0].T] * B), suf[0].T)
        ref, _, tol, _ = reference(qq, pre and pre[1], held, form[2], n.tolist(), 128 ** -0.5, 8.0)
        assert bool(((outs[1].double() - ref).abs() <= tol).all())
    assert lens.tolist() == (sl - 30).tolist() and q.get_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_offsets_past_32_bits(D):
    """Sequences, heads and tiles that lie more than 4 GB into the cache."""
    g = gen(43)
    T, H, B, cell = 1000, 2, 2, 36 * D
    base = torch.zeros(9 << 30, dtype=torch.uint8, device="cuda")
    for strides in ((4 << 30, cell * 32, cell), (cell * 32, 4 << 30, cell), (cell, cell * 2, 200 << 20)):
        data = torch.as_strided(base, (B, H, 32, cell), strides + (1,))
        c = q.Kv4Cache(B, T, H, D, data=data)
        c.append(rnd(g, B, T, H, D), rnd(g, B, T, H, D), i32([T, T]))
        before = counts()
        check(rnd(g, B, 129, 16, D), None, (c, c.read(i32([T, T]), T)), None, [1000, 966])
        assert tuple(b - a for a, b in zip(before, counts())) == (1, 0)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L,lens,Hq,Hkv", [(40, [40, 39, 1, 0], 8, 2), (257, [257, 256, 33], 14, 2), (1000, [1000, 999, 128, 0], 16, 2),
                                           (4000, [4000], 7, 1)])
def test_whole_prompts(D, L, lens, Hq, Hkv):
    """As many new tokens as keys, of sequences as long and shorter."""
    g = gen(L + D)
    check(rnd(g, len(lens), L, Hq, D) * 1.5, None, filled(g, len(lens), L, Hkv, D), None, lens)


def test_whole_answers_after_a_prefix():
    g = gen(44)
    check(rnd(g, 3, 300, 16, 128), filled(g, 3, 600, 2, 128, 0.5, 1.0), filled(g, 3, 300, 2, 128), [600, 1, 0], [300, 299, 100])
