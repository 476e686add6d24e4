"""Attention over 4-bit caches at the ends of what the factors may be.

Queries of zeros weigh all keys alike: the output is the mean of the values a row sees (each probability is then exact, the FP32
sums over n keys in parts are off by (2^-21 + 128 2^-24) of mean |v|, the output's rounding by 2^-8 of itself), lse the
logarithm of their number (off by as much, and 2^-22 of itself)."""
import math

import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q
from test_gpu_kv4 import gen, i32, rnd

pytestmark = pytest.mark.gpu
SUMS = 2.0 ** -21 + 128 * 2.0 ** -24


def check_means(cache, held, Hq, Lq, lens, scale=None):
    """held: the values in 64 bits."""
    B, D = cache.n, cache.D
    qq = torch.zeros(B, Lq, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Lq, Hq, device="cuda")
    out = q.Kv4Attention(cache, Hq, Lq, scale=scale).run(qq, i32(lens), lse=lse)
    torch.cuda.synchronize()
    assert q.get_error() == 0
    gs = Hq // cache.Hkv
    for b in range(B):
        for l in range(Lq):
            n = lens[b] - Lq + 1 + l
            v = held[b, :n].repeat_interleave(gs, 1)
            ref, A = v.mean(0), v.abs().mean(0)
            assert bool(((out[b, l].double() - ref).abs() <= 1.02 * (2.0 ** -8 * ref.abs() + SUMS * A)).all()), (b, l)
            assert bool(((lse[b, l].double() - math.log(n)).abs() <= 1.02 * (SUMS + 2.0 ** -22 * math.log(n))).all()), (b, l)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("k_scale", [1.0, 1e-8, 1e-20, 1e-30])
@pytest.mark.parametrize("Lq,S,lens,kernel", [(1, 100, [77, 1], 4), (3, 100, [77, 5], 4), (129, 1000, [999, 700, 641, 130], 5)])
def test_queries_of_zeros(D, k_scale, Lq, S, lens, kernel):
    g, B = gen(1), len(lens)
    cache = q.Kv4Cache(B, S, 2, D, k_scale, 1.0)
    cache.append(rnd(g, B, S, 2, D), rnd(g, B, S, 2, D), i32([S] * B))
    before = q.kernel_launch_count(kernel)
    check_means(cache, cache.read(i32([S] * B), S)[1].double(), 16, Lq, lens)
    assert q.kernel_launch_count(kernel) == before + 1


@pytest.mark.parametrize("S,Lq,lens", [(30001, 1, [30001]), (30001, 33, [30000])])
def test_values_near_the_top_of_the_largest_factor(S, Lq, lens):
    g = gen(2)
    cache, unit = q.Kv4Cache(1, S, 1, 64, 1.0, 1e30), q.Kv4Cache(1, S, 1, 64)
    k, v = rnd(g, 1, S, 1, 64), (torch.rand(1, S, 1, 64, generator=g, device="cuda") * 1000 + 1500).to(torch.bfloat16)
    cache.append(k, (v.float() * 1e30).to(torch.bfloat16), i32([S]))
    # the codes and scales alone: the same bytes read with a factor of one
    unit.data.copy_(cache.data)
    held = unit.read(i32([S]), S)[1].double() * float(torch.tensor(1e30, dtype=torch.float32))
    check_means(cache, held, 8, Lq, lens)


def test_prefix_and_own_tokens_with_factors_far_apart():
    """Values of a factor of 1e-30 beside values of 1e30: the small ones count in the weights alone."""
    g = gen(3)
    pre, own = q.Kv4Cache(1, 64, 1, 64, 1.0, 1e-30), q.Kv4Cache(2, 64, 1, 64, 1.0, 1e30)
    k, v = rnd(g, 1, 64, 1, 64), rnd(g, 1, 64, 1, 64)
    pre.append(k, (v.float() * 1e-30).to(torch.bfloat16), i32([64]))
    k, v = rnd(g, 2, 64, 1, 64), (torch.rand(2, 64, 1, 64, generator=g, device="cuda") * 1000 + 1500).to(torch.bfloat16)
    own.append(k, (v.float() * 1e30).to(torch.bfloat16), i32([64, 64]))
    held = own.read(i32([64, 64]), 64)[1].double()
    out = q.Kv4Attention(own, 4, prefix=pre).run(torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([64, 64]))
    ref = held.sum(1) / 128  # [2, 1, 64]; read's rounding of the values: 2^-8 of each, of one sign all
    assert bool(((out[:, 0].double() - ref).abs() <= 1.02 * (2 * 2.0 ** -8 + SUMS) * ref).all())
