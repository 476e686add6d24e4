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
