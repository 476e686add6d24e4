"""Attention over 4-bit caches whose values are small against the cache's factor, under one key that takes nearly all the
weight and whose own value is zero: what is left is the sum over keys of 10 to 16 nats less.

Per output with A = sum_k p_k |v_k|, p the probabilities and p_max the largest (first order, times 1.02 for the rest):
  - the output's rounding to bf16: 2^-8 |ref|;
  - each probability's rounding to fp16: 2^-11 A.  It is held as p / p_max times 2^8 or more, so that below fp16's normal
    numbers it is off by 2^-25, which is 2^-33 p_max: 2^-33 p_max sum_k |v_k|.  Values times their scales are exact;
  - the logit's error e = (D + 4) 2^-24 scale sum |q| |k| (the largest over the keys), in numerator and denominator: 2 e A;
    ex2 (2^-22) and FP32 sums: (2^-21 + 128 2^-24) A.
None of these grows with the cache's factor."""
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q
from test_gpu_kv4 import gen, i32, rnd

pytestmark = pytest.mark.gpu


def small_values(D, B, S, Hkv, Hq, Lq, ratio, gap, seed):
    """Queries [B, Lq, Hq, D], a full cache, its keys and values: key 5 is `gap` nats above the rest, its value 0."""
    g = gen(seed)
    cache = q.Kv4Cache(B, S, Hkv, D, 1.0, 1.0)
    k, v, qq = rnd(g, B, S, Hkv, D), rnd(g, B, S, Hkv, D) * ratio, rnd(g, B, Lq, Hq, D)
    k[..., 0], qq[..., 0] = 0, 8
    k[:, 5, :, 0] = gap * D ** 0.5 / 8
    v[:, 5] = 0
    cache.append(k, v, i32([S] * B))
    return qq, cache, cache.read(i32([S] * B), S)


def check(qq, cache, held, lens):
    B, Lq, Hq, D = qq.shape
    gs, scale = Hq // cache.Hkv, D ** -0.5
    out = q.Kv4Attention(cache, Hq, Lq).run(qq, i32(lens))
    torch.cuda.synchronize()
    assert q.get_error() == 0
    worst = 0.0
    for b in range(B):
        for h in range(Hq):
            k, v = (t[b, :lens[b], h // gs].double() for t in held)
            x = qq[b, :, h].double()
            a = scale * (x @ k.T)
            sees = torch.arange(lens[b], device="cuda") <= lens[b] - Lq + torch.arange(Lq, device="cuda")[:, None]
            a = a.masked_fill(~sees, -torch.inf)
            e = (D + 4) * 2.0 ** -24 * scale * (x.abs() @ k.abs().T).amax(1, keepdim=True)
            p = torch.softmax(a, 1)
            ref, A = p @ v, p @ v.abs()
            tail = 2.0 ** -33 * p.amax(1, keepdim=True) * (sees.double() @ v.abs())
            tol = 1.02 * (2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * e + 2.0 ** -21 + 128 * 2.0 ** -24) * A + tail)
            err = (out[b, :, h].double() - ref).abs()
            worst = max(worst, float((err / tol).max()))
    assert worst <= 1.0, worst


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ratio", [0.005, 0.02, 0.05])
@pytest.mark.parametrize("gap", [10.0, 12.0, 14.0, 16.0])
def test_few_rows(D, ratio, gap):
    before = q.kernel_launch_count(q.KERNEL_KV4_ROWS8)
    check(*small_values(D, 2, 400, 2, 8, 1, ratio, gap, int(gap)), [400, 171])
    assert q.kernel_launch_count(q.KERNEL_KV4_ROWS8) == before + 1


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ratio", [0.005, 0.02, 0.05])
@pytest.mark.parametrize("gap", [10.0, 12.0, 14.0, 16.0])
def test_many_rows(D, ratio, gap):
    before = q.kernel_launch_count(q.KERNEL_KV4_ROWS128)
    check(*small_values(D, 4, 1000, 2, 16, 129, ratio, gap, int(gap)), [999, 700, 641, 140])
    assert q.kernel_launch_count(q.KERNEL_KV4_ROWS128) == before + 1


def test_a_long_cache_under_one_key():
    """131072 keys of values near the factor's lower end, one of which takes five sixths of the weight."""
    qq, cache, held = small_values(128, 1, 131072, 1, 7, 1, 0.01, 14.0, 3)
    check(qq, cache, held, [131072])
