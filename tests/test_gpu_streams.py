"""Calls with stream=: what they allocate for themselves meets neither work that is still queued on the current stream nor
what the current stream allocates next, and objects' own memory outlives a launch elsewhere."""
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q
from nvfp4_weight_only_quantize_gb300 import synth

pytestmark = pytest.mark.gpu


def busy(stream):
    """Some 25 ms of work."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(50_000_000)


def policy():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(300, 1000, generator=g, device="cuda")
    ids = torch.randint(1000, (300,), generator=g, device="cuda")
    old, adv = torch.randn(300, generator=g, device="cuda") * 0.1 - 7.0, torch.randn(300, generator=g, device="cuda")
    return lambda **kw: q.qerl_policy_loss(x, ids, old, adv, **kw)


def logp():
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(300, 1000, generator=g, device="cuda")
    ids = torch.randint(1000, (300,), generator=g, device="cuda")
    return lambda **kw: q.qerl_token_logp(x, ids, **kw)


def attention():
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    t = [r(8, 1, 8, 128), r(2, 700, 2, 128), r(2, 700, 2, 128), r(8, 100, 2, 128), r(8, 100, 2, 128)]
    lens = torch.full((8,), 77, dtype=torch.int32, device="cuda")
    return lambda **kw: (q.qerl_prefix_attention(*t, lens, **kw),)


def backward():
    M, N, K, r = 64, 384, 512, 16
    codes, scales, ts = q.qerl_nvfp4_quantize(synth.weight(N, K, 1, "cuda"))
    x, dy = synth.activations(M, K, 2, "cuda"), synth.activations(M, N, 3, "cuda")
    A, B = synth.lora_A(r, K, 4, "cuda"), synth.lora_B(N, r, 5, "cuda")
    return lambda **kw: q.qerl_nvfp4_lora_linear_bwd(dy, x, codes, scales, ts, A, B, 2.0, **kw)


SIZES = [1 << k for k in range(9, 22)]  # bytes: every size that the calls allocate meets one of them, or a part of it


@pytest.mark.parametrize("make", [policy, logp, backward, attention])
def test_work_still_queued_on_the_current_stream(make):
    call = make()
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    call(stream=s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in SIZES]
    busy(torch.cuda.current_stream())
    for b in blocks:
        b.fill_(0xFF)
    del blocks, b
    got = call(stream=s)
    torch.cuda.synchronize()
    assert q.get_error() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("make", [policy, logp, backward, attention])
def test_what_the_current_stream_allocates_next(make):
    call = make()
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    call(stream=s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy(s)
    got = call(stream=s)
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF) for n in SIZES for _ in range(4)]
    torch.cuda.synchronize()
    assert all(bool((j == 0xFF).all()) for j in junk)
    assert q.get_error() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_objects_dropped_before_their_launch_elsewhere():
    """The states of an optimizer and the workspace of an attention stay until the other stream has used them."""
    g = torch.Generator(device="cuda").manual_seed(4)
    p, grad = (torch.randn(100000, generator=g, device="cuda") for _ in range(2))
    want = p.clone()
    q.AdamW([want], [grad], state_bits=8).step(1e-2, 1, seed=1, max_grad_norm=1.0)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    t = [r(2, 700, 2, 128), r(2, 700, 2, 128), r(8, 100, 2, 128), r(8, 100, 2, 128)]
    qq, lens = r(8, 1, 8, 128), torch.full((8,), 77, dtype=torch.int32, device="cuda")
    out = q.PrefixAttention(*t, 8).run(qq, lens)
    again = torch.empty_like(out)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    opt, attn = q.AdamW([p], [grad], state_bits=8), q.PrefixAttention(*t, 8)
    s.wait_stream(torch.cuda.current_stream())
    busy(s)
    opt.step(1e-2, 1, seed=1, max_grad_norm=1.0, stream=s)
    attn.run(qq, lens, out=again, stream=s)
    del opt, attn
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF) for n in SIZES for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((j == 0xFF).all()) for j in junk)
    assert q.get_error() == 0 and torch.equal(p, want) and torch.equal(out, again)
