"""A rollout step out of the operators it is made of: new keys and values into the 4-bit caches, attention over the prompt
and the answers, the LM head, the next tokens; captured once and replayed, with lengths and uniform numbers on the device.
What each operator gives is checked by its own tests; here they run together and are compared with the definitions, step by
step, from the same inputs."""
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q
from test_gpu_kv4 import filled, gen, i32, reference, rnd
from test_gpu_sample import check as check_sample

pytestmark = pytest.mark.gpu


def test_rollout_steps_in_a_graph():
    g = gen(31)
    B, G, Hq, Hkv, D, V, T = 12, 4, 14, 2, 128, 5003, 40
    pre, pre_held = filled(g, B // G, 70, Hkv, D, 0.5, 1.0)
    pl = i32([70, 33, 1])
    own = q.Kv4Cache(B, T, Hkv, D, 1.0, 2.0)
    plan = q.Kv4Attention(own, Hq, prefix=pre)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    k, v, qq = (torch.zeros(B, 1, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, Hq))
    head = rnd(g, V, Hq * D) * 0.05
    u = torch.zeros(B, device="cuda")
    out, lse, logits = torch.empty_like(qq), torch.empty(B, 1, Hq, device="cuda"), torch.empty(B, V, dtype=torch.bfloat16, device="cuda")
    ids, logp, logq = torch.empty(B, dtype=torch.int64, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, device="cuda")

    def step():
        lens.add_(1)
        own.append(k, v, lens)
        plan.run(qq, lens, pl, out=out, lse=lse)
        torch.matmul(out.view(B, Hq * D), head.T, out=logits)
        q.qerl_sample(logits, u, temperature=0.8, top_k=50, top_p=0.9, ids=ids, logp=logp, logq=logq)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # the library's and cuBLAS's set-up, outside the capture
        lens.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    for t in range(1, T + 1):
        k.copy_(rnd(g, B, 1, Hkv, D)), v.copy_(rnd(g, B, 1, Hkv, D)), qq.copy_(rnd(g, B, 1, Hq, D) * 1.5)
        u.copy_(torch.rand(B, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        if t % 13 != 1:
            continue
        assert lens.tolist() == [t] * B and q.get_error() == 0
        held = own.read(i32([T] * B), T)
        ref, rl, tol, ltol = reference(qq, pre_held, held, [70, 33, 1], [t] * B, D ** -0.5, 16.0)
        assert bool(((out.double() - ref).abs() <= tol).all()) and bool(((lse.double() - rl).abs() <= ltol).all())
        want = check_sample(logits, u, temperature=0.8, top_k=50, top_p=0.9)
        for a, b in zip(want, (ids, logp, logq)):
            assert torch.equal(a, b)
        again, _ = q.qerl_token_logp(logits, ids, temperature=0.8)  # the policy loss's old log-probabilities
        assert bool(((again - logp).abs() <= 4e-6 + 2.0 ** -20).all())
