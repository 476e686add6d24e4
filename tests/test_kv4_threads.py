"""Threads that call one cache or attention object with tensors of other strides: each call's strides are its own (CPU only;
nothing is launched)."""
import sys
import threading

import torch

import nvfp4_weight_only_quantize_gb300 as q


def run_threads(calls):
    threads, switch = [threading.Thread(target=calls, args=(w,)) for w in (64, 80, 96, 112)], sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(switch)


def test_cache():
    cache, lens, wrong = q.Kv4Cache(2, 40, 2, 64, device="cpu"), torch.zeros(2, dtype=torch.int32), []

    def calls(width):
        k, v = (torch.zeros(2, 3, 2, w, dtype=torch.bfloat16)[..., :64] for w in (width, width + 8))
        for _ in range(20000):
            _, ks, _, vs = cache._tokens(k, v, lens)
            if tuple(ks) != k.stride()[:3] or tuple(vs) != v.stride()[:3]:
                wrong.append((width, tuple(ks), tuple(vs)))

    run_threads(calls)
    assert not wrong, wrong[:3]


class Library:
    """Stands in for the library: notes the strides that a call brings."""

    def __init__(self):
        self.wrong = []

    def qerl_kv4_attention_ws_bytes(self, *args):
        return 16

    def qerl_kv4_attention(self, dims, x, pre, pl, suf, sl, scale, out, *rest):
        d = dims._obj
        for address, strides in ((x, d.q_stride), (out, d.out_stride)):
            if tuple(strides) != self.strides[address]:
                self.wrong.append(tuple(strides))
        return 0


def test_attention(monkeypatch):
    fake, lens = Library(), torch.zeros(2, dtype=torch.int32)
    cache = q.Kv4Cache(2, 40, 2, 64, device="cpu")
    monkeypatch.setattr(q, "lib", lambda: fake)
    monkeypatch.setattr(q, "_stream", lambda stream=None: 0)
    monkeypatch.setattr(q, "_here", lambda *tensors: None)
    cache._launched_on.add(0)
    plan = q.Kv4Attention(cache, 4, 3)
    tensors = {w: [torch.zeros(2, 3, 4, x, dtype=torch.bfloat16)[..., :64] for x in (w, w + 8)] for w in (64, 80, 96, 112)}
    fake.strides = {t.data_ptr(): t.stride()[:3] for pair in tensors.values() for t in pair}

    def calls(width):
        for _ in range(10000):
            plan.run(tensors[width][0], lens, out=tensors[width][1])

    run_threads(calls)
    assert not fake.wrong, fake.wrong[:3]
