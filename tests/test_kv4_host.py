"""What the 4-bit cache's calls refuse on the host (CPU only): sizes whose products pass 64 bits, caches of different devices."""
import types

import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q
from test_kv4_abi import L, attn, cache, tokens  # noqa: F401


@pytest.mark.parametrize("call", ["append", "read"])
@pytest.mark.parametrize("n,Hkv,new", [(1 << 30, 65536, 1 << 30), (1 << 30, 65536, 1 << 23), (1 << 30, 65536, 1 << 22), (1 << 30, 1, 1 << 30),
                                       (1 << 30, 65535, 1 << 30), (1 << 26, 32768, 1)])
def test_grids_beyond_any_launch(L, call, n, Hkv, new):  # noqa: F811
    assert tokens(L, cache(n=n, Hkv=Hkv, T=1 << 30), n=new, call=call) == 2


def test_attention_takes_caches_and_workspace_of_one_device(monkeypatch):
    """Caches whose tensors say that they lie on two made-up devices."""
    q.build()
    monkeypatch.setattr(q, "_stream", lambda stream=None: 0)
    prefix, suffix = q.Kv4Cache(2, 40, 2, 64, device="cpu"), q.Kv4Cache(4, 40, 2, 64, device="cpu")
    q.Kv4Attention(suffix, 4, prefix=prefix)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    q.Kv4Attention(suffix, 4, prefix=prefix, ws=ws)
    elsewhere = types.SimpleNamespace(device=torch.device("cuda", 1), numel=ws.numel, data_ptr=ws.data_ptr)
    with pytest.raises(AssertionError):
        q.Kv4Attention(suffix, 4, prefix=prefix, ws=elsewhere)
    prefix.data = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(AssertionError):
        q.Kv4Attention(suffix, 4, prefix=prefix)
    with pytest.raises(AssertionError):
        q.Kv4Attention(suffix, 4, prefix=prefix, ws=ws)
    with pytest.raises(AssertionError):
        q.Kv4Attention(None, 4, prefix=prefix, batch=4, ws=ws)


def test_outputs_whose_elements_share_an_address(L):  # noqa: F811
    """A stride of 0 repeats an input; what is written needs an address each."""
    for strides in ((0, 512, 128), (1024, 0, 128), (1024, 512, 0)):
        assert tokens(L, cache(), call="read", ks=strides) == 2 and tokens(L, cache(), call="read", vs=strides) == 2
        assert attn(L, Lq=2, os_=strides)[0] == 2
        # nothing is repeated along a dimension of one; inputs may be.  The workspace and the lengths, looked at later, are what is wrong here
        assert attn(L, Lq=2, qs=strides, ws=None)[0] == 8
        assert tokens(L, cache(), ks=strides, lens=1 << 20 | 2) == 3
    assert tokens(L, cache(n=1), n=1, call="read", ks=(0, 0, 128), lens=1 << 20 | 2) == 3
    assert attn(L, B=1, pre=None, suf=cache(n=1), os_=(0, 0, 128), ws=None)[0] == 8
