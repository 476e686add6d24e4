"""Settings of token sampling beyond what the library's own fields hold."""
import pytest
import torch

import nvfp4_weight_only_quantize_gb300 as q

pytestmark = pytest.mark.gpu


def test_top_k_beyond_32_bits_is_no_cut():
    x = torch.randn(4, 300, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    u = torch.tensor([0.1, 0.6, 0.9, 0.99], device="cuda")
    for k in (300, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 40 + 7):
        for a, b in zip(q.qerl_sample(x, u), q.qerl_sample(x, u, top_k=k)):
            assert torch.equal(a, b)
    with pytest.raises(q.QerlError):
        q.qerl_sample(x, u, top_k=5 - 2 ** 32)
