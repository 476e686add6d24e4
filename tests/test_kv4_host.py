"""What the 4-bit cache's calls refuse on the host (CPU only): sizes whose products pass 64 bits."""
import pytest

from test_kv4_abi import L, cache, tokens  # noqa: F401


@pytest.mark.parametrize("call", ["append", "read"])
@pytest.mark.parametrize("n,Hkv,new", [(1 << 30, 65536, 1 << 30), (1 << 30, 65536, 1 << 23), (1 << 30, 65536, 1 << 22), (1 << 30, 1, 1 << 30),
                                       (1 << 30, 65535, 1 << 30), (1 << 26, 32768, 1)])
def test_grids_beyond_any_launch(L, call, n, Hkv, new):  # noqa: F811
    assert tokens(L, cache(n=n, Hkv=Hkv, T=1 << 30), n=new, call=call) == 2
