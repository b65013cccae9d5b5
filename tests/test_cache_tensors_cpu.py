"""A cache's tensors are those it was made of: its calls go by their addresses, so they cannot be replaced (CPU only)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from bind_util import Fake
from comm_gemm_tile_gb300 import build as mkbuild


@pytest.mark.parametrize("name", ["k", "v", "k_scale", "v_scale"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_caches_tensors_cannot_be_replaced(dtype, name):
    mkbuild.build()
    kv = [Fake((8, 2, 16, 64), dtype) for _ in range(2)]
    scales = [Fake((8, 2), torch.float32) if dtype == torch.float8_e4m3fn else None for _ in range(2)]
    cache = mk.KVCache(*kv, *scales)
    was = getattr(cache, name)
    assert was is dict(k=kv[0], v=kv[1], k_scale=scales[0], v_scale=scales[1])[name]
    with pytest.raises(AttributeError):
        setattr(cache, name, Fake((16, 2, 16, 64), dtype))
    with pytest.raises(AttributeError):
        delattr(cache, name)
    assert getattr(cache, name) is was
