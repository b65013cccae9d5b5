"""Decode attention with everything out of the caches: the loads of pages and scales then hold up the tiles' own, and a stage that
was filled again before every lane had its values would change the result (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P
from test_paged_gpu import BF, HF, _check, _problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("dtype,cache_dtype", [(BF, BF), (HF, HF), (BF, P.E4M3)])
@pytest.mark.parametrize("heads,heads_q,d,new", [(2, 8, 128, 1), (4, 16, 64, 2), (2, 32, 128, 1)])
def test_cold_caches(heads, heads_q, d, new, dtype, cache_dtype):
    lengths = [(new, 3000 + 517 * i) for i in range(12)]
    batch, q, cache = _problem(lengths, heads, heads_q // heads, d, 16, dtype, cache_dtype, seed=160)
    _check(batch, q, cache)
    call = lambda: mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, max_q=new)  # noqa: E731
    want = call()
    flush = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(12):
        flush.add_(1)
        assert torch.equal(call(), want)
    assert mk.device_status()[0] == mk.MK_OK
