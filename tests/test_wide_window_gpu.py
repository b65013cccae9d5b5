"""Windows as wide as their type allows hide nothing (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_paged_gpu import PROMPTS, STEP, TYPES, _check, _ok, _problem

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window,sinks", [(MOST, 0), (MOST, MOST), (MOST - 40, 0), (7, MOST)])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("lengths", ["step", "prompts"])
def test_every_key_is_seen(lengths, dtype, cache_dtype, window, sinks, causal):
    problem = _problem(STEP if lengths == "step" else PROMPTS, 2, 3, 64, 16, dtype, cache_dtype, seed=25)
    out, lse = _check(*problem, causal=causal, window=window, sinks=sinks)
    batch, q, cache = problem
    want = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, causal=causal)
    _ok()
    assert torch.equal(out, want)
