"""Paged attention when a wait runs out: an error status, and the next call on the same workspace as ever (GPU)."""
import time

import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_paged_gpu import TYPES, _check, _problem

pytestmark = pytest.mark.gpu
LENGTHS = {"steps": [(1, 9000), (1, 700), (2, 3000)], "prompts": [(300, 900), (130, 700), (16, 2000)],
           "both": [(1, 4000), (300, 900), (1, 70)]}


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_a_loader_that_stops(dtype, cache_dtype, lengths):
    """With a few CTAs each has more tiles than the loader of the first one brings."""
    problem = _problem(LENGTHS[lengths], 2, 4, 128, 16, dtype, cache_dtype, seed=500)
    batch, q, cache = problem
    args = (q, cache, batch.cu_q, batch.kv_len, batch.pages)
    ws = mk.Workspace()
    want = mk.paged_attention(*args, workspace=ws, cfg=mk.Config(max_ctas=8))
    assert mk.device_status(ws)[0] == mk.MK_OK
    t0 = time.perf_counter()
    mk.paged_attention(*args, workspace=ws, cfg=mk.Config(max_ctas=8, inject=1, wait_limit_ns=20_000_000))
    status, _ = mk.device_status(ws)
    assert status == mk.MK_ERR_TIMEOUT and time.perf_counter() - t0 < 5.0
    again = mk.paged_attention(*args, workspace=ws, cfg=mk.Config(max_ctas=8))
    assert mk.device_status(ws)[0] == mk.MK_OK
    assert torch.equal(again, want)
    _check(*problem, workspace=ws)


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_waits_given_no_time(dtype, cache_dtype, lengths):
    """Whether a wait runs out is the moment's; nothing is left in flight either way."""
    batch, q, cache = _problem(LENGTHS[lengths], 2, 4, 128, 16, dtype, cache_dtype, seed=510)
    args = (q, cache, batch.cu_q, batch.kv_len, batch.pages)
    ws = mk.Workspace()
    want = mk.paged_attention(*args, workspace=ws)
    for _ in range(10):
        mk.paged_attention(*args, workspace=ws, cfg=mk.Config(wait_limit_ns=1))
        assert mk.device_status(ws)[0] in (mk.MK_OK, mk.MK_ERR_TIMEOUT)
        assert torch.equal(mk.paged_attention(*args, workspace=ws), want)
        assert mk.device_status(ws)[0] == mk.MK_OK
