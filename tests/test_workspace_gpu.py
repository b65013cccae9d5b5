"""The default workspace under graphs: a graph keeps the buffer that it was captured with, and a buffer made while
capturing is cleared before a call outside the graph uses it (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P
from test_paged_gpu import BF, _check, _problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def test_a_graph_outlives_the_growth_of_its_workspace():
    batch, q, cache = _problem([(1, 700), (1, 90)], 2, 4, 128, 16, BF, BF, seed=150)
    large = _problem([(600, 900), (1, 40)], 2, 4, 128, 16, BF, BF, seed=151)
    ws = mk.Workspace()
    call = lambda: mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, workspace=ws, max_q=1)  # noqa: E731
    want = call().clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    old = ws.buf.data_ptr()
    _check(*large, workspace=ws)
    assert ws.buf.data_ptr() != old
    torch.cuda.synchronize()
    free = [torch.full((1 << 18,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert all(not t.data_ptr() <= old < t.data_ptr() + t.numel() for t in free)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(bool((t == 7).all()) for t in free)


def test_a_call_after_a_capture_that_made_the_workspace():
    batch, q, cache = _problem([(1, 3000)], 2, 4, 128, 16, BF, BF, seed=152)
    want = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, max_q=1)
    ws = mk.Workspace()
    call = lambda: mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, workspace=ws, max_q=1)  # noqa: E731
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    ws.buf.fill_(1)                     # what such memory may hold
    assert torch.equal(call(), want)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(call(), want)
