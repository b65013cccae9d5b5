"""A default or own workspace whose first use is inside a capture: every graph captured before a call outside clears it
(GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_paged_gpu import BF, _problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def _capture(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


@pytest.mark.parametrize("grown", [False, True])
def test_the_second_of_two_captures_is_replayed_first(grown):
    """One sequence over every CTA: its cut rows are joined only if the counts of CTAs start from zero."""
    batch, q, cache = _problem([(1, 9000)], 2, 4, 128, 16, BF, BF, seed=160)
    args = (q, cache, batch.cu_q, batch.kv_len, batch.pages)
    want = mk.paged_attention(*args, max_q=1)
    ws = mk.Workspace()
    if grown:                                   # made by a call outside, outgrown by the first capture
        ws.get(256)
    torch.cuda.synchronize()
    first, a = _capture(lambda: mk.paged_attention(*args, max_q=1, workspace=ws))
    second, b = _capture(lambda: mk.paged_attention(*args, max_q=1, workspace=ws))
    ws.buf.fill_(1)                             # what such memory may hold
    second.replay()
    torch.cuda.synchronize()
    assert torch.equal(b, want)
    first.replay()
    second.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)
    assert torch.equal(mk.paged_attention(*args, max_q=1, workspace=ws), want)
    assert mk.device_status(ws)[0] == mk.MK_OK


def test_a_capture_on_a_stream_given_by_name():
    """The clearing is ordered before the call on the call's own stream."""
    batch, q, cache = _problem([(1, 9000)], 2, 4, 128, 16, BF, BF, seed=161)
    args = (q, cache, batch.cu_q, batch.kv_len, batch.pages)
    want = mk.paged_attention(*args, max_q=1)
    ws, side = mk.Workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        out = mk.paged_attention(*args, max_q=1, workspace=ws, stream=side)
        here.wait_stream(side)
    ws.buf.fill_(1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
