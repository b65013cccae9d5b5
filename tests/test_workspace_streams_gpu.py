"""A workspace outgrown while a call on another stream still uses it (GPU)."""
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


@pytest.mark.parametrize("named", [True, False])
def test_an_outgrown_buffer_is_not_handed_out_while_it_is_in_use(named):
    """Small call, then a larger one, both on a side stream that is busy for a while; what the default stream allocates
    meanwhile must not be the memory that the small call still writes."""
    small = _problem([(1, 3000), (1, 90)], 2, 4, 128, 16, BF, BF, seed=170)
    large = _problem([(600, 900), (1, 40)], 2, 4, 128, 16, BF, BF, seed=171)
    call = lambda problem, n, **how: mk.paged_attention(problem[1], problem[2], problem[0].cu_q, problem[0].kv_len,  # noqa: E731
                                                        problem[0].pages, max_q=n, **how)
    wants = [call(small, 1), call(large, 600)]
    ws, side = mk.Workspace(), torch.cuda.Stream()
    call(small, 1, workspace=ws)                # the buffer is the default stream's
    torch.cuda.synchronize()
    old, size = ws.buf.data_ptr(), ws.buf.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)          # about 0.2 s
    if named:
        outs = [call(p, n, workspace=ws, stream=side) for p, n in ((small, 1), (large, 600))]
    else:
        with torch.cuda.stream(side):
            outs = [call(p, n, workspace=ws) for p, n in ((small, 1), (large, 600))]
    assert ws.buf.data_ptr() != old
    new = []
    for share in (1, 2, 4):
        new += [torch.full((size // share,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not any(t.data_ptr() < old + size and old < t.data_ptr() + t.numel() for t in new)
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in new)
    assert all(torch.equal(o, w) for o, w in zip(outs, wants))


def test_a_workspace_that_grows_step_by_step_keeps_little():
    ws = mk.Workspace()
    for n in range(1, 400):
        ws.get(n << 12)
    held = ws.buf.numel() + sum(t.numel() for t in ws.kept)
    assert held <= 4 * (400 << 12) and len(ws.kept) <= 12
