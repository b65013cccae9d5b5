"""One Workspace for calls that keep flags and status in it and calls whose scratch holds nothing: each gives what it gives
with a Workspace of its own, in any order (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_paged_gpu import _problem

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def draw(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def _flat(r):
    if isinstance(r, torch.Tensor):
        return [r]
    r = r.values() if isinstance(r, dict) else r
    return [t for x in r if x is not None for t in _flat(x)]


def test_one_workspace():
    x, dy, w = draw((500, 1024), BF, 1), draw((500, 1024), BF, 2), draw((1024,), F32, 3)
    logits = draw((5000, 96), F32, 4)
    a, b = [draw((256, 512), BF, 5 + r) for r in range(2)], draw((512, 512), BF, 7)
    few, four = draw((48, 8192), BF, 9), mk.W4Weight.quantize(draw((4096, 8192), F32, 10))
    batch, q, cache = _problem([(1, 3000), (1, 90)], 2, 4, 128, 16, BF, BF, seed=11)
    route = lambda ws: mk.moe_route(logits, 4, workspace=ws)   # noqa: E731
    grad = lambda ws: mk.rms_norm_backward(dy, x, w, workspace=ws)   # noqa: E731
    fused = [lambda ws: mk.ag_gemm(a, b, workspace=ws), lambda ws: mk.w4_gemm(few, four, workspace=ws)]
    decode = [lambda ws: mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, max_q=1, workspace=ws)]
    for others in (fused, decode):                     # (attention keeps its counts where the fused calls keep flags)
        calls = [route, grad, *others]
        want = [[t.clone() for t in _flat(c(mk.Workspace()))] for c in calls]
        ws = mk.Workspace()
        for turn in range(3):
            for i in [0, 2, 1, *range(2, len(calls)), 0, 1, *range(2, len(calls))]:
                got = _flat(calls[i](ws))
                assert len(got) == len(want[i]) and all(torch.equal(g, h) for g, h in zip(got, want[i])), (turn, i)
                assert mk.device_status(ws)[0] == mk.MK_OK, (turn, i)
