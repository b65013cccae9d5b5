"""Row offsets (cu_q) that are no offsets: nothing outside the call's rows is read or written, and the sequences whose own
offsets are right have their results (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_paged_gpu import TYPES, _problem

pytestmark = pytest.mark.gpu
LOW, MOST = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("bad", [LOW, LOW + 3, -1, MOST])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_decode_steps(dtype, cache_dtype, bad):
    lengths = [(2, 200), (1, 90), (2, 150), (1, 70)]
    batch, q, cache = _problem(lengths, 2, 4, 128, 16, dtype, cache_dtype, seed=700)
    want = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, max_q=2)
    assert mk.device_status()[0] == mk.MK_OK
    cu = batch.cu_q.clone()
    cu[2] = bad                                  # the end of sequence 1 and the start of sequence 2
    room = torch.full((batch.tokens + 64, 8, 128), 7.0, dtype=q.dtype, device="cuda")
    out = room[32:32 + batch.tokens]
    mk.paged_attention(q, cache, cu, batch.kv_len, batch.pages, max_q=2, out=out)
    mk.device_status()
    # sequence 1 may reach past its rows, to the last row of the call: sequence 0's are before them
    assert torch.equal(out[:2], want[:2])
    if bad < 0:                                  # neither of the two has rows
        assert torch.equal(out[5:], want[5:]) and bool((out[2:5] == 7).all())
    assert bool((room[:32] == 7).all()) and bool((room[32 + batch.tokens:] == 7).all())
