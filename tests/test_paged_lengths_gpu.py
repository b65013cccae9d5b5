"""Lengths that a sequence cannot have: past its page table, negative, at the ends of int32 (GPU).  Such rows see nothing, the
device status says so where the length is past the table, and the other sequences' results are as ever."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P
from test_paged_gpu import BF, HF, TYPES, _problem, _randn

pytestmark = pytest.mark.gpu
LENGTHS = {"steps": [(1, 200), (1, 150), (2, 90)], "prompts": [(130, 200), (64, 150), (40, 90)],
           "both": [(1, 200), (100, 150), (1, 90)]}
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("bad", [MOST, MOST - 31, MOST - 127, MOST - 8191, MOST - 8192, 16 * 14 + 1, -1, -MOST - 1, 0])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0)])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_rows_see_nothing(dtype, cache_dtype, lengths, causal, window, bad):
    batch, q, cache = _problem(LENGTHS[lengths], 2, 3, 64, 16, dtype, cache_dtype, seed=600)     # 13 + 1 pages a row
    assert batch.pages.shape[1] == 14
    how = dict(causal=causal, window=window, sinks=3, return_lse=True)
    want, want_lse = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, **how)
    assert mk.device_status()[0] == mk.MK_OK
    for which in (0, 1):
        length = batch.kv_len.clone()
        length[which] = bad
        out, lse = mk.paged_attention(q, cache, batch.cu_q, length, batch.pages, **how)
        assert mk.device_status()[0] == (mk.MK_ERR_CAPACITY if bad > 16 * 14 else mk.MK_OK)
        rows = torch.zeros(batch.tokens, dtype=torch.bool, device="cuda")
        rows[batch.cu[which]:batch.cu[which + 1]] = True
        assert bool((out[rows] == 0).all()) and bool((lse[rows] == float("-inf")).all())
        assert torch.equal(out[~rows], want[~rows]) and torch.equal(lse[~rows], want_lse[~rows])


@pytest.mark.parametrize("cache_dtype", [BF, HF, P.E4M3])
@pytest.mark.parametrize("bad", [MOST, -1, -MOST - 1, 3])
def test_tokens_without_a_slot_are_not_stored(cache_dtype, bad):
    dtype = HF if cache_dtype == HF else BF
    batch = P.Batch([(20, 40), (5, 60)], 16, seed=610)
    caches = [mk.KVCache.empty(batch.n_pages, 2, 16, 64, cache_dtype) for _ in range(2)]
    k, v = (_randn((25, 2, 64), dtype, s) for s in (1, 2))
    freqs, _ = mk.rope_freqs(64)
    mk.kv_append(caches[0], k[20:], v[20:], batch.cu_q[1:] - 20, batch.kv_len[1:], batch.pages[1:], freqs=freqs)
    assert mk.device_status()[0] == mk.MK_OK
    length = batch.kv_len.clone()
    length[0] = bad
    mk.kv_append(caches[1], k, v, batch.cu_q, length, batch.pages, freqs=freqs)
    assert mk.device_status()[0] == mk.MK_ERR_CAPACITY
    mine = [p for p in range(batch.n_pages) if p != batch.table[0][0]]      # bad = 3: the last three tokens have slots there
    for a, b in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
        assert torch.equal(a.view(torch.uint8)[mine], b.view(torch.uint8)[mine])
