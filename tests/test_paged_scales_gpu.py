"""Attention over 8-bit caches whose page scales and queries span many orders of magnitude, against 64 bits (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P

pytestmark = pytest.mark.gpu
LENGTHS = {"steps": [(1, 200), (2, 65), (1, 1000), (4, 4)], "prompts": [(300, 300), (130, 700), (64, 64), (1, 90)]}


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def _run(lengths, d, page, group, k_scales, v_scales, rows, causal, window, seed):
    batch = P.Batch(LENGTHS[lengths], page, seed=seed)
    k, v, ks, vs = P.random_cache(batch.n_pages, 2, page, d, P.E4M3, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    pick = lambda values: torch.tensor(values)[torch.randint(len(values), ks.shape, generator=g)].cuda()
    ks, vs = pick(k_scales), pick(v_scales)
    P.poison(k, ks, batch)
    P.poison(v, vs, batch)
    q = torch.randn(batch.tokens, 2 * group, d, generator=g)
    q *= torch.tensor(rows)[torch.randint(len(rows), (batch.tokens, 2 * group, 1), generator=g)]
    q = q.bfloat16().cuda()
    cache = mk.KVCache(k, v, ks, vs)
    out, lse = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, return_lse=True, causal=causal,
                                  window=window)
    want, want_lse, tol, tol_lse = P.attention(q, k, v, ks, vs, batch, causal=causal, window=window)
    assert mk.device_status()[0] == mk.MK_OK
    assert float(((out.double().cpu() - want).abs() - tol).max()) <= 0
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse.cpu()), empty)
    assert float(((lse.double().cpu() - want_lse).abs() - tol_lse)[~empty].max()) <= 0


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 37)])
@pytest.mark.parametrize("d,page,group", [(128, 16, 4), (64, 64, 3)])
@pytest.mark.parametrize("lengths", list(LENGTHS))
def test_key_scales(lengths, d, page, group, causal, window):
    """Scales of zero and next to it, beside masked keys; queries of zero, tiny ones and large ones."""
    _run(lengths, d, page, group, [0.0, 2.0 ** -120, 1e-20, 2.0 ** -9, 2.0 ** -6], [2.0 ** -7], [0.0, 2.0 ** -100, 2.0 ** -35, 1.0, 8.0],
         causal, window, seed=71)


@pytest.mark.parametrize("d,page,group", [(128, 16, 4), (64, 64, 3)])
@pytest.mark.parametrize("lengths", list(LENGTHS))
def test_value_scales(lengths, d, page, group):
    _run(lengths, d, page, group, [2.0 ** -8, 2.0 ** -5], [0.0, 2.0 ** -30, 2.0 ** -7, 2.0 ** 10], [1.0], True, 0, seed=72)


@pytest.mark.parametrize("lengths", list(LENGTHS))
def test_large_queries(lengths):
    """Query rows far outside fp16's range, brought back by the keys' scales."""
    _run(lengths, 128, 32, 4, [2.0 ** -48, 2.0 ** -47], [2.0 ** -7], [2.0 ** 40], True, 0, seed=73)
