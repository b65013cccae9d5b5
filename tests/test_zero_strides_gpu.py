"""Expanded tensors through the public calls (GPU): inputs that are only read may be, others are refused."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P
from test_paged_gpu import BF, _ok, _problem, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def test_inputs_that_are_read_row_by_row_may_be_expanded():
    freqs, _ = mk.rope_freqs(64)
    x = _randn((5, 1, 64), BF, 1)
    assert torch.equal(mk.rope(x.expand(5, 3, 64), freqs), mk.rope(x.repeat(1, 3, 1), freqs))
    batch = P.Batch([(3, 20), (2, 2)], 16, seed=2)
    caches = [mk.KVCache.empty(batch.n_pages, 3, 16, 64) for _ in range(2)]
    k, v, q = (_randn((5, 1, 64), BF, s) for s in (3, 4, 5))
    args = (batch.cu_q, batch.kv_len, batch.pages)
    a = mk.kv_append(caches[0], k.expand(5, 3, 64), v.expand(5, 3, 64), *args, q=q.expand(5, 6, 64), freqs=freqs)
    b = mk.kv_append(caches[1], k.repeat(1, 3, 1), v.repeat(1, 3, 1), *args, q=q.repeat(1, 6, 1), freqs=freqs)
    assert torch.equal(a, b) and torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    _ok()


@pytest.mark.parametrize("n", [1, 100])
def test_attention_takes_expanded_queries_and_refuses_expanded_caches_and_outputs(n):
    batch, q, cache = _problem([(n, 200), (n, 150)], 2, 2, 64, 16, BF, BF, seed=6)
    args = (batch.cu_q, batch.kv_len, batch.pages)
    for wide in (q[:, :1].expand_as(q), q[:1].expand_as(q), q[:1, :1].expand_as(q)):
        got, lse = mk.paged_attention(wide, cache, *args, return_lse=True)
        want, want_lse, tol, tol_lse = P.attention(wide, cache.k, cache.v, None, None, batch)
        assert bool(((got.double().cpu() - want).abs() <= tol).all())
        assert bool(((lse.double().cpu() - want_lse).abs() <= tol_lse).all())
    shared = mk.KVCache(cache.k[:, :1].expand_as(cache.k), cache.v[:, :1].expand_as(cache.v))
    with pytest.raises(mk.MkError):
        mk.paged_attention(q, shared, *args)
    with pytest.raises(mk.MkError):
        mk.paged_attention(q, cache, *args, out=torch.empty(1, 4, 64, dtype=BF, device="cuda").expand_as(q))
    with pytest.raises(mk.MkError):
        mk.rope(q, mk.rope_freqs(64)[0], out=torch.empty(1, 4, 64, dtype=BF, device="cuda").expand_as(q))
    one = P.Batch([(1, 9)], 16, seed=7, spare=0)       # one page, one head: no stride to speak of
    k, v, _, _ = P.random_cache(1, 1, 16, 64, BF, 8)
    q1 = _randn((1, 2, 64), BF, 9)
    out = mk.paged_attention(q1, mk.KVCache(k, v), one.cu_q, one.kv_len, one.pages)
    want, _, tol, _ = P.attention(q1, k, v, None, None, one)
    assert bool(((out.double().cpu() - want).abs() <= tol).all())
    _ok()
