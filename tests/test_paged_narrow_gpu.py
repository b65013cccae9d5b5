"""Attention over a paged cache for sequences of a few dozen packed rows: more than a decode step, less than a prompt's
tile, where the key tiles of a segment are shared out between two accumulators (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P
from test_paged_gpu import BF, HF, TYPES, _check, _ok, _problem

pytestmark = pytest.mark.gpu
# new tokens, tokens in all: key tiles 1, 2, 3, many; fewer tokens than rows; ends inside pages and tiles
FEW = [(9, 9), (8, 128), (8, 129), (12, 300), (16, 2500), (10, 7), (5, 1000), (20, 384), (0, 50), (1, 513)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 60, 4), (True, 300, 0), (True, 1, 1)])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("d,page,heads,group", [(128, 16, 2, 4), (64, 64, 1, 6), (128, 256, 1, 3)])
def test_few_rows(d, page, heads, group, dtype, cache_dtype, causal, window, sinks):
    problem = _problem(FEW, heads, group, d, page, dtype, cache_dtype, seed=90)
    _check(*problem, causal=causal, window=window, sinks=sinks)
    _ok()


@pytest.mark.parametrize("ctas", [1, 2, 7, 50])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_runs_cut_anywhere(ctas, dtype, cache_dtype):
    # narrow and wide items in one CTA's run, cut at every kind of place
    problem = _problem(FEW + [(150, 700), (33, 40), (70, 70)], 2, 4, 128, 32, dtype, cache_dtype, seed=91)
    first, _ = _check(*problem, cfg=mk.Config(max_ctas=ctas))
    _ok()
    second, _ = _check(*problem, cfg=mk.Config(max_ctas=ctas))
    assert torch.equal(first, second)


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("at", [3, 140, 200, 290])
def test_nan_values_reach_the_rows_that_see_them(at, dtype, cache_dtype):
    batch, q, cache = _problem([(12, 300)], 1, 4, 64, 16, dtype, cache_dtype, seed=92)
    page, slot = batch.table[0][at // 16], at % 16
    if cache_dtype == P.E4M3:
        cache.v.view(torch.uint8)[page, 0, slot, 5] = 0x7f
    else:
        cache.v[page, 0, slot, 5] = float("nan")
    out = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, window=100)
    _ok()
    pos = 288 + torch.arange(12)
    sees = (at <= pos) & (at > pos - 100)
    nan = torch.isnan(out.float()).cpu()
    assert torch.equal(nan[:, :, 5].all(dim=1), sees) and torch.equal(nan[:, :, 5].any(dim=1), sees)
    nan[:, :, 5] = False
    assert not bool(nan.any())


def test_scores_that_grow_along_the_keys():
    # the running maxima of both halves move many times
    batch, q, cache = _problem([(9, 2000)], 2, 4, 128, 16, BF, BF, seed=93)
    for i, page in enumerate(batch.table[0]):
        cache.k[page] *= 0.05 * (1 + i)
    _check(batch, q, cache, scale=1.0)
    _ok()
