"""Prompts with scores far from 0, where the softmax's reference has steps of many units (GPU)."""
import pytest
import torch

import far_scores as F
import paged_util as P
from test_paged_gpu import BF, HF, TYPES, _check, _problem

pytestmark = pytest.mark.gpu
LENGTHS = [(100, 100), (130, 200), (0, 50), (40, 30), (33, 110), (64, 64)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("sign", ["+", "-", "+-"])
@pytest.mark.parametrize("power", [19, 23, 26, 28, 30])
@pytest.mark.parametrize("d,page,heads,group", [(128, 16, 2, 4), (64, 64, 1, 3)])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_the_largest_score_takes_all(dtype, cache_dtype, d, page, heads, group, power, sign):
    F.one_key_wins(LENGTHS, d, page, heads, group, dtype, cache_dtype, sign, power, seed=300)


@pytest.mark.parametrize("power", [35, 60])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
@pytest.mark.parametrize("cache_dtype", [BF, P.E4M3])
def test_larger_than_fp16_holds(cache_dtype, causal, window, power):
    F.one_key_wins(LENGTHS, 128, 32, 1, 4, BF, cache_dtype, "+-", power, seed=310, causal=causal, window=window)


@pytest.mark.parametrize("one_run", [True, False])
@pytest.mark.parametrize("power", [20, 27, 30])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_equal_scores(dtype, cache_dtype, power, one_run):
    F.all_keys_alike(LENGTHS, 64, 16, 1, 3, dtype, cache_dtype, power, 320, one_run)


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
def test_ordinary_rows_beside_far_ones(dtype, cache_dtype, causal):
    F.ordinary_rows_beside(_problem([(300, 300), (130, 700), (33, 400)], 1, 6, 128, 16, dtype, cache_dtype, seed=330), _check,
                           causal=causal)
