"""Decode steps with scores far from 0 (GPU)."""
import pytest
import torch

import far_scores as F
import paged_util as P
from test_paged_gpu import BF, TYPES, _check, _problem

pytestmark = pytest.mark.gpu
LENGTHS = [(1, 200), (2, 130), (4, 64), (1, 1), (3, 2), (0, 20), (1, 142)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("sign", ["+", "-", "+-"])
@pytest.mark.parametrize("power", [19, 23, 26, 27, 28, 30])
@pytest.mark.parametrize("d,page,heads,group", [(128, 16, 2, 4), (64, 64, 1, 3), (128, 32, 1, 2)])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_the_largest_score_takes_all(dtype, cache_dtype, d, page, heads, group, power, sign):
    F.one_key_wins(LENGTHS, d, page, heads, group, dtype, cache_dtype, sign, power, seed=400, max_q=4)


@pytest.mark.parametrize("power", [35, 60])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 50)])
@pytest.mark.parametrize("cache_dtype", [BF, P.E4M3])
def test_larger_than_fp16_holds(cache_dtype, causal, window, power):
    F.one_key_wins(LENGTHS, 128, 32, 1, 4, BF, cache_dtype, "+-", power, seed=410, causal=causal, window=window, max_q=4)


@pytest.mark.parametrize("one_run", [True, False])
@pytest.mark.parametrize("power", [20, 26, 27, 30])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_equal_scores(dtype, cache_dtype, power, one_run):
    F.all_keys_alike(LENGTHS + [(1, 3000)], 64, 16, 1, 3, dtype, cache_dtype, power, 420, one_run, max_q=4)


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("causal", [True, False])
def test_ordinary_rows_beside_far_ones(dtype, cache_dtype, causal):
    F.ordinary_rows_beside(_problem([(1, 300), (2, 700), (1, 5000)], 2, 6, 128, 16, dtype, cache_dtype, seed=430), _check,
                           causal=causal, max_q=2)
