"""The tcgen05 kernel of the 4-bit products, at sizes that reach it (GPU); tolerances of test_w4_gpu."""
import ctypes

import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_w4_gpu import BF, F32, HF, formula, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def reaches(w, m):
    """Whether a call takes scratch: only this kernel does."""
    return mk.lib().mk_w4_gemm_scratch_size(ctypes.byref(mk._W4.from_buffer_copy(w._w)), m) > 0


@pytest.mark.parametrize("m,n,k,group", [(16, 8200, 8288, 32), (40, 4104, 8320, 32), (16, 8200, 8256, 64), (64, 4104, 8256, 64),
                                         (64, 4104, 8320, 128)])
def test_sums_of_x_are_their_own_steps(m, n, k, group):
    """Groups of x whose sums are far from each other's, so that a sum of another step would be far off; everything out of
    the caches and rows of scales that lie anywhere, so that their loads hold up the others."""
    x, w = problem(m, n, k, group, True, BF, seed=21)
    groups = torch.arange(k // group, device="cuda")
    x = (x.float().abs() * (4.0 ** (groups * 5 % 7)).repeat_interleave(group)).to(BF)
    assert reaches(w, m)
    want, size = formula(x, w)
    flush = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(12):
        flush.add_(1)
        y = mk.w4_gemm(x, w, out_dtype=F32)
        assert bool(((y.double() - want).abs() <= (k / 16 + k // group + 32) * 2.0 ** -22 * size).all())
