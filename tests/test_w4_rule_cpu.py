"""Which calls of the 4-bit products are the tcgen05 kernel's (those that take scratch): the sides that were measured faster, and
both sides of every size the rule has (CPU only)."""
import ctypes

import pytest

import comm_gemm_tile_gb300 as mk
from comm_gemm_tile_gb300 import build as mkbuild
from test_layer_calls_cpu import GOOD, weight


@pytest.fixture(scope="module")
def L():
    mkbuild.build()
    return mk.lib()


def tiles(L, m, n, k, group, zeros):
    return L.mk_w4_gemm_scratch_size(ctypes.byref(weight(n=n, k=k, group=group, zeros=GOOD if zeros else None)), m) > 0


@pytest.mark.parametrize("m,n,k,group,zeros,want", [
    (1, 28672, 8192, 128, False, False), (1, 28672, 8192, 128, True, True), (8, 28672, 8192, 32, False, True),
    (1, 16384, 8192, 64, True, True), (1, 16383, 8192, 64, True, False), (1, 8192, 8192, 32, True, False),
    (16, 4096, 4096, 32, True, False), (9, 4097, 4096, 64, True, True), (16, 8192, 4096, 32, False, False), (9, 8193, 4096, 128, False, True),
    (17, 4096, 4096, 64, False, False), (32, 4096, 4096, 64, False, False), (32, 4096, 4096, 128, True, False), (17, 4097, 4096, 64, False, True),
    (64, 2048, 4096, 64, False, False), (33, 2049, 4096, 32, True, True), (128, 2048, 2048, 64, False, False), (128, 2048, 4096, 64, False, True),
    (1 << 21, 1, 32, 32, False, True)])
def test_sides(L, m, n, k, group, zeros, want):
    assert tiles(L, m, n, k, group, zeros) == want


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_more_tokens_of_a_large_matrix_stay(L, zeros, group):
    """Once a matrix is this kernel's it stays that for more tokens, from 17 on."""
    for n, k in ((4097, 4096), (1024, 4096), (300, 256)):
        was = False
        for m in (17, 32, 33, 64, 65, 128, 1000, 8192, 100000):
            now = tiles(L, m, n, k, group, zeros)
            assert now or not was
            was = now
