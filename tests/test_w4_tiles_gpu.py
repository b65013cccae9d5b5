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


def whole(m, n, k, group, zeros, dtype, seed):
    """x, a weight and y in 64 bits, of small whole numbers and scales of powers of two: every product and sum is a multiple of
    1/4 below 2^22, so that fp32 has each exactly, in any order."""
    g = torch.Generator().manual_seed(seed)
    # |x| <= 4, |c - z| <= 15, scales 1/4 .. 2: at most 120 k, and k is below 2^15
    x = torch.randint(-4, 5, (m, k), generator=g).to(dtype).cuda()
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).cuda()
    scales = (2.0 ** torch.randint(-2, 2, (n, k // group), generator=g)).to(dtype).cuda()
    z = torch.randint(0, 16, (n, k // group), generator=g).to(dtype).cuda() if zeros else None
    w = mk.W4Weight(codes, scales, z)
    return x, w, formula(x, w)[0]


# every number of tokens a tile has (16, 32, 64) and what is past it; k with a half of a step at its end, and one step or less
SIZES = [(9, 4104, 8320), (16, 4104, 8320), (17, 2100, 8320), (32, 4104, 4224), (33, 4104, 4224), (64, 2100, 8320), (65, 2100, 4224),
         (130, 1001, 8320), (1100, 4096, 128), (1100, 4097, 256), (600, 4100, 384)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_whole_numbers_are_exact(m, n, k, group, dtype):
    """fp32 outputs are the 64-bit sums, 16-bit ones those rounded once: one wrong code, scale or sum of x shows."""
    for zeros in (False, True):
        x, w, want = whole(m, n, k, group, zeros, dtype, seed=m + n)
        assert reaches(w, m)
        assert torch.equal(mk.w4_gemm(x, w, out_dtype=F32).double(), want)
        assert torch.equal(mk.w4_gemm(x, w), want.to(dtype))


@pytest.mark.parametrize("m,k", [(1400, 96), (4200, 32), (2200, 64), (900, 160), (700, 224)])
def test_rows_of_few_groups(m, k):
    for zeros in (False, True):
        x, w, want = whole(m, 4100, k, 32, zeros, BF, seed=k)
        assert reaches(w, m)
        assert torch.equal(mk.w4_gemm(x, w, out_dtype=F32).double(), want)
        assert torch.equal(mk.w4_gemm(x, w), want.to(BF))


@pytest.mark.parametrize("ctas", [1, 2, 5, 151])
@pytest.mark.parametrize("m,n,k,group", [(16, 4104, 8320, 32), (40, 2100, 8320, 64), (1400, 4100, 96, 32), (130, 1001, 8320, 128)])
def test_runs_of_any_length(m, n, k, group, ctas):
    """Steps cut into any number of runs and joined: the same whole numbers."""
    x, w, want = whole(m, n, k, group, True, HF, seed=22)
    assert reaches(w, m)
    assert torch.equal(mk.w4_gemm(x, w, out_dtype=F32, cfg=mk.Config(max_ctas=ctas)).double(), want)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("m,n,k,group,zeros", [(16, 4104, 8320, 64, True), (16, 8200, 4224, 32, False), (48, 2100, 8320, 128, False),
                                               (70, 2100, 8320, 64, True), (40, 2100, 8320, 32, True)])
def test_any_numbers(m, n, k, group, zeros, dtype):
    """Both outputs within the bound of test_w4_gpu, rounded once to theirs."""
    x, w = problem(m, n, k, group, zeros, dtype, seed=23)
    assert reaches(w, m)
    want, size = formula(x, w)
    fp32 = (k / 16 + k // group + 32) * 2.0 ** -22 * size
    y = mk.w4_gemm(x, w, out_dtype=F32)
    assert bool(((y.double() - want).abs() <= fp32).all())
    assert torch.equal(mk.w4_gemm(x, w), y.to(dtype))        # (the same sums)
    # what such sums are off as a rule: each of k / 16 + groups additions by 2^-24 of sums that grow with the square root of k
    rms = float((y.double() - want).square().mean().sqrt() / want.square().mean().sqrt())
    assert rms <= (k / 16 + k // group) * 2.0 ** -24


@pytest.mark.parametrize("m,zeros", [(16, True), (48, False), (70, True)])
def test_strides_and_outputs(m, zeros):
    n, k = 4104, 8320
    x, w = problem(m, n, k, 64, zeros, HF, seed=24)
    assert reaches(w, m)
    want = mk.w4_gemm(x, w)
    for dtype in (HF, F32):
        room = torch.full((m, n + 40), 5.0, dtype=dtype, device="cuda")
        got = mk.w4_gemm(x, w, out_dtype=dtype, out=room[:, 3:3 + n])
        assert torch.equal(got.to(HF), want)
        assert bool((room[:, :3] == 5).all()) and bool((room[:, 3 + n:] == 5).all())
    wide = torch.full((2 * m, k + 64), float("nan"), dtype=HF, device="cuda")
    wide[::2, 64:] = x
    assert torch.equal(mk.w4_gemm(wide[::2, 64:], w), want)
    one = mk.w4_gemm(x[:1].expand(m, k), w)
    assert torch.equal(one, want[:1].expand(m, n))


@pytest.mark.parametrize("m,group,zeros", [(16, 64, True), (20, 32, True), (64, 128, False), (70, 64, True)])
def test_tokens_do_not_depend_on_each_other(m, group, zeros):
    x, w = problem(m, 4104, 8320, group, zeros, BF, seed=25)
    assert reaches(w, m)
    want = mk.w4_gemm(x, w)
    x[3, 5] = float("nan")
    x[4] = 0
    x[m - 1, 8319] = float("inf")
    got = mk.w4_gemm(x, w)
    rest = [i for i in range(m) if i not in (3, 4, m - 1)]
    assert torch.equal(got[rest], want[rest])
    assert bool(got[3].isnan().all()) and bool((got[4] == 0).all()) and not bool(got[m - 1].isfinite().any())


def test_no_rows_and_no_tokens():
    x, w = problem(3, 5, 128, 64, True, BF)
    assert mk.w4_gemm(x[:0], w).shape == (0, 5)
    none = mk.W4Weight(w.codes[:0], w.scales[:0], w.zeros[:0])
    assert mk.w4_gemm(x, none).shape == (3, 0)
