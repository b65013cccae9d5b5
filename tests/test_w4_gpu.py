"""w4_gemm against the formula in 64 bits (GPU).

Tolerance.  Every term x (c - z) s is a product of numbers that fp32 holds; sums are fp32 with at most k / 16 + groups + 32
additions one after another, each off by at most 2^-22 of the sum of the terms' sizes (tensor cores may cut instead of rounding).  With zero points a group's sum is
made of sum x (c - 8) and (8 - z) sum x: their sizes count.  The output is rounded once."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def problem(m, n, k, group, zeros, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, k, generator=g).to(dtype).cuda()
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8).cuda()
    scales = ((torch.rand(n, k // group, generator=g) - 0.3) * 0.1).to(dtype).cuda()
    z = (torch.rand(n, k // group, generator=g) * 15).to(dtype).cuda() if zeros else None
    return x, mk.W4Weight(codes, scales, z)


def formula(x, w):
    """(y, the sum of the sizes of its terms) in 64 bits."""
    n, groups = w.scales.shape
    code = torch.stack((w.codes & 15, w.codes >> 4), dim=-1).view(n, groups, -1).double()
    s = w.scales.double()[..., None]
    zero = torch.full_like(s, 8.0) if w.zeros is None else w.zeros.double()[..., None]
    x = x.double()
    size = (((code - 8).abs() + (8 - zero).abs()) * s.abs()).flatten(1)
    return x @ ((code - zero) * s).flatten(1).t(), x.abs() @ size.t()


def check(x, w, dtype=None, **kw):
    y = mk.w4_gemm(x, w, out_dtype=dtype, **kw)
    want, size = formula(x, w)
    k, groups = x.shape[1], w.scales.shape[1]
    f = torch.finfo(y.dtype)
    tol = want.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2 + (k / 16 + groups + 32) * 2.0 ** -22 * size
    assert y.dtype == (dtype or x.dtype) and y.shape == (x.shape[0], w.codes.shape[0])
    assert bool(((y.double() - want).abs() <= tol).all())
    return y


# tokens: one, a column group's edges, both sides of every tile; rows and k odd, small, several pieces a warp
SIZES = [(1, 1, 1), (1, 16, 1), (2, 17, 2), (3, 100, 3), (7, 33, 5), (8, 640, 8), (9, 129, 9), (16, 333, 4), (17, 64, 17),
         (31, 250, 2), (33, 50, 3), (64, 200, 6), (65, 48, 2), (130, 90, 3), (1, 3584, 16), (10, 20, 1), (40, 129, 1), (3, 8192, 65)]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,groups", SIZES)
def test_products(m, n, groups, group, dtype):
    for zeros in (False, True):
        x, w = problem(m, n, groups * group, group, zeros, dtype, seed=m + n)
        check(x, w)
        check(x, w, F32)


@pytest.mark.parametrize("group,k", [(128, 8192), (64, 8256), (32, 8224)])
@pytest.mark.parametrize("m", [1, 5, 16, 40])
def test_long_rows(m, group, k):
    x, w = problem(m, 80, k, group, True, BF, seed=7)
    check(x, w, F32)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 16136, 8320), (8, 16136, 8320), (9, 4104, 8320), (16, 2056, 8320), (16, 4104, 8320),
                                   (17, 2056, 8320), (32, 4104, 4224), (24, 1000, 8320), (33, 2056, 8320), (64, 2100, 4224),
                                   (65, 1030, 8320), (130, 1001, 4224), (8192, 300, 256), (3000, 77, 128)])
def test_large_matrices(m, n, k, group):
    """Both sides of the sizes from which few tokens are taken another way."""
    for zeros, dtype in ((False, HF), (True, BF)):
        x, w = problem(m, n, k, group, zeros, dtype, seed=m)
        check(x, w, F32)


def test_scales_off_whole_pieces():
    x, w = problem(5, 40, 512, 32, True, BF, seed=14)
    room = torch.zeros(2, 40 * 16 + 8, dtype=BF, device="cuda")
    for off in (1, 2, 4):
        s, z = (r[off:off + 640].view(40, 16) for r in room)
        s.copy_(w.scales)
        z.copy_(w.zeros)
        for a, b in ((s, z), (s, w.zeros), (w.scales, z)):
            check(x, mk.W4Weight(w.codes, a, b))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("m,n,k,group", [(9, 4104, 8320, 32), (40, 4104, 8320, 32), (40, 4224, 8192, 64), (40, 4104, 8320, 128)])
def test_cold_matrices(m, n, k, group, zeros, dtype):
    """Many steps a CTA with everything out of the caches, so that loads of scales hold up the sums and fill the rings."""
    x, w = problem(m, n, k, group, zeros, dtype, seed=15)
    want, size = formula(x, w)
    flush = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(12):
        flush.add_(1)
        y = mk.w4_gemm(x, w, out_dtype=F32)
        assert bool(((y.double() - want).abs() <= (k / 16 + k // group + 32) * 2.0 ** -22 * size).all())


def test_whole_numbers_are_exact():
    """Small whole numbers: every product and sum is exact in fp32, so the bits are those of the 64-bit sums."""
    g = torch.Generator().manual_seed(8)
    for m in (1, 8, 24, 64):
        x = torch.randint(-8, 9, (m, 1024), generator=g).to(HF).cuda()
        codes = torch.randint(0, 256, (96, 512), generator=g, dtype=torch.uint8).cuda()
        scales = (2.0 ** torch.randint(-2, 3, (96, 16), generator=g)).to(HF).cuda()
        zeros = torch.randint(0, 16, (96, 16), generator=g).to(HF).cuda()
        for w in (mk.W4Weight(codes, scales), mk.W4Weight(codes, scales, zeros)):
            assert torch.equal(mk.w4_gemm(x, w, out_dtype=F32).double(), formula(x, w)[0])


def test_strides_and_outputs():
    x, w = problem(12, 70, 256, 64, True, HF)
    want = check(x, w)
    room = torch.full((12, 96), 5.0, dtype=HF, device="cuda")
    assert torch.equal(mk.w4_gemm(x, w, out=room[:, 3:73]), want)
    assert bool((room[:, :3] == 5).all()) and bool((room[:, 73:] == 5).all())
    wide = torch.zeros(24, 320, dtype=HF, device="cuda")
    wide[::2, 64:] = x
    assert torch.equal(mk.w4_gemm(wide[::2, 64:], w), want)
    assert torch.equal(mk.w4_gemm(x[:1].expand(9, 256), w), mk.w4_gemm(x[:1], w).expand(9, 70))
    assert mk.w4_gemm(x[:0], w).shape == (0, 70)


def test_tokens_do_not_depend_on_each_other():
    for m in (8, 16, 64):
        x, w = problem(m, 100, 512, 128, False, BF, seed=9)
        want = mk.w4_gemm(x, w)
        x[3, 5] = float("nan")
        x[4] = 0
        got = mk.w4_gemm(x, w)
        rest = [i for i in range(m) if i not in (3, 4)]
        assert torch.equal(got[rest], want[rest]) and bool(got[3].isnan().all()) and bool((got[4] == 0).all())


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantized_weights(symmetric, dtype):
    """Every weight is within half a scale of its 4-bit form (a little more where the scale or zero point was rounded)."""
    g = torch.Generator().manual_seed(10)
    full = torch.randn(64, 512, generator=g).cuda()
    full[3, :64] = 0
    w = mk.W4Weight.quantize(full, group=64, symmetric=symmetric, dtype=dtype)
    step = w.scales.float().repeat_interleave(64, dim=1)
    eps = torch.finfo(dtype).eps
    assert bool(((w.dequantize(F32) - full).abs() <= step * (0.5 + 16 * eps) + 1e-6).all())
    x = torch.randn(3, 512, generator=g).to(dtype).cuda()
    check(x, w)
    assert bool((w.dequantize(F32)[3, :64] == 0).all()) and w.dequantize().dtype == dtype


@pytest.mark.parametrize("m,n,k", [(4, 300, 1024), (40, 4100, 4224)])
def test_streams_and_graphs(m, n, k):
    x, w = problem(m, n, k, 128, True, BF, seed=11)
    want = mk.w4_gemm(x, w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mk.w4_gemm(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mk.w4_gemm(x, w))
        graphs.append(g)
    for _ in range(3):
        graphs[1].replay()
        with torch.cuda.stream(side):
            graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_a_wait_that_runs_out_is_reported():
    """One CTA stops loading: its waits end, the call returns, and the next one serves."""
    x, w = problem(48, 4100, 4096, 128, True, BF, seed=12)
    want = mk.w4_gemm(x, w)
    ws = mk.Workspace()
    mk.w4_gemm(x, w, cfg=mk.Config(wait_limit_ns=20_000_000, inject=1), workspace=ws)
    assert mk.device_status(ws)[0] == mk.MK_ERR_TIMEOUT
    assert torch.equal(mk.w4_gemm(x, w, workspace=ws), want) and mk.device_status(ws)[0] == mk.MK_OK


@pytest.mark.parametrize("ctas", [1, 3, 7, 64])
def test_any_number_of_ctas(ctas):
    """Runs that hold many tiles, one, or a part: the joins differ, the sums' tolerance does not."""
    for m, n, k, group in ((50, 2060, 8320, 128), (40, 4100, 4160, 64), (8192, 300, 96, 32), (600, 1000, 1152, 128)):
        x, w = problem(m, n, k, group, True, HF, seed=13)
        check(x, w, F32, cfg=mk.Config(max_ctas=ctas))


def test_a_gradient_is_refused():
    x, w = problem(2, 32, 64, 32, False, BF)
    x.requires_grad_()
    with pytest.raises(ValueError):
        mk.w4_gemm(x, w)
    with torch.no_grad():
        assert not mk.w4_gemm(x, w).requires_grad
