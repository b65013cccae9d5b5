"""The codes of rms_norm's 8-bit rows are y / scale to the nearest (GPU).

The fp32 output of the same rows is the y that the codes are of, bit for bit, and an fp32 division rounds once: so they are equal,
not near.  The rows hold values of 8 significant bits, of which two in a hundred thousand quotients lie within a rounding of the
middle of two codes."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk

pytestmark = pytest.mark.gpu
F32, E4 = torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def draw(shape, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).bfloat16().float().cuda()


def codes(y, scale):
    """e4m3 codes of y / scale, whose infinities saturate."""
    return (y / scale[..., None]).clamp(-448, 448).to(E4)


# whole pieces, rows that begin inside of pieces, single elements (where a residual's strides differ from x's); few rows and many
@pytest.mark.parametrize("rows,n,gap", [(400, 4096, 0), (3, 16384, 0), (8192, 129, 0), (900, 1001, 0), (500, 2050, 1)])
def test_codes_are_of_the_quotient(rows, n, gap):
    x, w = draw((rows, n + gap), 1, 2.0)[:, :n], draw((n,), 2)
    zero = torch.zeros(rows, n, device="cuda") if gap else None          # (its rows begin elsewhere than x's)
    y, c, scale = mk.rms_norm(x, w, residual=zero), *mk.rms_norm(x, w, residual=zero, out_dtype=E4)[:2]
    y = y[0] if gap else y
    assert torch.equal(scale, (y.abs().amax(dim=-1) / torch.full((), 448.0, device="cuda")).clamp_min(2.0 ** -100))
    assert torch.equal(c.view(torch.uint8), codes(y, scale).view(torch.uint8))


def test_tiny_and_huge_rows():
    """Rows whose scale is at its least, rows past 2^100, and weights that are infinite or not numbers."""
    x, w = draw((64, 512), 3), draw((512,), 4)
    x[:, 100:110], x[:, 110:120], x[5] = 0.0, -0.0, -0.0      # codes of -0 keep the sign
    for size in (2.0 ** -118, 2.0 ** -100, 2.0 ** -60, 2.0 ** 100):
        y = mk.rms_norm(x, w * size)
        c, scale = mk.rms_norm(x, w * size, out_dtype=E4)
        assert torch.equal(c.view(torch.uint8), codes(y, scale).view(torch.uint8))
    w[7], w[8], w[9] = float("inf"), -float("inf"), float("nan")
    c, scale = (t.float() for t in mk.rms_norm(x, w, out_dtype=E4))
    some = x[:, 7] != 0                                      # (0 times an infinity is not a number)
    assert torch.equal(c[some, 7], 448 * x[some, 7].sign()) and torch.equal(c[some, 8], -448 * x[some, 8].sign())
    assert bool(c[:, 9].isnan().all()) and bool(c[~some, 7:9].isnan().all())
    keep = torch.arange(512, device="cuda") > 9
    y = mk.rms_norm(x, w.nan_to_num(1.0, 1.0, 1.0))
    assert torch.equal(c[:, keep], codes(y, scale)[:, keep].float())
