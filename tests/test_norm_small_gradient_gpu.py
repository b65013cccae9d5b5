"""The norm's gradient of small rows for small gradients, whose products with each other are below fp32's range (GPU).

Tolerances of test_norm_gpu, and what g = dy w is off where it is below 2^-126 itself: 2^-150, half of fp32's spacing there, in
dx = r (g - u mean(g u)) r 2^-150 (1 + |u| mean |u|), and as much again for g u."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_norm_gpu import BF, F32, SUM, between, draw, formula, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def gradient_check(h, w, dy, dh=None, eps=1e-6):
    dx, dw = mk.rms_norm_backward(dy, h, w, dh=dh, eps=eps)
    _, u, r = formula(h, w, eps)
    g = dy.double() if w is None else dy.double() * w.double()
    want = r * (g - u * (g * u).mean(dim=-1, keepdim=True))
    size = r * (g.abs() + u.abs() * (g * u).abs().mean(dim=-1, keepdim=True))
    low = 2 * r * 2.0 ** -150 * (1 + u.abs() * u.abs().mean(dim=-1, keepdim=True))
    if dh is not None:
        want, size = want + dh.double(), size + dh.double().abs()
    assert bool(((dx.double() - want).abs() <= half_step(want, h.dtype) + 2 * SUM * size + low).all())
    if w is not None:
        t = dy.double() * u
        assert bool(((dw.double() - t.sum(dim=0)).abs() <= half_step(t.sum(dim=0), w.dtype)
                     + (SUM + 64 * 2.0 ** -24) * t.abs().sum(dim=0) + len(t) * 2.0 ** -149).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [96, 1001, 5000, 16384])
@pytest.mark.parametrize("size,eps", [(1e-14, 1e-28), (1e-10, 1e-22), (1e-7, 1e-13), (1e-18, 1e-37)])
def test_small_rows(size, eps, n, dtype):
    h, dy = (draw((20, n), F32, 1) * size).to(dtype), (draw((20, n), F32, 2) * (1e-44 / size)).to(dtype)
    h[3] = 0
    h[5] *= 2.0 ** 40
    w = draw((n,), F32, 3)
    gradient_check(h, w, dy, eps=eps)
    gradient_check(h, None, dy, dh=(draw((20, n), F32, 4) * float(dy.float().abs().max()) / size).to(dtype), eps=eps)


@pytest.mark.parametrize("gap", [1, 3])
def test_small_rows_by_elements(gap):
    h = between(30, 130, gap, 0, F32, 0.0)[0].copy_(draw((30, 130), F32, 5) * 1e-14)
    dy = draw((30, 130), F32, 6) * 1e-30
    gradient_check(h, draw((130,), F32, 7), dy, eps=1e-28)
