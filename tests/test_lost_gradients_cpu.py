"""Gradients and tangents that a call would drop are refused (CPU only: before anything touches a GPU)."""
import pytest
import torch
from torch.autograd import forward_ad

import comm_gemm_tile_gb300 as mk
from bind_util import FakeWorkspace, library, stand_in
from comm_gemm_tile_gb300 import build as mkbuild
from test_layer_calls_cpu import route, t, w4

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture()
def lib(monkeypatch, tmp_path):
    mkbuild.build()
    lib = library(tmp_path, "static int n; int entry(void) { ++n; return 0; } int count(void) { return n; } unsigned long size(void) { return 0; }")
    stand_in(monkeypatch, lib.entry, lib.size)
    yield lib
    monkeypatch.undo()
    mk._bound = None


@pytest.mark.parametrize("which", ["scales", "zeros"])
def test_4_bit_weights_that_require_a_gradient(which, lib):
    parts = dict(scales=t(40, 4), zeros=t(40, 4))
    parts[which].requires_grad = True
    w = w4(**parts)
    call = lambda: mk.w4_gemm(t(3, 256), w, out=t(3, 40), workspace=FakeWorkspace())   # noqa: E731
    with pytest.raises(ValueError, match="gradient"):
        call()
    assert lib.count() == 0
    with torch.no_grad():
        call()
    assert lib.count() == 1


def test_outputs_beside_a_gradient():
    x = torch.randn(4, 64, requires_grad=True)
    for name in ("out", "scale_out", "h_out"):
        with pytest.raises(ValueError, match="given out"):
            mk.rms_norm(x, None, **{name: torch.empty(4)})


def test_tangents(lib):
    x, w = torch.randn(4, 64), torch.randn(64)
    freqs = torch.randn(32, dtype=torch.float64)
    with forward_ad.dual_level():
        d = lambda v: forward_ad.make_dual(v, torch.ones_like(v))   # noqa: E731
        calls = [lambda: mk.rms_norm(d(x), w), lambda: mk.rms_norm(x, d(w)), lambda: mk.rms_norm(x, w, residual=d(x)),
                 lambda: mk.rms_norm_backward(d(x), x, w), lambda: mk.rms_norm_backward(x, d(x), w), lambda: mk.rms_norm_backward(x, x, w, dh=d(x)),
                 lambda: mk.moe_route(d(x), 2), lambda: mk.moe_route_backward(d(x), route(), x), lambda: mk.moe_route_backward(x, route(), d(x)),
                 lambda: mk.moe_route_backward(x, route(), None, d(w)), lambda: mk.rope(d(x[:, None]), freqs), lambda: mk.w4_gemm(d(x), w4())]
        for i, call in enumerate(calls):
            with pytest.raises(ValueError, match="tangent"):
                call()
            assert lib.count() == 0, i
        mk.rms_norm(t(4, 64), t(64), out=t(4, 64))          # inputs without one pass
    assert lib.count() == 1
