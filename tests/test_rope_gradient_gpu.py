"""rope under autograd: the gradient of the rotation reaches the input (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P

pytestmark = pytest.mark.gpu
HOWS = [dict(), dict(interleaved=True, magnitude=1.25), dict(inverse=True, magnitude=0.5), dict(start=1000)]


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def _inputs(dtype, shape=(17, 3, 64)):
    g = torch.Generator().manual_seed(5)
    x, dy = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
    return x, dy, mk.rope_freqs(32)[0]


@pytest.mark.parametrize("how", HOWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_backward_is_the_inverse_rotation(dtype, how):
    x, dy, freqs = _inputs(dtype)
    want = mk.rope(x, freqs, **how)
    leaf = x.clone().requires_grad_()
    y = mk.rope(leaf, freqs, **how)
    assert y.requires_grad and torch.equal(y, want)
    y.backward(dy)
    assert torch.equal(leaf.grad, mk.rope(dy, freqs, **{**how, "inverse": not how.get("inverse", False)}))
    assert not mk.rope(leaf.detach(), freqs, **how).requires_grad
    with torch.no_grad():
        assert not mk.rope(leaf, freqs, **how).requires_grad


def test_gradient_against_the_formula_and_differences():
    """loss = sum dy rope(x): linear in x, so a difference of any length is exact but for the rounding of the two outputs
    (bounded by rotate_tolerance at each point)."""
    x, dy, freqs = _inputs(torch.float32, (5, 2, 64))
    pos = torch.tensor([0, 3, 1 << 19, 7, 100], device="cuda")
    leaf = x.clone().requires_grad_()
    mk.rope(leaf, freqs, pos).backward(dy)
    want, tol = P.rotate_tolerance(dy, pos, freqs, torch.float32, inverse=True)
    assert bool(((leaf.grad.double().cpu() - want).abs() <= tol).all())
    for at in ((0, 0, 0), (2, 1, 17), (2, 1, 31), (4, 0, 63)):
        up, down = x.clone(), x.clone()
        up[at] += 4.0
        down[at] -= 4.0
        loss, slack = [], 0.0
        for t in (up, down):
            loss.append(float((mk.rope(t, freqs, pos).double() * dy.double()).sum()))
            _, tol = P.rotate_tolerance(t, pos, freqs, torch.float32)
            slack += float((tol * dy.double().cpu().abs()).sum())
        step = float(up[at].double() - down[at].double())
        assert abs((loss[0] - loss[1]) / step - float(leaf.grad[at])) <= slack / step + float(tol.max())


def test_shared_strided_and_broadcast_inputs():
    base = torch.randn(9, 1, 64, generator=torch.Generator().manual_seed(6)).cuda().requires_grad_()
    freqs, _ = mk.rope_freqs(64)
    y = mk.rope(base.expand(9, 4, 64), freqs) + mk.rope(base.expand(9, 4, 64).transpose(0, 1).contiguous().transpose(0, 1), freqs)
    dy = torch.randn(9, 4, 64, generator=torch.Generator().manual_seed(7)).cuda()
    y.backward(dy)
    one = mk.rope(dy, freqs, inverse=True).double().sum(dim=1, keepdim=True) * 2
    assert torch.allclose(base.grad.double(), one, rtol=0, atol=16 * 2.0 ** -24 * float(one.abs().max()))


@pytest.mark.parametrize("how", HOWS)
def test_gradients_of_any_strides(how):
    """A sum's gradient is expanded, a transposed result's has its last dimension elsewhere."""
    x, dy, freqs = _inputs(torch.float32)
    back = lambda g: mk.rope(g, freqs, **{**how, "inverse": not how.get("inverse", False)})   # noqa: E731
    leaf = x.clone().requires_grad_()
    mk.rope(leaf, freqs, **how).sum().backward()
    assert torch.equal(leaf.grad, back(torch.ones_like(x)))
    leaf = x.clone().requires_grad_()
    mk.rope(leaf, freqs, **how).permute(2, 0, 1).backward(dy.permute(2, 0, 1).contiguous())
    assert torch.equal(leaf.grad, back(dy))


def test_second_derivative():
    x, dy, freqs = _inputs(torch.float32)
    leaf, seed = x.clone().requires_grad_(), dy.clone().requires_grad_()
    dx, = torch.autograd.grad(mk.rope(leaf, freqs), leaf, seed, create_graph=True)
    back, = torch.autograd.grad(dx, seed, x)
    assert torch.equal(back, mk.rope(x, freqs))


def test_an_output_of_ones_own_takes_no_gradient():
    x, _, freqs = _inputs(torch.float32)
    leaf = x.clone().requires_grad_()
    with pytest.raises(ValueError):
        mk.rope(leaf, freqs, out=torch.empty_like(x))
    with torch.no_grad():
        mk.rope(leaf, freqs, out=leaf)
    assert torch.equal(leaf.detach(), mk.rope(x, freqs))


def test_on_a_given_stream():
    x, dy, freqs = _inputs(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    leaf = x.clone().requires_grad_()
    torch.cuda.synchronize()
    y = mk.rope(leaf, freqs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    y.backward(dy)
    torch.cuda.synchronize()
    assert torch.equal(y, mk.rope(x, freqs)) and torch.equal(leaf.grad, mk.rope(dy, freqs, inverse=True))
