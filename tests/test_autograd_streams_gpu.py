"""rms_norm, moe_route and rope under autograd on a given stream: backward runs on the stream that was current in forward, and
the memory of what forward saved must not be used again before that stream has read it (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def draw(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def late_backward(make, side, like):
    """Backward of make(side)'s result, held up on the current stream while the side stream fills all memory of the shapes
    of `like` that it gets."""
    torch.cuda.synchronize()
    out, grads = make(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    torch.autograd.backward(out, grads)
    del out
    with torch.cuda.stream(side):
        for _ in range(4):
            junk = [torch.full_like(t, 1) for t in like]
            junk += [torch.full_like(t, 1) for t in like]
    torch.cuda.synchronize()
    return junk


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm(dtype):
    x, r, dy, dh = (draw((700, 1024), dtype, i) for i in range(4))
    w = draw((1024,), F32, 4)
    h = mk.rms_norm(x, w, residual=r)[1]
    dx, dw = mk.rms_norm_backward(dy, h, w, dh=dh)
    for _ in range(3):
        leaves = [t.clone().requires_grad_() for t in (x, w, r)]
        late_backward(lambda s: (mk.rms_norm(leaves[0], leaves[1], residual=leaves[2], stream=s), (dy, dh)),
                      torch.cuda.Stream(), (x, x, h))
        for leaf, want in zip(leaves, (dx, dw, dx)):
            assert torch.equal(leaf.grad, want)


def test_norm_of_a_side_streams_input():
    """x itself is of the side stream's pool, and autograd alone keeps it."""
    x, dy, w = draw((700, 1024), F32, 5), draw((700, 1024), F32, 6), draw((1024,), F32, 7).requires_grad_()
    want = mk.rms_norm_backward(dy, x, w.detach())[1]

    def make(side):
        with torch.cuda.stream(side):
            own = x.clone()
        return mk.rms_norm(own, w, stream=side), dy

    late_backward(make, torch.cuda.Stream(), (x, x))
    assert torch.equal(w.grad, want)


@pytest.mark.parametrize("normalize", [True, False])
def test_route(normalize):
    logits, dg = draw((3000, 64), F32, 8), draw((3000, 4), F32, 9)
    one = torch.ones((), device="cuda")
    plain = mk.moe_route(logits, 4, normalize=normalize)
    want = mk.moe_route_backward(logits, plain, dg, one, one, normalize=normalize)
    for _ in range(3):
        leaf = logits.clone().requires_grad_()

        def make(side):
            got = mk.moe_route(leaf, 4, normalize=normalize, stream=side)
            return [got[n] for n in ("gates", "balance_loss", "z_loss")], [dg, one, one]

        late_backward(make, torch.cuda.Stream(), tuple(plain.values()))
        assert torch.equal(leaf.grad, want)


def test_rope_of_a_side_streams_frequencies():
    """rope saves only the caller's tensors; those may be of the side stream's pool too."""
    x, dy = draw((700, 8, 128), F32, 10), draw((700, 8, 128), F32, 11)
    freqs, _ = mk.rope_freqs(128)
    at = torch.arange(700, device="cuda")
    want = mk.rope(dy, freqs, at, inverse=True)
    leaf = x.clone().requires_grad_()

    def make(side):
        with torch.cuda.stream(side):
            own = freqs.clone(), at.clone()
        return mk.rope(leaf, *own, stream=side), dy

    late_backward(make, torch.cuda.Stream(), (freqs, at))
    assert torch.equal(leaf.grad, want)
