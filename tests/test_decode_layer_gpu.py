"""Norm, 4-bit products, attention, router and experts together (GPU): the decode example end to end, a training step through
autograd, and the 8-bit norm into AllGather + GEMM.

The bound on max |error| / rms(stream) of the example.  With u = 2^-8 the relative half step of bf16: the stream is
rounded at its three additions (u each), the branches carry the normalised input, q, k, v, the rotated ones, the
attention's weights and output, the projection (8 u), and the normalised input, the expert's rows twice, the returned
rows, their sum (5 u); a branch is no larger than the stream, and the largest of 1e5 values is at most 6 rms:
6 * 16 * 2^-8 < 0.38 if every rounding went the same way."""
import importlib.util
import os

import pytest
import torch

import comm_gemm_tile_gb300 as mk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from comm_gemm_tile_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("symmetric,group", [(True, 64), (False, 128), (True, 32)])
def test_prompts_then_steps(example, symmetric, group):
    error, load, _ = example.run(symmetric=symmetric, group=group)
    assert error <= 0.38, error
    assert int(load.sum()) == 2 * (60 + 33 + 1 + 8 * 3)


def test_a_training_step(example):
    """x -> rms_norm -> logits -> moe_route -> a loss of the gates and both losses, and of the stream: gradients of x, the
    residual and both weights against the same in 64 bits.  fp32 throughout: every step's relative error is below
    2^-16 (sums of 256 terms, in products that torch may round to 2^-24 each), so the gradients' are below 2^-12 of their largest."""
    g = torch.Generator().manual_seed(3)
    T, H, E, K = 200, 256, 16, 2
    x, r = (torch.randn(T, H, generator=g).cuda() for _ in range(2))
    w, wr = (1 + 0.1 * torch.randn(H, generator=g)).cuda(), (torch.randn(E, H, generator=g) * H ** -0.5).cuda()
    dg, dh = torch.randn(T, K, generator=g).cuda(), torch.randn(T, H, generator=g).cuda()
    mine = [t.clone().requires_grad_() for t in (x, r, w, wr)]
    n, h = mk.rms_norm(mine[0], mine[2], residual=mine[1], eps=1e-5)
    route = mk.moe_route(n @ mine[3].t(), K, scale=2.0)
    ((route["gates"] * dg).sum() + 0.5 * route["balance_loss"] + 0.1 * route["z_loss"] + (h * dh).sum()).backward()

    want = [t.double().requires_grad_() for t in (x, r, w, wr)]
    hh = want[0] + want[1]
    nn = hh * (hh.square().mean(dim=-1, keepdim=True) + 1e-5).rsqrt() * want[2]
    z = nn @ want[3].t()
    idx = route["topk_idx"].long()
    gates = torch.softmax(z.gather(1, idx), dim=-1) * 2.0
    f = torch.bincount(idx.flatten(), minlength=E).double() / (K * T)
    loss = (gates * dg).sum() + 0.5 * E * (f * z.softmax(dim=-1).mean(dim=0)).sum() + 0.1 * z.logsumexp(dim=-1).square().mean()
    (loss + (hh * dh).sum()).backward()
    for a, b in zip(mine, want):
        assert float((a.grad.double() - b.grad).abs().max()) <= 2.0 ** -12 * float(b.grad.abs().max())


def test_a_captured_training_step(example):
    """The gradient calls in a graph, while an eager graph of the same leaf lives."""
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn(96, 512, generator=g).bfloat16().cuda(), torch.ones(512, device="cuda")
    dg = torch.randn(96, 2, generator=g).cuda()
    leaf = x.clone().requires_grad_()
    alive = mk.rms_norm(leaf, w).float().sum()             # not yet run backward

    def step():
        n = mk.rms_norm(x, w)
        route = mk.moe_route(n[:, :32], 2)
        dl = mk.moe_route_backward(n[:, :32], route, dg)
        dn = torch.zeros_like(n)
        dn[:, :32] = dl
        return mk.rms_norm_backward(dn, x, w)

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        graph.replay()
    alive.backward()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and leaf.grad is not None


def test_the_8_bit_norm_feeds_all_gather(example):
    """rms_norm into e4m3, gathered and multiplied, rows times their scales: what the codes stand for, times B, exactly but
    for sums in fp32 (512 terms: 2^-14) and one rounding to bf16."""
    g = torch.Generator().manual_seed(5)
    R, m, k, n = 2, 128, 512, 256
    x, r = ([torch.randn(m, k, generator=g).bfloat16().cuda() for _ in range(R)] for _ in range(2))
    w = (1 + 0.1 * torch.randn(k, generator=g)).bfloat16().cuda()
    b = torch.randn(n, k, generator=g).cuda().to(mk.FP8)
    made = [mk.rms_norm(a, w, residual=c, out_dtype=mk.FP8) for a, c in zip(x, r)]
    _, c = mk.ag_gemm([t[0] for t in made], b, out_dtype=torch.float32)
    y = c * torch.cat([t[1] for t in made])[:, None]
    a = torch.cat([t[0].double() * t[1].double()[:, None] for t in made])
    want, size = a @ b.double().t(), a.abs() @ b.double().abs().t()
    assert bool(((y.double() - want).abs() <= 2.0 ** -14 * size).all())
