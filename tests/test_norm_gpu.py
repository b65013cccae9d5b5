"""rms_norm and its gradient against the formula in 64 bits (GPU).

Tolerances.  A row's sums run over at most 64 elements of a thread, 5 shuffles, 32 warps' values: relative error of a sum of
n <= 16384 positive terms below SUM = 128 * 2^-24, of 1 / sqrt(...) below half of it and a few roundings.  Each output
is rounded once more to its type: half a step, finfo.eps / 2 of the value (below the least normal number: half of
its spacing there)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk

pytestmark = pytest.mark.gpu
BF, HF, F32, E4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
SUM = 128 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def half_step(v, dtype):
    f = torch.finfo(dtype)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def draw(shape, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(dtype).cuda()


def formula(h, w, eps):
    """(y, u, r) in 64 bits."""
    h = h.double()
    r = (h.square().mean(dim=-1, keepdim=True) + eps).rsqrt()
    u = h * r
    return (u if w is None else u * w.double()), u, r


def check(x, w, residual=None, eps=1e-6, e4m3=False, **kw):
    got = mk.rms_norm(x, w, residual=residual, eps=eps, out_dtype=E4 if e4m3 else None, **kw)
    got = got if isinstance(got, tuple) else (got,)
    h = x
    if residual is not None:
        h = (x.float() + residual.float()).to(x.dtype)
        assert torch.equal(got[-1], h)
    y, _, _ = formula(h, w, eps)
    if e4m3:
        scale = torch.maximum(y.abs().amax(dim=-1) / 448, torch.full((), 2.0 ** -100).double().cuda())
        assert got[0].dtype == E4 and got[1].shape == x.shape[:-1]
        assert bool(((got[1].double() - scale).abs() <= 2 * SUM * scale).all())
        v = y / scale[..., None]
        # half a step of e4m3 (3 bits; 2^-9 apart below 2^-6), and what the scale and y are off
        assert bool(((got[0].double() - v).abs() <= torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))
                     + 4 * SUM * v.abs()).all())
    else:
        assert got[0].dtype == x.dtype and got[0].shape == x.shape
        assert bool(((got[0].double() - y).abs() <= half_step(y, x.dtype) + SUM * y.abs()).all())
    return got


# one element, odd, one warp's part, a warp, a block, several pieces a thread; rows that fill one block, some, many
SHAPES = [(1, 1), (3, 7), (5, 8), (33, 64), (2, 100), (700, 128), (17, 1000), (400, 1023), (3, 4096), (310, 4104), (2, 8200),
          (305, 16384), (1, 16383)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("rows,n", SHAPES)
def test_forward(rows, n, dtype):
    x, r = draw((rows, n), dtype, 1), draw((rows, n), dtype, 2, 3.0)
    w = draw((n,), F32, 3)
    check(x, w.to(dtype))
    check(x, w, residual=r)
    check(x, None, eps=0.5)
    check(x, w.to(dtype), residual=r, e4m3=True)
    check(x, w, e4m3=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_heads_and_strides(dtype):
    big = draw((37, 12, 72), dtype, 4)
    w = draw((64,), dtype, 5)
    for x in (big[:, 2:9, :64], big[:, :, 8:].transpose(0, 1), big[::3, ::2, 4:68], big[:, :1, 1:65]):
        check(x, w)
        check(x, w, residual=draw(x.shape, dtype, 6))
        check(x, w, e4m3=True)
        out = torch.full((x.shape[0], x.shape[1], 80), 7.0, dtype=dtype, device="cuda")
        check(x, w, out=out[..., 8:72])
        assert bool((out[..., :8] == 7).all()) and bool((out[..., 72:] == 7).all())
    one = draw((1, 1, 64), dtype, 7)
    check(one.expand(9, 5, 64), w, residual=draw((9, 1, 64), dtype, 8).expand(9, 5, 64))


def test_weights_off_whole_pieces():
    w = draw((513,), BF, 50)[1:]
    x, r, dy = draw((20, 512), BF, 51), draw((20, 512), BF, 52), draw((20, 512), BF, 53)
    check(x, w, residual=r)
    check(x, w, e4m3=True)
    gradient_check(x, w, dy)
    assert torch.allclose(mk.rms_norm(x, w).float(), mk.rms_norm(x, w.clone()).float(), rtol=2.0 ** -7, atol=0)


def between(rows, n, gap, off, dtype, fill):
    """[rows, n] inside of a buffer of `fill`: `gap` elements between rows, the first `off` elements into it; the buffer,
    and where it is not the rows."""
    buf = torch.full((off + rows * (n + gap) + 9,), fill, dtype=dtype, device="cuda")
    view = buf[off:off + rows * (n + gap)].view(rows, n + gap)[:, :n]
    rest = torch.ones(buf.shape, dtype=torch.bool, device="cuda")
    rest[off:off + rows * (n + gap)].view(rows, n + gap)[:, :n] = False
    return view, buf, rest


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("rows,n", [(1, 16), (1, 1001), (7, 17), (9, 31), (40, 129), (310, 130), (700, 1001), (320, 4095),
                                    (5, 8191), (310, 16383)])
@pytest.mark.parametrize("gap,off,apart", [(0, 0, 0), (0, 3, 0), (1, 1, 0), (5, 8, 8), (2, 0, 1), (11, 5, 7)])
def test_rows_that_begin_inside_of_pieces(rows, n, gap, off, apart, dtype):
    """Rows that begin anywhere in 16 bytes, NaN between them, alike in all tensors (apart 0 or 8) and not; what lies
    between the rows of the outputs stays."""
    nan = float("nan")
    x, r, dy = (between(rows, n, gap, off, dtype, nan)[0].copy_(draw((rows, n), dtype, 70 + i)) for i in range(3))
    y, ybuf, yrest = between(rows, n, gap, off + apart, dtype, 7)
    h, hbuf, hrest = between(rows, n, gap, off, dtype, 7)
    c, cbuf, crest = between(rows, n, gap, off, E4, 7)
    w = between(1, n, 0, 1, dtype, nan)[0][0].copy_(draw((n,), dtype, 73))
    check(x, w, residual=r, out=y, h_out=h)
    check(x, w.float(), out=y)
    check(x, w, residual=r, out=c, h_out=h, e4m3=True)
    check(x, None, out=c, e4m3=True)
    got = mk.rms_norm_backward(dy, x, w, dh=r, out=y)
    gradient_check(x, w, dy, dh=r, got=got)
    gradient_check(x, w, dy, got=mk.rms_norm_backward(dy, x, w, out=y))
    stays = torch.full((), 7, dtype=E4, device="cuda").view(torch.uint8)
    assert bool((ybuf[yrest] == 7).all()) and bool((hbuf[hrest] == 7).all())
    assert bool((cbuf.view(torch.uint8)[crest] == stays).all())
    own, stream = dy.clone(), r.clone()                       # in place
    gradient_check(x, w, dy, dh=r, got=mk.rms_norm_backward(own, x, w, dh=r.clone(), out=own))
    assert torch.equal(mk.rms_norm(x.clone(), w, residual=stream, h_out=stream)[1], h) and torch.equal(stream, h)


def test_rows_far_apart():
    """Rows more than 2^31 bytes from each other."""
    big = torch.empty(3, (1 << 30) + 64, dtype=BF, device="cuda")
    x = big[:, :64]
    x.copy_(draw((3, 64), BF, 54))
    w = draw((64,), F32, 55)
    y = check(x, w, out=big[:, 1 << 30:])[0]
    assert torch.equal(y, mk.rms_norm(x.contiguous(), w))
    dx, dw = mk.rms_norm_backward(y, x, w)
    want = mk.rms_norm_backward(y.contiguous(), x.contiguous(), w)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_the_stream_in_place_and_equal_forms():
    x, r, w = draw((50, 512), BF, 9), draw((50, 512), BF, 10), draw((512,), BF, 11)
    y, h = mk.rms_norm(x, w, residual=r)
    assert torch.equal(mk.rms_norm(h, w), y)                  # the norm is of the rounded stream
    stream = r.clone()
    y2, h2 = mk.rms_norm(x, w, residual=stream, h_out=stream)
    assert h2 is stream and torch.equal(stream, h) and torch.equal(y2, y)
    own = x.clone()
    assert mk.rms_norm(own, w, out=own) is own and torch.equal(own, mk.rms_norm(x, w))
    c, s = torch.empty((50, 512), dtype=E4, device="cuda"), torch.empty(50, device="cuda")
    got = mk.rms_norm(x, w, out_dtype=E4, out=c, scale_out=s)
    assert got[0] is c and got[1] is s
    assert torch.equal(c.view(torch.uint8), mk.rms_norm(x, w, out_dtype=E4)[0].view(torch.uint8))


@pytest.mark.parametrize("n", [96, 1001, 5000])
def test_a_row_does_not_depend_on_the_others(n):
    """Rows alone, and among zeros, huge and NaN rows, give the same bits."""
    x, w = draw((40, n), F32, 12), draw((n,), F32, 13)
    x[3] = 0
    x[7] *= 1e30
    x[11, 5] = float("nan")
    x[12] *= 1e-30
    every = mk.rms_norm(x, w)
    for i in (2, 3, 6, 7, 8, 11, 12, 13):
        alone = mk.rms_norm(x[i:i + 1], w)
        if n == 96 or i == 11:                              # (longer rows have more threads when they are few)
            assert torch.equal(every[i:i + 1].view(torch.int32), alone.view(torch.int32))
        else:
            assert torch.allclose(every[i:i + 1], alone, rtol=2 * SUM, atol=0)
    assert bool(every[11].isnan().all()) and not bool(every[torch.arange(40) != 11].isnan().any())
    assert bool((every[3] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [1e-38, 1e-25, 1e-12, 1e15, 1e25, 2e38])
@pytest.mark.parametrize("eps", [1e-5, 1e-37])
def test_far_sizes(dtype, size, eps):
    """Sums of squares past fp32's range, and below it."""
    x = (draw((20, 300), F32, 14).clamp(-1.5, 1.5) * size).to(dtype)
    check(x, draw((300,), F32, 15), eps=eps)
    check(x, None, eps=eps, e4m3=True)


def test_infinities():
    """An infinite element makes its row's others 0 and itself NaN, as the formula does; the other rows are not touched."""
    x = draw((4, 256), BF, 16)
    x[1, 3] = float("inf")
    y = mk.rms_norm(x, None)
    assert bool(y[1, 3].isnan()) and bool((y[1, :3] == 0).all()) and bool(y[[0, 2, 3]].isfinite().all())
    w = torch.ones(256, device="cuda")
    w[9] = float("inf")
    c, s = mk.rms_norm(x[2:3], w, out_dtype=E4)
    assert bool(s.isfinite().all()) and float(c[0, 9].float().abs()) == 448.0     # saturates; the scale is the others'
    zero, s = mk.rms_norm(torch.zeros(2, 64, device="cuda"), None, out_dtype=E4)
    assert bool((zero.float() == 0).all()) and bool((s == 2.0 ** -100).all())


# ------------------------------------------------------------------ gradient

def gradient_check(h, w, dy, dh=None, eps=1e-6, got=None):
    dx, dw = got or mk.rms_norm_backward(dy, h, w, dh=dh, eps=eps)
    _, u, r = formula(h, w, eps)
    g = dy.double() if w is None else dy.double() * w.double()
    want = r * (g - u * (g * u).mean(dim=-1, keepdim=True))
    size = r * (g.abs() + u.abs() * (g * u).abs().mean(dim=-1, keepdim=True))
    if dh is not None:
        want, size = want + dh.double(), size + dh.double().abs()
    assert bool(((dx.double() - want).abs() <= half_step(want, h.dtype) + 2 * SUM * size).all())
    if w is None:
        assert dw is None
        return dx, dw
    t = (dy.double() * u).flatten(0, -2)
    want, rows = t.sum(dim=0), t.shape[0]
    # a column's sum: rows of a block in order, then at most 456 blocks, 8 or (past 64) 32 at a time, then those
    assert bool(((dw.double() - want).abs() <= half_step(want, w.dtype)
                 + (SUM + (rows / 300 + 64) * 2.0 ** -24) * t.abs().sum(dim=0)).all())
    return dx, dw


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("rows,n", SHAPES + [(5000, 64), (2500, 520)])
def test_gradient(rows, n, dtype):
    h, dy, dh = draw((rows, n), dtype, 21, 2.0), draw((rows, n), dtype, 22), draw((rows, n), dtype, 23)
    w = draw((n,), F32, 24)
    gradient_check(h, w, dy)
    gradient_check(h, w.to(dtype), dy, dh=dh)
    gradient_check(h, None, dy, dh=dh, eps=0.3)


def test_gradient_of_strided_heads():
    big = draw((37, 12, 72), HF, 25)
    w = draw((64,), HF, 26)
    for h in (big[:, 2:9, :64], big[:, :, 8:].transpose(0, 1), big[::3, ::2, 3:67]):
        dy = draw(h.shape, HF, 27)
        gradient_check(h, w, dy)
        gradient_check(h, w, dy[:1].expand(h.shape), dh=dy[:, :1].expand(h.shape))
        own = dy.clone()
        dx, _ = mk.rms_norm_backward(own, h, w, out=own)
        assert dx is own and torch.equal(own, mk.rms_norm_backward(dy, h, w)[0])


@pytest.mark.parametrize("size", [1e-30, 1e24])
def test_gradient_at_far_sizes(size):
    h, dy = draw((9, 200), F32, 28) * size, draw((9, 200), F32, 29)
    gradient_check(h, draw((200,), F32, 30), dy, eps=1e-37 if size < 1 else 1e-6)


def test_gradient_of_no_rows():
    for shape in ((0, 64), (0, 3, 64), (3, 0, 64)):
        h = torch.empty(shape, device="cuda")
        w = torch.ones(64, device="cuda")
        dx, dw = mk.rms_norm_backward(h, h, w)
        assert dx.shape == h.shape and bool((dw == 0).all())
        assert mk.rms_norm(h, w).shape == h.shape
        y, s, hh = mk.rms_norm(h, w, residual=h, out_dtype=E4)
        assert s.shape == shape[:-1] and hh.shape == shape


@pytest.mark.parametrize("n", [6, 64])
def test_gradient_against_differences(n):
    """Central differences of the kernel's own forward, sum(dy y) + sum(dh h): off from the kernel's gradient by no more
    than the same differences of the 64-bit formula are, and the roundings of the two outputs over the step."""
    x, dy, dh, w = draw((3, n), F32, 31), draw((3, n), F32, 32), draw((3, n), F32, 33), draw((n,), F32, 34)
    dx, dw = mk.rms_norm_backward(dy, x, w, dh=dh)
    step = 2.0 ** -5

    def loss(xx, ww, exact):
        y = formula(xx, ww, 1e-6)[0] if exact else mk.rms_norm(xx, ww).double()
        return float((dy.double() * y).sum() + (dh.double() * xx.double()).sum())

    y, u, r = formula(x, w, 1e-6)
    slack = 4 * SUM * float((dy.double() * y).abs().sum()) / step
    g = dy.double() * w.double()
    exact = r * (g - u * (g * u).mean(dim=-1, keepdim=True)) + dh.double()
    for at in ((0, 0), (1, n // 2), (2, n - 1)):
        d = [0.0, 0.0]
        for which in (0, 1):
            up, down = x.clone(), x.clone()
            up[at] += step
            down[at] -= step
            d[which] = (loss(up, w, which) - loss(down, w, which)) / float(up[at].double() - down[at].double())
        assert abs(d[0] - float(dx[at])) <= slack + abs(d[1] - float(exact[at])) + 2 * SUM * float(exact.abs().max() + 10)
    for c in (0, n - 1):
        up, down = w.clone(), w.clone()
        up[c] += 1.0
        down[c] -= 1.0                                      # linear in w
        d = (loss(x, up, 0) - loss(x, down, 0)) / float(up[c].double() - down[c].double())
        assert abs(d - float(dw[c])) <= slack


def test_autograd():
    x, r, w = draw((60, 768), BF, 35), draw((60, 768), BF, 36), draw((768,), F32, 37)
    dy, dh = draw((60, 768), BF, 38), draw((60, 768), BF, 39)
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    y, h = mk.rms_norm(leaves[0], leaves[1], residual=leaves[2])
    want_y, want_h = mk.rms_norm(x, w, residual=r)
    assert torch.equal(y, want_y) and torch.equal(h, want_h)
    torch.autograd.backward([y, h], [dy, dh])
    dx, dw = mk.rms_norm_backward(dy, want_h, w, dh=dh)
    for leaf, want in zip(leaves, (dx, dw, dx)):
        assert torch.equal(leaf.grad, want)
    assert leaves[0].grad.data_ptr() != leaves[2].grad.data_ptr()
    # only one of the outputs used; a sum's gradient is expanded; only the weight wants one
    leaf = x.clone().requires_grad_()
    mk.rms_norm(leaf, w, residual=r)[1].sum().backward()
    assert torch.equal(leaf.grad, torch.ones_like(x))
    leaf = x.clone().requires_grad_()
    mk.rms_norm(leaf, w).sum().backward()
    assert torch.equal(leaf.grad, mk.rms_norm_backward(torch.ones_like(x), x, w)[0])
    leaf = w.clone().requires_grad_()
    mk.rms_norm(x, leaf).backward(dy)
    assert torch.equal(leaf.grad, mk.rms_norm_backward(dy, x, w)[1])
    # a shared (expanded) input gets the sum of its gradients
    one = draw((1, 768), F32, 40).requires_grad_()
    mk.rms_norm(one.expand(60, 768), w).backward(dy.float())
    parts = mk.rms_norm_backward(dy.float(), one.detach().expand(60, 768), w)[0].double()
    assert bool(((one.grad.double() - parts.sum(dim=0)).abs() <= 60 * 2.0 ** -24 * parts.abs().sum(dim=0)).all())
    with torch.no_grad():
        assert not mk.rms_norm(leaf[None].expand(3, 768), leaf).requires_grad


def test_autograd_refusals():
    x = draw((4, 64), F32, 41).requires_grad_()
    for kw in (dict(out_dtype=E4), dict(out=torch.empty(4, 64, device="cuda")),
               dict(residual=x, h_out=torch.empty(4, 64, device="cuda"))):
        with pytest.raises(ValueError):
            mk.rms_norm(x, None, **kw)
    dx, = torch.autograd.grad(mk.rms_norm(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):                       # no second derivative, and none is made up
        dx.sum().backward()


def test_the_same_bits_every_time():
    h, dy, w = draw((3000, 384), BF, 42), draw((3000, 384), BF, 43), draw((384,), F32, 44)
    first = mk.rms_norm_backward(dy, h, w)
    for _ in range(3):
        again = mk.rms_norm_backward(dy, h, w)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


class Guarded:
    """A workspace of exactly the bytes that are asked for, with others behind it."""
    def get(self, size, stream=None):
        self.size, self.buffer = size, torch.full((size + 4096 * 1024,), 77, dtype=torch.uint8, device="cuda")
        return self.buffer[:size]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 7, 8, 9, 15, 17, 100, 1000])
@pytest.mark.parametrize("n", [1, 33, 64, 1001, 4096, 9001])
def test_the_workspace_is_no_larger_than_asked(rows, n, dtype):
    """Partial sums stay in it, also where there are fewer rows than places for a row to begin in 16 bytes."""
    h, dy, w = draw((rows, n), dtype, 80), draw((rows, n), dtype, 81), draw((n,), dtype, 82)
    ws = Guarded()
    gradient_check(h, w, dy, got=mk.rms_norm_backward(dy, h, w, workspace=ws))
    assert bool((ws.buffer[ws.size:] == 77).all())


def test_streams_graphs_and_workspaces():
    x, r, w, dy = draw((600, 512), BF, 45), draw((600, 512), BF, 46), draw((512,), BF, 47), draw((600, 512), BF, 48)
    want = mk.rms_norm(x, w, residual=r)
    grads = mk.rms_norm_backward(dy, want[1], w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mk.rms_norm(x, w, residual=r, stream=side)
    got2 = mk.rms_norm_backward(dy, got[1], w, stream=side)
    side.synchronize()
    ws = mk.Workspace()
    got3 = mk.rms_norm_backward(dy, want[1], w, workspace=ws)
    for a, b in zip((*got, *got2, *got3), (*want, *grads, *grads)):
        assert torch.equal(a, b)
    # two graphs, replayed in turn and together on two streams: scratch of their own
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, h = mk.rms_norm(x, w, residual=r)
            outs.append((y, h, *mk.rms_norm_backward(dy, h, w)))
        graphs.append(g)
    for _ in range(3):
        graphs[1].replay()
        with torch.cuda.stream(side):
            graphs[0].replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, (*want, *grads)):
            assert torch.equal(a, b)
