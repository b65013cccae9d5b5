"""moe_route and its gradient against the formula in 64 bits, and against what the dispatch chooses (GPU).

Tolerances.  exp(l - top) is off by |l - top| 2^-24 (the difference's rounding) and about 2 steps, a sum of 256 terms by 13
roundings: with D the largest |l - top|, a probability is off by REL(D) = (2 D + 40) 2^-24 of itself; logsumexp by
(|top| + 40) 2^-24."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def draw(shape, dtype, seed, size=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * size).to(dtype).cuda()


def formula(logits, topk, normalize=True, scale=1.0, mask=None):
    """The route in 64 bits; tokens that count nowhere have real = False."""
    z = logits.detach().double()
    T, E = z.shape
    # (stable: equal logits keep their order; -0 and +0 are equal)
    value, idx = torch.sort(z, dim=-1, descending=True, stable=True)
    value, idx = value[:, :topk], idx[:, :topk]
    real = value[:, 0] > -INF if mask is None else (value[:, 0] > -INF) & mask
    slot = (value > -INF) & real[:, None]
    safe = torch.where(real[:, None], z, 0.0)
    p = torch.softmax(safe, dim=-1)
    lse = torch.logsumexp(safe, dim=-1)
    w = torch.where(slot, p.gather(1, idx), 0.0)
    share = w / w.sum(dim=-1, keepdim=True).clamp_min(1e-300) if normalize else w
    counts = torch.bincount(idx[slot], minlength=E)
    N = int(real.sum())
    f = counts.double() / max(1, topk * N)
    mean = p[real].sum(dim=0) / max(1, N)
    return dict(idx=torch.where(slot, idx, -1), gates=share * scale, counts=counts, tokens=N, real=real, slot=slot, p=p,
                lse=lse, f=f, share=share, balance=float(E * (f * mean).sum()), z=float(lse[real].square().sum() / max(1, N)))


def rel(logits):
    z = logits.detach().double()
    z = torch.where(z.isfinite(), z, z.new_full((), 0.0))
    return (2 * float(z.max() - z.min()) + 40) * 2.0 ** -24 if z.numel() else 0.0


def check(logits, topk, **how):
    got, want = mk.moe_route(logits, topk, **how), formula(logits, topk, **how)
    R, T = rel(logits), max(1, logits.shape[0])
    assert torch.equal(got["topk_idx"].long(), want["idx"])
    assert torch.equal(got["counts"].long(), want["counts"]) and int(got["tokens"]) == want["tokens"]
    assert bool(((got["gates"].double() - want["gates"]).abs() <= 2 * R * want["gates"].abs() + 1e-37).all())
    # the means over tokens: at most T / 2432 of a warp in order, then 8 warps, 304 blocks
    S = (T / 2432 + 400) * 2.0 ** -24
    assert abs(float(got["balance_loss"]) - want["balance"]) <= (R + S) * want["balance"]
    top = float(want["lse"][want["real"]].abs().max()) if want["tokens"] else 0.0
    if want["z"] > torch.finfo(F32).max:                   # (logits of -3.4e38: their square, 1.2e77, has no fp32 number)
        assert float(got["z_loss"]) == INF
        return got, want
    assert abs(float(got["z_loss"]) - want["z"]) <= 2 * top * (top + rel(logits) * 2 ** 24) * 2.0 ** -24 + S * want["z"]
    return got, want


SIZES = [(1, 1, 1), (1, 2, 2), (3, 5, 3), (16, 64, 2), (64, 60, 6), (65, 33, 8), (300, 64, 2), (1000, 128, 4), (777, 200, 7),
         (5000, 256, 8), (257, 8, 8), (9, 255, 1)]


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_route(T, E, K, dtype):
    logits = draw((T, E), dtype, 1)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(2)).cuda() < 0.8
    for normalize, scale in ((True, 1.0), (False, 2.5)):
        check(logits, K, normalize=normalize, scale=scale)
        check(logits, K, normalize=normalize, scale=scale, mask=mask)


def test_ties_and_zeros():
    logits = torch.zeros(70, 40, device="cuda")
    logits[1::2] = -0.0
    logits[5, 7], logits[5, 30] = 1.0, 1.0
    got, _ = check(logits, 3)
    assert got["topk_idx"][0].tolist() == [0, 1, 2] and got["topk_idx"][5].tolist() == [7, 30, 0]
    mixed = torch.where(torch.arange(40, device="cuda") % 2 == 0, -0.0, 0.0).expand(70, 40).contiguous()
    assert mk.moe_route(mixed, 4)["topk_idx"][9].tolist() == [0, 1, 2, 3]


def test_rows_that_masks_leave_nothing():
    logits = draw((200, 48), F32, 3)
    logits[::3] = -INF                                     # no expert
    logits[1::3, 2:] = -INF                                # two of the four slots
    logits[2::3, 17] = -INF
    got, want = check(logits, 4)
    assert want["tokens"] == 133 and got["topk_idx"][0].tolist() == [-1] * 4 and got["gates"][0].abs().sum() == 0
    assert got["topk_idx"][1, 2:].tolist() == [-1, -1] and not bool((got["topk_idx"] == 17)[2::3].any())
    lowest = torch.full((3, 8), torch.finfo(F32).min, device="cuda")     # a mask of the type's lowest value is a logit
    check(lowest, 2)
    nothing = torch.zeros(200, dtype=torch.bool, device="cuda")
    for T in (200, 20, 0):
        got, _ = check(logits[:T], 4, mask=nothing[:T])
        assert float(got["balance_loss"]) == 0 == float(got["z_loss"]) and int(got["counts"].sum()) == 0


def test_far_logits():
    logits = draw((130, 64), F32, 4, 30.0) + 5e4
    check(logits, 4)
    check(draw((130, 64), F32, 5, 200.0), 4, normalize=False)


def test_nan_stays_with_its_token():
    logits = draw((100, 32), F32, 6)
    logits[10, 3] = float("nan")
    got = mk.moe_route(logits, 2)
    clean = mk.moe_route(torch.where(torch.arange(100, device="cuda")[:, None] == 10, 0.0, logits), 2)
    rest = torch.arange(100, device="cuda") != 10
    assert torch.equal(got["gates"][rest], clean["gates"][rest]) and bool(got["gates"][10].isnan().all())
    assert bool(got["balance_loss"].isnan()) and bool(got["z_loss"].isnan())


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("experts", [24, 200])
@pytest.mark.parametrize("topk", [1, 2, 3, 8])
def test_where_nan_stands(topk, experts, dtype):
    """NaN is above every logit and NaN with a sign below every one, as the dispatch has it: ids as integers would order them."""
    logits = draw((40, experts), dtype, 61)
    logits[3, 5] = float("nan")
    logits[4, 7] = logits[4, 2] = logits[4, 19] = float("nan")
    logits[5, 1] = -logits[3, 5]
    logits[6] = -logits[3, 5]
    logits[7] = float("nan")
    logits[8, :20] = -INF
    logits[8, 1] = float("nan")
    got = mk.moe_route(logits, topk)
    key = logits.float().view(torch.int32).long()
    key = torch.where(key < 0, -(key & 0x7fffffff), key)
    value, idx = torch.sort(key, dim=-1, descending=True, stable=True)
    want = torch.where(value[:, :topk] > -0x7f800000, idx[:, :topk], -1)
    assert torch.equal(got["topk_idx"].long(), want)          # (16-bit types lose NaN's sign when it is negated)
    assert int(got["tokens"]) == int((want[:, 0] >= 0).sum()) and torch.equal(got["counts"].long(), torch.bincount(want[want >= 0], minlength=experts))
    for t in (0, 20, 39):
        clean = mk.moe_route(logits[t:t + 1], topk)
        assert torch.equal(got["gates"][t:t + 1], clean["gates"])


def test_strides():
    big = draw((150, 100), BF, 7)
    for logits in (big[:, 3:67], big[::2, :64], big[:1].expand(90, 100)[:, :50]):
        check(logits, 4)
        got = mk.moe_route(logits, 4)
        dl = mk.moe_route_backward(logits, got, torch.ones(logits.shape[0], 4, device="cuda"), normalize=False)
        room = torch.full((logits.shape[0], 128), 9.0, dtype=BF, device="cuda")
        mk.moe_route_backward(logits, mk.moe_route(logits, 4), torch.ones(logits.shape[0], 4, device="cuda"),
                              normalize=False, out=room[:, 5:5 + logits.shape[1]])
        assert torch.equal(room[:, 5:5 + logits.shape[1]], dl)
        assert bool((room[:, :5] == 9).all()) and bool((room[:, 5 + logits.shape[1]:] == 9).all())


def test_rows_far_apart():
    big = torch.empty(3, (1 << 29) + 32, device="cuda")
    logits = big[:, :32]
    logits.copy_(draw((3, 32), F32, 40))
    got, _ = check(logits, 3)
    dg = draw((3, 3), F32, 41)
    dl = mk.moe_route_backward(logits, got, dg, out=big[:, 1 << 29:])
    assert torch.equal(dl, mk.moe_route_backward(logits.contiguous(), got, dg))


def test_equal_logits_of_many_experts():
    """More equal logits than a warp has lanes, of 16-bit types too: rounds instead of lists, the same choice."""
    for dtype in (F32, BF):
        for E in (64, 130, 256):
            logits = draw((90, E), F32, 42).round().to(dtype)
            logits[::4] = 2.0
            check(logits, 8)
            gradient_check(logits, 8, normalize=False)


def test_the_dispatch_chooses_the_same():
    R, T, E, K, H, N = 2, 300, 16, 4, 64, 64
    logits = draw((R * T, E), F32, 8).bfloat16().float()     # ties
    x = [draw((T, H), BF, 9 + r) for r in range(R)]
    w = [draw((E // R, H, N), BF, 20 + r) for r in range(R)]
    d = mk.moe_dispatch_gemm(x, list(logits.view(R, T, E)), w, E_loc=E // R, topk=K)
    route = mk.moe_route(logits, K)
    assert torch.equal(route["topk_idx"], d["topk_idx"]) and torch.equal(route["counts"], d["counts"].sum(dim=0).int())
    parts = [mk.moe_route(logits[r * T:(r + 1) * T], K)["counts"] for r in range(R)]
    assert torch.equal(torch.stack(parts), d["counts"])


# ------------------------------------------------------------------ gradient

def gradient(logits, route, dg, db, dz, normalize, scale):
    """(dlogits, the sum of the sizes of its terms) in 64 bits."""
    p, f, share, slot = route["p"], route["f"], route["share"], route["slot"]
    T, E = p.shape
    N = max(1, route["tokens"])
    d, size = torch.zeros_like(p), torch.zeros_like(p)
    if dg is not None:
        v = torch.where(slot, dg.double() * scale, 0.0)
        at = route["idx"].clamp_min(0)
        dot, absdot = (share * v).sum(dim=-1, keepdim=True), (share * v).abs().sum(dim=-1, keepdim=True)
        if normalize:
            d.scatter_add_(1, at, share * (v - dot) * slot)
            size.scatter_add_(1, at, share * (v.abs() + absdot) * slot)
        else:
            d.scatter_add_(1, at, share * v)
            size.scatter_add_(1, at, share * v.abs())
            d -= p * dot
            size += p * absdot
    if db is not None:
        pf = (p * f).sum(dim=-1, keepdim=True)
        d += float(db) * E / N * p * (f - pf)
        size += abs(float(db)) * E / N * p * (f + pf)
    if dz is not None:
        t = float(dz) * 2 / N * route["lse"][:, None] * p
        d += t
        size += t.abs()
    return d * route["real"][:, None], size * route["real"][:, None]


def gradient_check(logits, topk, mask=None, normalize=True, scale=1.0, parts=(1, 1, 1)):
    how = dict(normalize=normalize, scale=scale)
    got = mk.moe_route(logits, topk, mask=mask, **how)
    want = formula(logits, topk, mask=mask, **how)
    T = logits.shape[0]
    dg = draw((T, topk), F32, 50, 1.0) if parts[0] else None
    db = torch.tensor(0.7, device="cuda") if parts[1] else None
    dz = torch.tensor(-0.3, device="cuda") if parts[2] else None
    dl = mk.moe_route_backward(logits, got, dg, db, dz, **how)
    d, size = gradient(logits, want, dg, db, dz, normalize, scale)
    f = torch.finfo(logits.dtype)
    tol = d.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2 + 4 * rel(logits) * size
    assert dl.dtype == logits.dtype and bool(((dl.double() - d).abs() <= tol).all())
    assert bool((dl[~want["real"]] == 0).all())
    return dl


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("T,E,K", SIZES)
def test_gradient(T, E, K, dtype):
    logits = draw((T, E), dtype, 30)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(31)).cuda() < 0.8
    gradient_check(logits, K, normalize=True, scale=2.0)
    gradient_check(logits, K, normalize=False, scale=2.5, mask=mask)
    for parts in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 0, 0)):
        gradient_check(logits, K, normalize=False, mask=mask, parts=parts)
        gradient_check(logits, K, normalize=True, parts=parts)


def test_gradient_of_masked_experts():
    logits = draw((200, 48), F32, 32)
    logits[::3] = -INF
    logits[1::3, 2:] = -INF
    for normalize in (True, False):
        dl = gradient_check(logits, 4, normalize=normalize)
        assert bool((dl[logits == -INF] == 0).all())


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(normalize):
    """Central differences of the kernel's gates and losses: off by what the same differences of the 64-bit formula are,
    and by the outputs' roundings over the step."""
    T, E, K, step = 6, 12, 3, 2.0 ** -6
    logits = draw((T, E), F32, 33)
    dg = draw((T, K), F32, 34, 1.0)
    how = dict(normalize=normalize, scale=1.5)

    def loss(z, exact):
        if exact:
            w = formula(z, K, **how)
            return float((w["gates"] * dg.double()).sum()) + 0.7 * w["balance"] - 0.3 * w["z"]
        r = mk.moe_route(z, K, **how)
        return float((r["gates"].double() * dg.double()).sum()) + 0.7 * float(r["balance_loss"]) - 0.3 * float(r["z_loss"])

    route = mk.moe_route(logits, K, **how)
    dl = mk.moe_route_backward(logits, route, dg, torch.tensor(0.7, device="cuda"), torch.tensor(-0.3, device="cuda"), **how)
    base = formula(logits, K, **how)
    exact, size = gradient(logits, base, dg, 0.7, -0.3, normalize, 1.5)
    slack = (2 * rel(logits) * (float((base["gates"] * dg.double()).abs().sum()) + base["balance"] + 2 * base["z"])
             + 500 * 2.0 ** -24 * (base["balance"] + base["z"])) / step
    used = 0
    for t in range(T):
        for e in range(0, E, 2):
            up, down = logits.clone(), logits.clone()
            up[t, e] += step
            down[t, e] -= step
            if not all(torch.equal(mk.moe_route(z, K)["topk_idx"], route["topk_idx"]) for z in (up, down)):
                continue                                   # the choice changes there: no derivative
            used += 1
            d = [(loss(up, w) - loss(down, w)) / float(up[t, e].double() - down[t, e].double()) for w in (0, 1)]
            assert abs(d[0] - float(dl[t, e])) <= slack + abs(d[1] - float(exact[t, e])) + 4 * rel(logits) * float(size[t, e])
    assert used > 20


def test_autograd():
    logits, dg = draw((300, 64), F32, 35), draw((300, 2), F32, 36, 1.0)
    mask = torch.arange(300, device="cuda") < 280
    leaf = logits.clone().requires_grad_()
    r = mk.moe_route(leaf, 2, mask=mask, scale=2.0)
    plain = mk.moe_route(logits, 2, mask=mask, scale=2.0)
    assert all(torch.equal(r[name], plain[name]) for name in plain)
    assert r["gates"].requires_grad and not r["topk_idx"].requires_grad and not r["counts"].requires_grad
    ((r["gates"] * dg).sum() + 0.01 * r["balance_loss"] + 0.001 * r["z_loss"]).backward()
    want = mk.moe_route_backward(logits, plain, dg, torch.tensor(0.01, device="cuda"), torch.tensor(0.001, device="cuda"), scale=2.0)
    assert torch.equal(leaf.grad, want)
    leaf = logits.bfloat16().requires_grad_()              # one output used; its gradient is expanded
    mk.moe_route(leaf, 2, normalize=False)["gates"].sum().backward()
    plain = mk.moe_route(leaf.detach(), 2, normalize=False)
    assert torch.equal(leaf.grad, mk.moe_route_backward(leaf.detach(), plain, torch.ones(300, 2, device="cuda"), normalize=False))
    leaf = logits.clone().requires_grad_()
    mk.moe_route(leaf, 2)["z_loss"].backward()
    assert torch.equal(leaf.grad, mk.moe_route_backward(logits, mk.moe_route(logits, 2), dz=torch.ones((), device="cuda")))
    with pytest.raises(ValueError):
        mk.moe_route(leaf, 2, out={"gates": torch.empty(300, 2, device="cuda")})
    with torch.no_grad():
        assert not mk.moe_route(leaf, 2)["gates"].requires_grad


def test_given_outputs_streams_graphs_and_the_same_bits():
    logits = draw((3000, 96), F32, 37)
    want = mk.moe_route(logits, 4)
    given = {name: torch.empty_like(t) for name, t in want.items()}
    got = mk.moe_route(logits, 4, out=given)
    assert all(got[n] is given[n] and torch.equal(got[n], want[n]) for n in want)
    side, ws = torch.cuda.Stream(), mk.Workspace()
    torch.cuda.synchronize()
    got = mk.moe_route(logits, 4, stream=side, workspace=ws)
    dg = torch.ones(3000, 4, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    dl = mk.moe_route_backward(logits, got, dg, got["balance_loss"], normalize=False, stream=side)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    want_dl = mk.moe_route_backward(logits, want, dg, want["balance_loss"], normalize=False)
    assert torch.equal(dl, want_dl)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = mk.moe_route(logits, 4)
            outs.append((r, mk.moe_route_backward(logits, r, dg, r["balance_loss"], normalize=False)))
        graphs.append(g)
    for _ in range(3):
        graphs[1].replay()
        with torch.cuda.stream(side):
            graphs[0].replay()
    torch.cuda.synchronize()
    for r, dl in outs:
        assert all(torch.equal(r[n], want[n]) for n in want) and torch.equal(dl, want_dl)
