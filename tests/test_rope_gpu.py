"""Rotary positions and the append to a paged cache against plain 64-bit arithmetic (GPU)."""
import math

import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def _ok(ws=None):
    st, detail = mk.device_status(ws)
    assert st == mk.MK_OK, (mk.status_string(st), detail)


def _randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _near(got, want, tol):
    bad = (got.double().cpu() - want).abs() - tol
    assert float(bad.max()) <= 0, float(bad.max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,H,d,rot", [(1, 1, 64, 64), (3, 5, 128, 64), (17, 40, 128, 128), (130, 2, 80, 20),
                                       (5, 3, 6, 2), (2, 2, 130, 130), (300, 7, 512, 512), (9, 4, 64, 0)])
def test_rope_matches_the_formula(T, H, d, rot, dtype, interleaved):
    x = _randn((T, H, d), dtype, 1)
    freqs, _ = mk.rope_freqs(rot)
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(2)).cuda()
    for inverse in (False, True):
        y = mk.rope(x, freqs, pos, interleaved=interleaved, inverse=inverse, magnitude=1.25)
        _near(y, *P.rotate_tolerance(x, pos, freqs, dtype, 1.25, interleaved, inverse))
        assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("start", [0, 7, -5, (1 << 31) + 12345, 1 << 40])
def test_rope_far_positions_keep_their_angles(start):
    x = _randn((33, 2, 128), F32, 3)
    freqs, _ = mk.rope_freqs(128)
    y = mk.rope(x, freqs, start=start)
    # the reference angle itself is a 53-bit product: start * 2^-53 of a radian, and the turn's own 53 bits as much again
    want, tol = P.rotate_tolerance(x, start + torch.arange(33), freqs, F32)
    _near(y, want, tol + 4 * abs(start) * 2.0 ** -52 * x.double().cpu().abs().amax())


def test_rope_position_types_and_empty():
    x = _randn((6, 2, 64), BF, 4)
    freqs, _ = mk.rope_freqs(64)
    pos = torch.tensor([5, 0, 77, 3, 3, 100000])
    a = mk.rope(x, freqs, pos.to(torch.int32).cuda())
    b = mk.rope(x, freqs, pos.cuda())
    assert torch.equal(a, b)
    assert mk.rope(x[:0], freqs).shape == (0, 2, 64)
    assert mk.rope(x[:, :0], freqs).shape == (6, 0, 64)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_strides_alignment_and_in_place(dtype):
    freqs, _ = mk.rope_freqs(64)
    base = _randn((4, 50, 96), dtype, 5)
    heads_first = base[:, :, :64].transpose(0, 1)            # [heads, s, d], rows 96 apart
    want = mk.rope(heads_first.contiguous(), freqs, start=9)
    assert torch.equal(mk.rope(heads_first, freqs, start=9), want)
    odd = _randn((50 * 4 * 64 + 3,), dtype, 6)[3:].view(50, 4, 64)   # not on a 16-byte boundary
    ref = mk.rope(odd.clone(), freqs, start=9)
    assert torch.equal(mk.rope(odd, freqs, start=9), ref)
    one_apart = _randn((50, 4, 65), dtype, 7)[:, :, 1:]
    assert torch.equal(mk.rope(one_apart, freqs), mk.rope(one_apart.contiguous(), freqs))
    mk.rope(odd, freqs, start=9, out=odd)
    assert torch.equal(odd, ref)
    x = base[:, :, :64].transpose(0, 1)
    untouched = base[:, :, 64:].clone()
    mk.rope(x, freqs, start=9, out=x)
    assert torch.equal(x, want) and torch.equal(base[:, :, 64:], untouched)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    # against the formula's own derivative (autograd of the 64-bit form) and against differences
    x = _randn((5, 2, 64), F32, 8)
    dy = _randn((5, 2, 64), F32, 9)
    freqs, mag = mk.rope_freqs(32, scaling="by_parts", factor=4.0)
    pos = torch.tensor([0, 1, 1000, 54321, 7]).cuda()
    dx = mk.rope(dy, freqs, pos, interleaved=interleaved, magnitude=mag, inverse=True)
    _near(dx, *P.rotate_tolerance(dy, pos, freqs, F32, mag, interleaved, inverse=True))
    f = lambda t: float((P.rotate(t, pos, freqs, mag, interleaved) * dy.double().cpu()).sum())   # noqa: E731
    for at in [(0, 0, 0), (2, 1, 5), (3, 0, 17), (4, 1, 31), (1, 0, 40)]:
        h = torch.zeros(5, 2, 64, dtype=torch.float64)
        h[at] = 1e-3
        xd = x.double().cpu()
        # linear in x: the difference is the derivative up to the rounding of the 64-bit sums
        assert abs((f(xd + h) - f(xd - h)) / 2e-3 - float(dx[at])) < 1e-5


def test_rope_freqs_scalings():
    plain, m = mk.rope_freqs(128)
    i = torch.arange(64, dtype=torch.float64)
    assert m == 1.0 and torch.allclose(plain.cpu(), 10000.0 ** (-2 * i / 128), rtol=1e-14, atol=0)
    linear, _ = mk.rope_freqs(128, scaling="linear", factor=4.0)
    assert torch.allclose(linear, plain / 4, rtol=1e-14, atol=0)
    ntk, _ = mk.rope_freqs(128, scaling="ntk", factor=4.0)
    assert float(ntk[0]) == 1.0 and abs(float(ntk[-1] / plain[-1]) - 0.25) < 1e-12
    parts, m = mk.rope_freqs(128, scaling="by_parts", factor=8.0, original_length=4096)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], plain[turns >= 32])
    assert torch.allclose(parts[turns <= 1], plain[turns <= 1] / 8, rtol=1e-14, atol=0)
    assert ((parts <= plain) & (parts >= plain / 8 * (1 - 1e-12))).all()
    assert abs(m - (1 + 0.1 * math.log(8.0))) < 1e-15


# ------------------------------------------------------------------ append

LENGTHS = {
    "step": [(1, 1), (1, 16), (1, 17), (0, 9), (1, 33), (1, 100)],
    "prompts": [(70, 70), (33, 40), (0, 0), (1, 5), (16, 48), (129, 131)],
}


def _new_rows(batch, heads, d, dtype, seed):
    return [_randn((batch.tokens, heads, d), dtype, seed + i) for i in range(2)]


def _positions(batch):
    return torch.cat([torch.arange(t - n, t) for n, t in batch.lengths]) if batch.tokens else torch.zeros(0)


@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,d,rot,page,inter", [(BF, 128, 128, 16, False), (HF, 64, 32, 64, True),
                                                    (BF, 64, 64, 8, True), (HF, 128, 64, 256, False),
                                                    (BF, 24, 12, 16, False)])
def test_append_16_bit(dtype, d, rot, page, inter, lengths, order):
    batch = P.Batch(LENGTHS[lengths], page, seed=3)
    k, v, _, _ = P.random_cache(batch.n_pages, 3, page, d, dtype, 4, order)
    before = [k.clone(), v.clone()]
    cache = mk.KVCache(k, v)
    nk, nv = _new_rows(batch, 3, d, dtype, 10)
    q = _randn((batch.tokens, 7, d), dtype, 12)
    freqs, _ = mk.rope_freqs(rot)
    q_out = mk.kv_append(cache, nk, nv, batch.cu_q, batch.kv_len, batch.pages, q=q, freqs=freqs, interleaved=inter,
                         magnitude=1.5)
    _ok()
    pos = _positions(batch)
    _near(q_out, *P.rotate_tolerance(q, pos, freqs, dtype, 1.5, inter))
    want_k, tol = P.rotate_tolerance(nk, pos, freqs, dtype, 1.5, inter)
    touched = torch.zeros(batch.n_pages, page, dtype=torch.bool)
    t = 0
    for b, (n, length) in enumerate(batch.lengths):
        for i in range(n):
            j = length - n + i
            page_id, slot = batch.table[b][j // page], j % page
            touched[page_id, slot] = True
            _near(k[page_id, :, slot], want_k[t], tol[t])
            assert torch.equal(v[page_id, :, slot], nv[t])
            t += 1
    free = (~touched).cuda()
    for now, was in zip((k, v), before):
        assert torch.equal(now.transpose(1, 2)[free], was.transpose(1, 2)[free])


@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,d,rot,page,heads,inter", [(BF, 128, 128, 16, 3, False), (HF, 64, 32, 64, 5, True),
                                                          (BF, 64, 64, 8, 1, True), (BF, 128, 64, 256, 2, False),
                                                          (BF, 128, 0, 32, 9, False)])
def test_append_e4m3(dtype, d, rot, page, heads, inter, lengths, order):
    batch = P.Batch(LENGTHS[lengths], page, seed=5)
    k, v, ks, vs = P.random_cache(batch.n_pages, heads, page, d, P.E4M3, 6, order)
    ks.mul_(0.25)                              # some pages' scales have to grow, others stay
    was = [t.clone() for t in (k, v, ks, vs)]
    nk, nv = _new_rows(batch, heads, d, dtype, 20)
    nv[batch.tokens // 2] *= 30.0
    nk[batch.tokens // 3] = 0.0
    q = _randn((batch.tokens, 4, d), dtype, 22)
    freqs, _ = mk.rope_freqs(rot)
    q_out = mk.kv_append(mk.KVCache(k, v, ks, vs), nk, nv, batch.cu_q, batch.kv_len, batch.pages, q=q, freqs=freqs,
                         interleaved=inter)
    _ok()
    pos = _positions(batch)
    _near(q_out, *P.rotate_tolerance(q, pos, freqs, dtype, 1.0, inter))
    fresh = {0: P.rotate(nk, pos, freqs, 1.0, inter), 1: nv.double().cpu()}
    codes = {i: t.float().double().cpu() for i, t in enumerate((k, v))}
    old = {i: t.float().double().cpu() for i, t in enumerate((was[0], was[1]))}
    scales = {i: t.double().cpu() for i, t in enumerate((ks, vs))}
    old_scales = {i: t.double().cpu() for i, t in enumerate((was[2], was[3]))}
    hit = torch.zeros(batch.n_pages, dtype=torch.bool)
    for b, (n, length) in enumerate(batch.lengths):
        first = length - n
        if n == 0:
            continue
        for lp in range(first // page, -(-length // page)):
            page_id = batch.table[b][lp]
            hit[page_id] = True
            lo, hi = max(first, lp * page), min(length, (lp + 1) * page)
            rows = slice(batch.cu[b] + lo - first, batch.cu[b] + hi - first)
            for i in range(2):
                for h in range(heads):
                    x = fresh[i][rows, h]
                    s = P.e4m3_scale(float(x.abs().max()))
                    had = float(old_scales[i][page_id, h])
                    if lo > lp * page:
                        s = max(s, had)
                    assert float(scales[i][page_id, h]) == s
                    a, z = lo - lp * page, hi - lp * page
                    # half a step: 2^-4 of the value, 2^-10 in the subnormal range; fp32 arithmetic before it
                    err = (codes[i][page_id, h, a:z] - x / s).abs()
                    assert bool((err <= x.abs() / s * (2.0 ** -4 + 1e-5) + 2.0 ** -10 + 1e-5).all())
                    kept = old[i][page_id, h, :a] * (had / s)
                    if had == s or a == 0:
                        assert torch.equal(codes[i][page_id, h, :a], kept)
                    else:
                        err = (codes[i][page_id, h, :a] - kept).abs()
                        assert bool((err <= kept.abs() * 2.0 ** -4 + 2.0 ** -10).all())
                    assert torch.equal(codes[i][page_id, h, z:], old[i][page_id, h, z:])
    for i in range(2):
        assert torch.equal(codes[i][~hit], old[i][~hit]) and torch.equal(scales[i][~hit], old_scales[i][~hit])


def test_append_e4m3_one_token_at_a_time_equals_the_whole():
    # the scale that a page ends with does not depend on how its tokens came; codes differ by the second rounding alone
    page, d = 32, 64
    whole, steps = (mk.KVCache.empty(4, 2, page, d, P.E4M3) for _ in range(2))
    rows = _randn((40, 2, d), BF, 30)
    rows[:, 0] *= torch.linspace(0.1, 8.0, 40, device="cuda")[:, None].to(BF)
    pages = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    mk.kv_append(whole, rows, rows, i32(0, 40), i32(40), pages)
    for j in range(40):
        mk.kv_append(steps, rows[j:j + 1], rows[j:j + 1], i32(0, 1), i32(j + 1), pages)
    _ok()
    assert torch.equal(whole.k_scale, steps.k_scale) and torch.equal(whole.v_scale, steps.v_scale)
    a, b = whole.k.float(), steps.k.float()
    assert bool(((a - b).abs() <= 2.0 ** -9).all())      # powers of two: only subnormal codes are rounded twice
    assert torch.equal(whole.k.view(torch.uint8), whole.v.view(torch.uint8))


def test_append_e4m3_special_values():
    cache = mk.KVCache.empty(1, 1, 16, 64, P.E4M3)
    rows = torch.zeros(3, 1, 64, dtype=BF, device="cuda")
    rows[0, 0, 0], rows[0, 0, 1] = float("inf"), float("-inf")
    rows[0, 0, 2], rows[1, 0, 3] = float("nan"), 448.0
    rows[2, 0, 4] = 7.0
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    mk.kv_append(cache, rows, rows, i32(0, 3), i32(3), i32(0).view(1, 1))
    _ok()
    assert float(cache.k_scale[0, 0]) == 1.0 == float(cache.v_scale[0, 0])
    got = cache.v.float()[0, 0]
    assert float(got[0, 0]) == 448.0 and float(got[0, 1]) == -448.0 and math.isnan(float(got[0, 2]))
    assert float(got[1, 3]) == 448.0 and float(got[2, 4]) == 7.0
    zero = mk.KVCache.empty(1, 1, 16, 64, P.E4M3)
    mk.kv_append(zero, rows[:0].new_zeros(2, 1, 64), rows.new_zeros(2, 1, 64), i32(0, 2), i32(2), i32(0).view(1, 1))
    assert float(zero.k_scale[0, 0]) == 2.0 ** -100 and not zero.k.float().any()


@pytest.mark.parametrize("cache_dtype", [BF, P.E4M3])
def test_append_bad_pages_and_lengths_set_the_status(cache_dtype):
    # a page outside the cache, a length past the table, more new tokens than the length: stored where there
    # is a slot, and reported
    def fresh():
        return mk.KVCache.empty(4, 1, 16, 64, cache_dtype)

    rows = _randn((20, 1, 64), BF, 40)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    for bad in (-1, 4, 1 << 30):
        cache = fresh()
        mk.kv_append(cache, rows, rows, i32(0, 20), i32(20), i32(1, bad).view(1, 2))
        assert mk.device_status()[0] == mk.MK_ERR_INVALID
        assert cache.v.float()[1].any() and not cache.v.float()[[0, 2, 3]].any()
    cache = fresh()
    mk.kv_append(cache, rows, rows, i32(0, 20), i32(20), i32(1).view(1, 1))
    assert mk.device_status()[0] == mk.MK_ERR_CAPACITY
    assert cache.v.float()[1].any() and not cache.v.float()[[0, 2, 3]].any()
    cache = fresh()
    mk.kv_append(cache, rows, rows, i32(0, 20), i32(4), i32(3).view(1, 1))
    assert mk.device_status()[0] == mk.MK_ERR_CAPACITY
    assert cache.v.float()[3, :, :4].any() and not cache.v.float()[3, :, 4:].any()
    _ok()


def test_append_explicit_positions_and_no_rotation():
    batch = P.Batch([(3, 5), (2, 2)], 16, seed=1)
    nk, nv = _new_rows(batch, 2, 64, BF, 50)
    freqs, _ = mk.rope_freqs(64)
    pos = torch.tensor([9, 9, 1000000, 0, 3]).cuda()
    k, v, _, _ = P.random_cache(batch.n_pages, 2, 16, 64, BF, 51)
    mk.kv_append(mk.KVCache(k, v), nk, nv, batch.cu_q, batch.kv_len, batch.pages, freqs=freqs, positions=pos)
    assert torch.equal(k[batch.table[0][0], :, 2:5].transpose(0, 1), mk.rope(nk, freqs, pos)[:3])
    mk.kv_append(mk.KVCache(k, v), nk, nv, batch.cu_q, batch.kv_len, batch.pages)
    assert torch.equal(k[batch.table[1][0], :, :2].transpose(0, 1), nk[3:])
    _ok()


def test_large_cache_offsets_pass_32_bits():
    # 2^31 elements and more: the last page's slots are past any 32-bit offset
    n_pages, heads, page, d = 8300, 8, 256, 128
    cache = mk.KVCache(*(torch.empty(n_pages, heads, page, d, dtype=P.E4M3, device="cuda") for _ in range(2)),
                       *(torch.zeros(n_pages, heads, device="cuda") for _ in range(2)))
    assert cache.k.numel() > 1 << 31
    rows = _randn((5, heads, d), BF, 60)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    pages = i32(n_pages - 1).view(1, 1)
    mk.kv_append(cache, rows, rows, i32(0, 5), i32(5), pages)
    out = mk.paged_attention(rows, cache, i32(0, 5), i32(5), pages)
    _ok()
    got = cache.v[n_pages - 1].float() * cache.v_scale[n_pages - 1][:, None, None]
    err = (got[:, :5].transpose(0, 1).double() - rows.double()).abs()
    assert bool((err <= rows.double().abs() * 2.0 ** -4 + cache.v_scale[n_pages - 1].max() * 2.0 ** -10).all())
    assert torch.isfinite(out).all() and out.float().abs().max() > 0


def test_refusals():
    x = _randn((4, 2, 64), BF, 70)
    freqs, _ = mk.rope_freqs(64)
    with pytest.raises(ValueError):
        mk.rope(x, freqs.float())
    with pytest.raises(ValueError):
        mk.rope(x, freqs, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mk.rope(x[0], freqs)
    with pytest.raises(ValueError):
        mk.rope(x.transpose(1, 2), freqs)
    with pytest.raises(ValueError):
        mk.rope(x, freqs, out=x.float())
    with pytest.raises(mk.MkError):
        mk.rope(x, mk.rope_freqs(128)[0])
    with pytest.raises(ValueError):
        mk.rope(x.to(torch.int16), freqs)
    with pytest.raises(ValueError):
        mk.rope_freqs(63)
    with pytest.raises(ValueError):
        mk.rope_freqs(64, scaling="other")
    cache = mk.KVCache.empty(4, 2, 16, 64)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    args = (i32(0, 4), i32(4), i32(0).view(1, 1))
    with pytest.raises(ValueError):
        mk.kv_append(cache, x.half(), x.half(), *args)
    with pytest.raises(ValueError):
        mk.kv_append(cache, x[:, :1], x[:, :1], *args)
    with pytest.raises(ValueError):
        mk.kv_append(cache, x, x[:3], *args)
    with pytest.raises(ValueError):
        mk.kv_append(cache, x, x, args[0].long(), *args[1:])
    with pytest.raises(ValueError):
        mk.kv_append(cache, x, x, args[1], *args[1:])
    with pytest.raises(ValueError):
        mk.kv_append(cache, x, x, *args, q=x)
    with pytest.raises(ValueError):
        mk.KVCache(cache.k, cache.v.half())
    with pytest.raises(ValueError):
        mk.KVCache(cache.k, cache.v, torch.zeros(4, 2, device="cuda"), torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        mk.KVCache(cache.k.to(P.E4M3), cache.v.to(P.E4M3))
    odd = mk.KVCache.empty(4, 2, 48, 64)
    with pytest.raises(mk.MkError):
        mk.kv_append(odd, x, x, *args)
    eight = mk.KVCache.empty(4, 2, 16, 24, P.E4M3)
    with pytest.raises(mk.MkError):
        mk.kv_append(eight, x[..., :24], x[..., :24], *args)
    _ok()


def test_append_captures_into_a_graph_and_runs_on_another_stream():
    batch = P.Batch([(1, 20), (1, 7)], 16, seed=8)
    nk, nv = _new_rows(batch, 2, 64, BF, 80)
    freqs, _ = mk.rope_freqs(64)
    k, v, ks, vs = P.random_cache(batch.n_pages, 2, 16, 64, P.E4M3, 81)
    ref = mk.KVCache(k.clone(), v.clone(), ks.clone(), vs.clone())
    want_q = mk.kv_append(ref, nk, nv, batch.cu_q, batch.kv_len, batch.pages, q=nk, freqs=freqs)
    cache, ws = mk.KVCache(k, v, ks, vs), mk.Workspace()
    ws.get(256)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got_q = mk.kv_append(cache, nk, nv, batch.cu_q, batch.kv_len, batch.pages, q=nk, freqs=freqs, workspace=ws,
                         stream=side)
    side.synchronize()
    assert torch.equal(got_q, want_q) and torch.equal(cache.k.view(torch.uint8), ref.k.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q_graph = mk.kv_append(cache, nk, nv, batch.cu_q, batch.kv_len, batch.pages, q=nk, freqs=freqs, workspace=ws)
    nk.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_graph, mk.kv_append(ref, nk, nv, batch.cu_q, batch.kv_len, batch.pages, q=nk, freqs=freqs))
    assert torch.equal(cache.k.view(torch.uint8), ref.k.view(torch.uint8))
