"""Attention over a paged cache against plain 64-bit arithmetic (GPU): decode steps, pieces of prompts, whole prompts.

Slots that hold no token are NaN in every test (and the scales of pages that hold none), table entries past a
sequence's end are nonsense, pages come in random order.
"""
import math

import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


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


def _problem(lengths, heads, group, d, page, dtype, cache_dtype, order="heads", seed=0):
    batch = P.Batch(lengths, page, seed=seed)
    k, v, ks, vs = P.random_cache(batch.n_pages, heads, page, d, cache_dtype, seed + 1, order)
    P.poison(k, ks, batch)
    P.poison(v, vs, batch)
    q = _randn((batch.tokens, heads * group, d), dtype, seed + 2)
    return batch, q, mk.KVCache(k, v, ks, vs)


def _check(batch, q, cache, got=None, **how):
    out, lse = got or mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, return_lse=True, **how)
    how.pop("max_q", None), how.pop("cfg", None), how.pop("workspace", None)
    want, want_lse, tol, tol_lse = P.attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, batch, **how)
    bad = ((out.double().cpu() - want).abs() - tol).max() if want.numel() else torch.tensor(0.0)
    assert float(bad) <= 0, float(bad)
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse.cpu()) & (lse.cpu() < 0), empty)
    assert bool((out.cpu()[empty] == 0).all())
    err = ((lse.double().cpu() - want_lse).abs() - tol_lse)[~empty]
    assert not err.numel() or float(err.max()) <= 0, float(err.max())
    return out, lse


# (type of q, type of the cache)
TYPES = [(BF, BF), (HF, HF), (BF, P.E4M3)]
# new tokens, tokens in all: one token, ends inside pages and tiles, a sequence without new tokens, an empty one,
# one with more new tokens than tokens, a few tokens at once
STEP = [(1, 1), (1, 63), (1, 64), (1, 65), (0, 30), (1, 130), (2, 2), (0, 0), (1, 0), (3, 2), (4, 200), (1, 1000)]
PROMPTS = [(130, 130), (1, 77), (0, 0), (257, 300), (64, 1000), (5, 3), (300, 300), (33, 33), (128, 128)]


@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("d,page,heads,group", [(128, 16, 2, 4), (64, 64, 1, 1), (128, 8, 1, 8), (64, 256, 3, 5),
                                                (128, 128, 1, 16), (64, 32, 2, 3)])
def test_steps(d, page, heads, group, dtype, cache_dtype, order):
    problem = _problem(STEP, heads, group, d, page, dtype, cache_dtype, order, seed=10)
    out, lse = _check(*problem)
    _ok()
    again = mk.paged_attention(problem[1], problem[2], problem[0].cu_q, problem[0].kv_len, problem[0].pages, max_q=4)
    assert torch.equal(out, again)              # the same bits, whatever the hint and whatever ran before


@pytest.mark.parametrize("causal,window,sinks", [(True, 1, 0), (True, 64, 4), (True, 100, 0), (True, 130, 70),
                                                 (True, 5000, 3), (False, 0, 0), (False, 40, 1), (True, 64, 1 << 20)])
@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("lengths", ["step", "prompts"])
def test_windows_and_sinks(lengths, dtype, cache_dtype, causal, window, sinks):
    _check(*_problem(STEP if lengths == "step" else PROMPTS, 2, 3, 64, 16, dtype, cache_dtype, seed=20), causal=causal,
           window=window, sinks=sinks)
    _ok()


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("d,page,heads,group,order", [(128, 16, 2, 4, "heads"), (64, 64, 1, 1, "tokens"),
                                                      (128, 8, 1, 7, "tokens"), (64, 256, 2, 3, "heads"),
                                                      (128, 128, 1, 40, "heads")])
def test_prompts(d, page, heads, group, order, dtype, cache_dtype):
    _check(*_problem(PROMPTS, heads, group, d, page, dtype, cache_dtype, order, seed=30))
    _ok()


@pytest.mark.parametrize("max_ctas", [1, 3, 40])
@pytest.mark.parametrize("lengths", ["step", "prompts"])
@pytest.mark.parametrize("dtype,cache_dtype", [(BF, BF), (BF, P.E4M3)])
def test_few_ctas(dtype, cache_dtype, lengths, max_ctas):
    _check(*_problem(STEP if lengths == "step" else PROMPTS, 2, 2, 128, 32, dtype, cache_dtype, seed=40),
           cfg=mk.Config(max_ctas=max_ctas))
    _ok()


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_long_sequence_is_joined(dtype, cache_dtype):
    # one sequence over every CTA: many partial rows to join
    _check(*_problem([(1, 40000)], 1, 4, 128, 64, dtype, cache_dtype, seed=50))
    _check(*_problem([(2, 9000), (1, 1), (1, 20000)], 2, 8, 64, 16, dtype, cache_dtype, seed=51), window=6000, sinks=5)
    _ok()


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
@pytest.mark.parametrize("n", [1, 200])
def test_large_scores(n, dtype, cache_dtype):
    # scale 1: scores with a standard deviation near 8 to 11, so maxima grow during a row and most weights vanish
    _check(*_problem([(n, 700), (n, 300)], 2, 2, 128, 16, dtype, cache_dtype, seed=60), scale=1.0)
    _ok()


@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("magnitude", [2.0 ** -60, 2.0 ** 40])
def test_8_bit_cache_ranges(n, magnitude):
    # rows and scales far from 1 keep their bits: q at 2^-60 / 2^40, key scales the other way round, value scales that
    # differ by 2^20 between pages
    batch, q, cache = _problem([(n, 500), (n, 200)], 2, 4, 128, 16, BF, P.E4M3, seed=70)
    q = (q.float() * magnitude).to(BF)
    cache.k_scale.div_(magnitude)
    cache.v_scale[::2] *= 2.0 ** 20
    cache.v_scale[1::3] *= 2.0 ** -20
    _check(batch, q, cache)
    _ok()


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_zero_queries_give_the_mean(dtype, cache_dtype):
    # every score 0: each weight is 1, sums of small integers are exact in fp32 and so is a power-of-two count
    batch = P.Batch([(1, 256), (40, 512)], 32, seed=80)
    k, v, ks, vs = P.random_cache(batch.n_pages, 2, 32, 64, cache_dtype, 81)
    g = torch.Generator().manual_seed(82)
    v.copy_(torch.randint(-2, 3, v.shape, generator=g).float().cuda().to(v.dtype))
    if vs is not None:
        vs.fill_(1.0)
    q = torch.zeros(batch.tokens, 4, 64, dtype=dtype, device="cuda")
    out = mk.paged_attention(q, mk.KVCache(k, v, ks, vs), batch.cu_q, batch.kv_len, batch.pages, causal=False)
    _ok()
    for b, (n, length) in enumerate(batch.lengths):
        mean = P.gather(v, vs, batch.table[b], length).mean(dim=1).to(dtype)
        for t in range(batch.cu[b], batch.cu[b] + n):
            assert torch.equal(out[t].cpu(), mean.repeat_interleave(2, dim=0))


@pytest.mark.parametrize("dtype,cache_dtype", TYPES)
def test_nan_in_a_seen_key_or_value_reaches_exactly_the_rows_that_see_it(dtype, cache_dtype):
    # a later token's NaN must not reach the rows before it, in the same tile or not
    for n in (4, 200):
        batch, q, cache = _problem([(n, 230), (n, 230)], 1, 2, 64, 16, dtype, cache_dtype, seed=90)
        clean = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages)
        at = 228
        page, slot = batch.table[0][at // 16], at % 16
        for t in (cache.v, cache.k):
            was = t[page, 0, slot].clone()
            if t.dtype == P.E4M3:
                t.view(torch.uint8)[page, 0, slot, 3] = 0x7f
            else:
                t[page, 0, slot, 3] = float("nan")
            out = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages)
            _ok()
            sees = torch.arange(230 - n, 230) >= at
            hit = out[:n].cpu()[sees]
            assert torch.isnan(hit[..., 3]).all()
            if t is cache.v:
                others = [c for c in range(64) if c != 3]
                assert not torch.isnan(hit[..., others]).any()
            else:
                assert torch.isnan(hit).all()
            assert torch.equal(out[:n].cpu()[~sees], clean[:n].cpu()[~sees])
            assert torch.equal(out[n:], clean[n:])
            t.view(torch.uint8)[page, 0, slot] = was.view(torch.uint8)


@pytest.mark.parametrize("n", [1, 140])
@pytest.mark.parametrize("bad", [-1, 1 << 20, 1 << 30])
def test_bad_pages_set_the_status(n, bad):
    batch, q, cache = _problem([(n, 200), (n, 150)], 1, 2, 64, 16, BF, BF, seed=100)
    want = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages)
    _ok()
    pages = batch.pages.clone()
    pages[0, 3] = bad
    out = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, pages)
    assert mk.device_status()[0] == mk.MK_ERR_INVALID
    assert torch.equal(out[n:], want[n:])
    short = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages[:, :11])     # 200 tokens need 13 pages
    assert mk.device_status()[0] == mk.MK_ERR_CAPACITY
    assert torch.equal(short[n:], want[n:])
    _ok()


def test_strides_streams_and_out():
    batch, q, cache = _problem([(1, 90), (70, 100)], 2, 2, 64, 16, BF, BF, seed=110)
    want, lse = _check(batch, q, cache)
    wide = torch.zeros(batch.tokens, 12, 64, dtype=BF, device="cuda")
    wide[:, 4:8] = q
    out = torch.full((4, batch.tokens, 64), 7.0, dtype=BF, device="cuda").transpose(0, 1)
    side, ws = torch.cuda.Stream(), mk.Workspace()
    side.wait_stream(torch.cuda.current_stream())
    got = mk.paged_attention(wide[:, 4:8], cache, batch.cu_q, batch.kv_len, batch.pages, out=out, stream=side,
                             workspace=ws)
    side.synchronize()
    _ok(ws)
    assert got is out and torch.equal(out, want)
    empty = mk.paged_attention(q[:0], cache, batch.cu_q[:1] * 0, batch.kv_len[:0], batch.pages[:0])
    assert empty.shape == (0, 4, 64)


@pytest.mark.parametrize("n", [1, 150])
def test_a_captured_call_follows_the_lengths(n):
    # lengths live on the device: a graph captured once serves every later step
    batch, q, cache = _problem([(n, 400), (n, 333)], 2, 4, 128, 32, BF, BF, seed=120)
    ws = mk.Workspace()
    call = lambda: mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, workspace=ws, max_q=n)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for lengths in ((400, 333), (160, 150), (398, 300)):
        batch.kv_len.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages))
    _ok(ws)


def test_more_sequences_than_one_launch_takes():
    lengths = [(1, 1 + (37 * i) % 90) for i in range(2500)]
    _check(*_problem(lengths, 1, 2, 64, 16, BF, BF, seed=130))
    _ok()


def test_random_batches():
    # seeded random shapes over the whole range of arguments
    import random
    r = random.Random(7)
    for i in range(24):
        dtype, cache_dtype = r.choice(TYPES)
        lengths = []
        for _ in range(r.randint(1, 6)):
            n = r.choice([0, 1, 1, 2, r.randint(1, 40), r.randint(1, 400)])
            lengths.append((n, max(0, n + r.choice([-2, 0, 0, 1, r.randint(0, 100), r.randint(0, 1500)]))))
        window = r.choice([0, 0, r.randint(1, 300)])
        _check(*_problem(lengths, r.choice([1, 2, 3]), r.choice([1, 2, 5, 8]), r.choice([64, 128]),
                         r.choice([8, 16, 32, 64, 128, 256]), dtype, cache_dtype, r.choice(["heads", "tokens"]), seed=200 + i),
               causal=r.random() < 0.85, window=window, sinks=r.choice([0, r.randint(1, 200)]),
               cfg=mk.Config(max_ctas=r.choice([0, 0, 1, 7])))
    _ok()


def test_refusals():
    batch, q, cache = _problem([(1, 20)], 2, 2, 64, 16, BF, BF, seed=140)
    rest = (batch.cu_q, batch.kv_len, batch.pages)
    with pytest.raises(ValueError):
        mk.paged_attention(q.half(), cache, *rest)
    with pytest.raises(ValueError):
        mk.paged_attention(q.float(), cache, *rest)
    with pytest.raises(ValueError):
        mk.paged_attention(q[..., :32], cache, *rest)
    with pytest.raises(ValueError):
        mk.paged_attention(q.cpu(), cache, *rest)
    with pytest.raises(ValueError):
        mk.paged_attention(q, cache, batch.cu_q.long(), *rest[1:])
    with pytest.raises(ValueError):
        mk.paged_attention(q, cache, *rest, out=q[:, :2])
    with pytest.raises(mk.MkError):
        mk.paged_attention(q[:, :3], cache, *rest)
    with pytest.raises(mk.MkError):
        mk.paged_attention(q, cache, *rest, scale=0.0)
    with pytest.raises(mk.MkError):
        mk.paged_attention(q, cache, *rest, window=-1)
    wide = mk.KVCache.empty(2, 2, 16, 96)
    with pytest.raises(mk.MkError):
        mk.paged_attention(_randn((1, 2, 96), BF, 1), wide, *rest)
    eight = mk.KVCache.empty(2, 2, 16, 64, P.E4M3)
    with pytest.raises(ValueError):
        mk.paged_attention(q.half(), eight, *rest)
    _ok()


def test_rope_append_attend_is_causal_attention_over_the_rotated_sequence():
    # the three operators together, a prompt in two pieces and then single tokens: as one pass over the whole sequence
    d, heads, group, page, T = 64, 2, 4, 16, 75
    q, k, v = (_randn((T, h, d), BF, 150 + h) for h in (heads * group, heads, heads))
    freqs, _ = mk.rope_freqs(d)
    cache = mk.KVCache.empty(6, heads, page, d)
    pages = torch.tensor([[4, 0, 5, 2, 1]], dtype=torch.int32, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    outs, at = [], 0
    for n in [30, 40, 1, 1, 3]:
        args = (i32(0, n), i32(at + n), pages)
        qr = mk.kv_append(cache, k[at:at + n], v[at:at + n], *args, q=q[at:at + n], freqs=freqs)
        outs.append(mk.paged_attention(qr, cache, *args, max_q=n))
        at += n
    _ok()
    qr, kr = mk.rope(q, freqs), mk.rope(k, freqs)
    whole = P.Batch([(T, T)], page, seed=1)
    whole.table = [[4, 0, 5, 2, 1]]
    assert torch.equal(cache.k[whole.table[0]].transpose(1, 2).reshape(-1, heads, d)[:T], kr)
    want, _, tol, _ = P.attention(qr, cache.k, cache.v, None, None, whole)
    assert bool(((torch.cat(outs).double().cpu() - want).abs() <= tol).all())
    # and the same rows as the framework's ring attention computes, with every query head its own key head
    ring = mk.ring_attention([t.transpose(0, 1).repeat_interleave(s, 0).expand(-1, -1, -1).contiguous()
                              for t, s in ((_pad(qr), 1),)],
                             [_pad(kr).transpose(0, 1).repeat_interleave(group, 0).contiguous()],
                             [_pad(v).transpose(0, 1).repeat_interleave(group, 0).contiguous()], causal=True,
                             scale=1.0 / math.sqrt(d))[0]
    both = (torch.cat(outs).float() - ring[:, :, :d].transpose(0, 1).float()).abs().double().cpu()
    assert bool((both <= 2 * tol + 2.0 ** -8 * want.abs()).all())


def _pad(t):
    """The d = 128 row that ring_attention wants: the upper half zeros."""
    return torch.cat((t, torch.zeros_like(t)), dim=-1)
