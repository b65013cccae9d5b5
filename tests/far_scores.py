"""Paged attention where scores are so large that fp32 has few bits below 1 left for them (GPU tests' helpers).

Keys and queries along one axis, so that every score is an exact product; its distance to any other one is far above the
exponential's range, so that a row's result is the value of its largest score, but for the rounding of its weight and of the
output."""
import math

import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P


def distinct(n, dtype, sign, g):
    """n distinct values of the type in random order, of neighbouring magnitudes: positive, negative or both."""
    if dtype == P.E4M3:
        x = torch.arange(0x38, 0x7f, dtype=torch.uint8).view(P.E4M3).float().double()     # 1 .. 448
    else:
        x = (1.0 + torch.arange(0, 128, dtype=torch.float64) / 128.0)
        x = torch.cat([x * 2.0 ** e for e in range(-4, 1)])
    x = {"+": x, "-": -x, "+-": torch.cat([x, -x])}[sign]
    return x[torch.randperm(x.numel(), generator=g)[:n]]


def one_key_wins(lengths, d, page, heads, group, dtype, cache_dtype, sign, power, seed, causal=True, window=0, **how):
    """Runs a batch with scores of about 2^power; returns nothing, asserts the result."""
    if cache_dtype == P.E4M3:                             # as many keys as there are distinct codes
        lengths = [(n, min(length, 142 if sign == "+-" else 71)) for n, length in lengths]
    batch = P.Batch(lengths, page, seed=seed)
    k, v, ks, vs = P.random_cache(batch.n_pages, heads, page, d, cache_dtype, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    k.zero_()
    up = power // 2 if dtype == torch.float16 else power - 2      # the key's share of the magnitude: within the type
    if ks is not None:
        ks.fill_(2.0 ** (up - 8))
        vs.copy_(torch.exp2(torch.randint(-20, 20, vs.shape, generator=g).float()))
    for table, (_, length) in zip(batch.table, lengths):
        for h in range(heads):
            b = distinct(max(length, 0), cache_dtype, sign, g)
            for i, at in enumerate(table):
                part = b[i * page:(i + 1) * page]
                k[at, h, :part.numel(), 0] = (part if ks is not None else part * 2.0 ** up).to(cache_dtype).cuda()
    P.poison(k, ks, batch)
    P.poison(v, vs, batch)
    q = torch.zeros(batch.tokens, heads * group, d, dtype=dtype, device="cuda")
    q[..., 0] = 2.0 ** (power - up)
    out, lse = mk.paged_attention(q, mk.KVCache(k, v, ks, vs), batch.cu_q, batch.kv_len, batch.pages, return_lse=True,
                                  scale=1.0, causal=causal, window=window, **how)
    assert mk.device_status(how.get("workspace"))[0] == mk.MK_OK
    out, lse = out.double().cpu(), lse.double().cpu()
    for b, (n, length) in enumerate(lengths):
        if n == 0 or length <= 0:
            continue
        kk, vv = P.gather(k, ks, batch.table[b], length), P.gather(v, vs, batch.table[b], length)
        j, p = torch.arange(length), length - n + torch.arange(n)[:, None]
        see = (j <= p) if causal else torch.ones(n, length, dtype=torch.bool)
        if window:
            see = see & (j > p - window)
        some = see.any(dim=1)
        for h in range(heads * group):
            z = torch.where(see, kk[h // group, :, 0] * float(q[0, 0, 0]), -math.inf)
            best = z.argmax(dim=1)
            rows = slice(batch.cu[b], batch.cu[b] + n)
            want = torch.where(some[:, None], vv[h // group][best], 0.0).to(dtype).double()
            u = P.HALF_STEP[dtype]
            assert bool(((out[rows, h] - want).abs() <= want.abs() * (2 * u + u * u + 2.0 ** -21)).all()), (b, h)
            top = torch.where(some, z.amax(dim=1), 0.0)    # seven roundings of 2^-24 on the way to lse
            assert bool(((lse[rows, h] - top).abs() <= top.abs() * 2.0 ** -21)[some].all())
            assert bool(torch.isinf(lse[rows, h][~some]).all())


def all_keys_alike(lengths, d, page, heads, group, dtype, cache_dtype, power, seed, one_run, **how):
    """Equal scores: the mean of the values, where a CTA has a unit to itself (a lse of this size has no room for the
    logarithm of the number of keys, so partial results of several CTAs join as if each had the same); else within
    the values' range."""
    batch = P.Batch(lengths, page, seed=seed)
    k, v, ks, vs = P.random_cache(batch.n_pages, heads, page, d, cache_dtype, seed + 1)
    k.zero_()
    k[..., 0] = 1.0
    up = power // 2
    if ks is not None:
        ks.fill_(2.0 ** up)
        vs.fill_(1.0 / 64)
    else:
        k[..., 0] = 2.0 ** up
    P.poison(k, ks, batch)
    P.poison(v, vs, batch)
    q = torch.zeros(batch.tokens, heads * group, d, dtype=dtype, device="cuda")
    q[..., 0] = 2.0 ** (power - up)
    cfg = mk.Config(max_ctas=1) if one_run else None
    out = mk.paged_attention(q, mk.KVCache(k, v, ks, vs), batch.cu_q, batch.kv_len, batch.pages, scale=1.0, cfg=cfg, **how)
    assert mk.device_status()[0] == mk.MK_OK
    step = P.HALF_STEP[dtype]
    for b, (n, length) in enumerate(lengths):
        for t in range(n):
            seen = length - n + t + 1
            if seen <= 0:
                assert bool((out[batch.cu[b] + t] == 0).all())
                continue
            vv = P.gather(v, vs, batch.table[b], length)[:, :seen].repeat_interleave(group, dim=0)
            got = out[batch.cu[b] + t].double().cpu()
            if one_run:     # equal weights; fp32 sums, one rounding of the output
                want, size = vv.mean(dim=1), vv.abs().mean(dim=1)
                assert bool(((got - want).abs() <= step * want.abs() + size * (seen + 4) * 2.0 ** -24 * (1 + step) + 1e-30).all())
            else:
                slack = vv.abs().amax(dim=1) * (step + (seen + 8) * 2.0 ** -22)
                assert bool((got <= vv.amax(dim=1) + slack).all() and (got >= vv.amin(dim=1) - slack).all())


def ordinary_rows_beside(problem, check, **how):
    """Every third query head has scores far from 0; the others' results keep their ordinary bounds."""
    batch, q, cache = problem
    heads = q.shape[1]
    far = torch.arange(heads) % 3 == 1
    large = q.clone()
    large[:, far.to(q.device)] *= 2.0 ** 13 if q.dtype == torch.float16 else 2.0 ** 30
    out, lse = mk.paged_attention(large, cache, batch.cu_q, batch.kv_len, batch.pages, return_lse=True, **how)
    assert mk.device_status()[0] == mk.MK_OK
    assert bool(torch.isfinite(out).all()) and not bool(torch.isnan(lse).any())
    plain, plain_lse = mk.paged_attention(q, cache, batch.cu_q, batch.kv_len, batch.pages, return_lse=True, **how)
    f = far.to(q.device)[None, :]
    check(batch, q, cache, got=(torch.where(f[..., None], plain, out), torch.where(f, plain_lse, lse)), **how)
    for b, (n, length) in enumerate(batch.lengths):       # a mean of values: within the largest of them
        if n and length > 0:
            v = P.gather(cache.v, cache.v_scale, batch.table[b], length).abs().amax(dim=1)
            v = v.repeat_interleave(heads // v.shape[0], dim=0)
            mine = out[batch.cu[b]:batch.cu[b] + n].double().cpu().abs()
            assert bool((mine <= v * (1 + 2.1 * P.HALF_STEP[q.dtype])).all())
