"""Cases of the cache-and-attention operators: rotary positions, appending to a paged key/value cache, attention over it.

`listed()` gives fixed cases, `draw(rng)` one more of the same ranges, `prepare` the tensors a serving program holds
before the call, `run` one pass (the plain torch form, or the framework's calls where `own` is set), `work` the bytes and
operations of a pass, and `exact` the result in 64 bits, computed sequence by sequence.

Definitions.  A sequence b of a batch has n_b new tokens (rows cu_q[b] .. cu_q[b+1]-1 of the token arrays) and, with them,
kv_len[b] tokens; its token j lives in slot j % page of page pages[b, j // page].  New token i has position
p_i = kv_len[b] - n_b + i.
  rotation  pair (a, b) of a head at position p, frequency f: (a cos - b sin, b cos + a sin) * magnitude, angle p * f
  append    k (rotated) and v go to their slots.  8-bit caches hold e4m3 codes and one power-of-two scale per (page, head):
            the least 2^e (e >= -100) with amax <= 448 * 2^e over the page's new tokens, and not below the scale the page
            already has when it holds earlier tokens, whose codes are rounded again where the scale grows
  attention token i sees key j of its sequence if j <= p_i and (no window, or j > p_i - window, or j < sinks)
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 16 sequences whose positions lie about a million tokens in: latency, and exact far angles
        {"name": "rope step", "op": "rope", "tokens": 16, "heads": 40, "d": 128, "rot": 128, "type": "bf16",
         "layout": "tokens", "interleaved": False, "scaled": False, "far": 1000003, "gradient": False},
        # part of each head rotated, interleaved pairs, a mid-size fp32 batch of odd length
        {"name": "rope part", "op": "rope", "tokens": 4099, "heads": 12, "d": 128, "rot": 64, "type": "fp32",
         "layout": "tokens", "interleaved": True, "scaled": False, "far": 0, "gradient": False},
        # the ring attention workload's 32768 positions of 8 heads in its [heads, positions, d] layout, long-context
        # scaling, with the gradient of a training step
        {"name": "rope prompt", "op": "rope", "tokens": 32768, "heads": 8, "d": 128, "rot": 128, "type": "bf16",
         "layout": "heads", "interleaved": False, "scaled": True, "far": 0, "gradient": True},
        # a decode step: one token for each of 64 short sequences
        {"name": "append step", "op": "append", "batch": 64, "new_lo": 1, "new_hi": 1, "past_lo": 0, "past_hi": 60,
         "heads_q": 32, "heads": 8, "d": 128, "rot": 128, "page": 16, "type": "bf16", "cache": "same",
         "interleaved": False, "order": "heads"},
        # a decode step into an 8-bit cache: page scales grow
        {"name": "append step e4m3", "op": "append", "batch": 128, "new_lo": 1, "new_hi": 1, "past_lo": 0, "past_hi": 130,
         "heads_q": 64, "heads": 8, "d": 128, "rot": 128, "page": 32, "type": "bf16", "cache": "e4m3",
         "interleaved": False, "order": "heads"},
        # prompts of ragged length into an 8-bit cache
        {"name": "append prompts e4m3", "op": "append", "batch": 5, "new_lo": 1000, "new_hi": 6001, "past_lo": 0,
         "past_hi": 40, "heads_q": 32, "heads": 8, "d": 128, "rot": 128, "page": 64, "type": "bf16", "cache": "e4m3",
         "interleaved": False, "order": "heads"},
        # one user's decode step: latency
        {"name": "decode one", "op": "attention", "batch": 1, "new_lo": 1, "new_hi": 1, "past_lo": 2001, "past_hi": 2001,
         "heads_q": 32, "heads": 8, "d": 128, "page": 16, "type": "bf16", "cache": "same", "window": 0, "sinks": 0},
        # a full serving batch over an 8-bit cache
        {"name": "decode many e4m3", "op": "attention", "batch": 128, "new_lo": 1, "new_hi": 1, "past_lo": 100,
         "past_hi": 32000, "heads_q": 64, "heads": 8, "d": 128, "page": 64, "type": "bf16", "cache": "e4m3", "window": 0,
         "sinks": 0},
        # long chats of a windowed model: a few first tokens and the last 4096 are read out of long caches
        {"name": "decode window", "op": "attention", "batch": 48, "new_lo": 1, "new_hi": 1, "past_lo": 1000,
         "past_hi": 60000, "heads_q": 32, "heads": 8, "d": 64, "page": 32, "type": "fp16", "cache": "same",
         "window": 4096, "sinks": 4},
        # the next piece of two long prompts, over an 8-bit cache
        {"name": "chunk e4m3", "op": "attention", "batch": 2, "new_lo": 700, "new_hi": 1025, "past_lo": 15000,
         "past_hi": 30000, "heads_q": 32, "heads": 8, "d": 128, "page": 32, "type": "bf16", "cache": "e4m3", "window": 0,
         "sinks": 0},
        # ragged prompts of a windowed model with an odd number of query heads for each key head
        {"name": "prompts window", "op": "attention", "batch": 6, "new_lo": 300, "new_hi": 3001, "past_lo": 0,
         "past_hi": 200, "heads_q": 10, "heads": 2, "d": 64, "page": 16, "type": "fp16", "cache": "same", "window": 512,
         "sinks": 16},
        # a whole prompt
        {"name": "prompt", "op": "attention", "batch": 1, "new_lo": 8192, "new_hi": 8192, "past_lo": 0, "past_hi": 0,
         "heads_q": 32, "heads": 8, "d": 128, "page": 64, "type": "bf16", "cache": "same", "window": 0, "sinks": 0},
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention"])
    if op == "rope":
        d = rng.choice([64, 128])
        tokens = _between(rng, 1, 32768)
        return {"op": op, "tokens": tokens, "heads": rng.randint(1, 8 if tokens > 8000 else 40), "d": d,
                "rot": rng.choice([d, d, d // 2]), "type": rng.choice(["bf16", "fp16", "fp32"]),
                "layout": rng.choice(["tokens", "heads"]), "interleaved": rng.random() < 0.5,
                "scaled": rng.random() < 0.5, "far": rng.choice([0, 0, rng.randint(1, 1 << 20)]),
                "gradient": rng.random() < 0.5}
    heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    page = rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128])
    kind = rng.choice(["bf16", "bf16", "fp16"])
    cache = "e4m3" if kind == "bf16" and rng.random() < 0.5 else "same"
    case = {"op": op, "heads_q": heads * group, "heads": heads, "d": d, "page": page, "type": kind, "cache": cache}
    if op == "append":
        step = rng.random() < 0.5
        batch = _between(rng, 1, 128) if step else rng.randint(1, 6)
        lo = 1 if step else _between(rng, 2, 1000)
        return {**case, "batch": batch, "new_lo": lo, "new_hi": 1 if step else rng.randint(lo, 4000), "past_lo": 0,
                "past_hi": rng.randint(0, 200), "rot": rng.choice([d, d, d // 2]), "interleaved": rng.random() < 0.5,
                "order": rng.choice(["heads", "tokens"])}
    window = rng.choice([0, 0, _between(rng, 16, 4096)])
    case.update(window=window, sinks=rng.randint(0, 64) if window else 0)
    if rng.random() < 0.6:   # decode, now and then with a few tokens at once
        batch = _between(rng, 1, 96)
        lo = rng.randint(0, 500)
        return {**case, "batch": batch, "new_lo": 1, "new_hi": rng.choice([1, 1, 1, 4]), "past_lo": lo,
                "past_hi": max(lo, _between(rng, 1, 24000))}
    lo = _between(rng, 16, 700)
    return {**case, "batch": rng.randint(1, 3), "new_lo": lo, "new_hi": rng.randint(lo, 2500), "past_lo": 0,
            "past_hi": rng.randint(0, 4000)}


def _spread(count, lo, hi, shift):
    """`count` whole numbers spread evenly over lo .. hi in a mixed order; the same for every seed."""
    return [lo + int(((i + shift) * GOLDEN % 1.0) * (hi - lo + 1)) for i in range(count)]


def _lengths(case):
    new = _spread(case["batch"], case["new_lo"], case["new_hi"], 1)
    past = _spread(case["batch"], case["past_lo"], case["past_hi"], 2)
    return new, [p + n for p, n in zip(past, new)]


# ------------------------------------------------------------------ inputs

def _frequencies(rot, scaled, device):
    """Frequencies in 64 bits: base 10000; scaled by parts for a context 8 times 4096 (slow ones divided by 8)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    if not scaled:
        return f, 1.0
    turns = 4096.0 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f * keep + f / 8.0 * (1.0 - keep), 1.0 + 0.1 * math.log(8.0)


def _normal(g, shape, dtype):
    return torch.randn(shape, dtype=torch.float32, device="cuda", generator=g).to(dtype)


def _cache(case, g, n_pages):
    """(k, v, k_scale, v_scale) with page indexes first, then heads, slots, d; random contents."""
    shape = (n_pages, case["heads"], case["page"], case["d"])
    if case.get("order") == "tokens":
        shape = (n_pages, case["page"], case["heads"], case["d"])
    got = []
    for _ in range(2):
        if case["cache"] == "e4m3":
            t = torch.empty(shape, dtype=E4M3, device="cuda")
            for part in t.split(max(1, (1 << 28) // (shape[1] * shape[2] * shape[3]))):
                part.copy_((torch.randn(part.shape, device="cuda", generator=g) * 96.0).clamp_(-E4M3_MAX, E4M3_MAX))
        else:
            t = torch.empty(shape, dtype=TYPES[case["type"]], device="cuda").normal_(generator=g)
        got.append(t.transpose(1, 2) if case.get("order") == "tokens" else t)
    if case["cache"] == "e4m3":
        for _ in range(2):
            e = torch.randint(-8, -5, (n_pages, case["heads"]), device="cuda", generator=g)
            got.append(torch.exp2(e.float()))
    else:
        got += [None, None]
    return got


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]
    if case["op"] == "rope":
        shape = (case["tokens"], case["heads"], case["d"])
        if case["layout"] == "heads":
            shape = (case["heads"], case["tokens"], case["d"])
        turn = (lambda t: t.transpose(0, 1)) if case["layout"] == "heads" else (lambda t: t)
        s = {"case": case, "x": turn(_normal(g, shape, dtype)), "dy": None}
        if case["gradient"]:
            s["dy"] = turn(_normal(g, shape, dtype))
        p = torch.arange(case["tokens"], device="cuda", dtype=torch.int64)
        # far: every token is the next one of a sequence of its own, so the positions are scattered
        s["positions"] = p if not case["far"] else case["far"] + torch.randint(0, 4096, p.shape, device="cuda", generator=g)
        s["freqs"], s["magnitude"] = _frequencies(case["rot"], case["scaled"], "cuda")
        return s
    new, total = _lengths(case)
    counts = [-(-t // case["page"]) for t in total]
    n_pages, width = sum(counts) + 3, max(counts)
    order = torch.randperm(n_pages, device="cuda", generator=g).to(torch.int32)
    pages = torch.zeros((case["batch"], max(1, width)), dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        pages[b, :c] = order[at:at + c]
        at += c
    k, v, ks, vs = _cache(case, g, n_pages)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = {"case": case, "k": k, "v": v, "k_scale": ks, "v_scale": vs, "pages": pages, "max_new": max(new),
         "max_kv": max(total), "q": _normal(g, (cu[-1], case["heads_q"], case["d"]), dtype),
         "cu_q": torch.tensor(cu, dtype=torch.int32, device="cuda"),
         "kv_len": torch.tensor(total, dtype=torch.int32, device="cuda")}
    if case["op"] == "append":
        s["new_k"] = _normal(g, (cu[-1], case["heads"], case["d"]), dtype)
        s["new_v"] = _normal(g, (cu[-1], case["heads"], case["d"]), dtype)
        s["freqs"], s["magnitude"] = _frequencies(case["rot"], False, "cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _rotate(x, positions, freqs, magnitude, interleaved, inverse=False):
    """x: [tokens, heads, d] rotated in 32 bits (angles in 64); the result in 32 bits."""
    rot = 2 * freqs.numel()
    angle = positions.to(torch.float64)[:, None] * freqs[None, :]
    c = (angle.cos() * magnitude).float()[:, None, :]
    s = (angle.sin() * (-magnitude if inverse else magnitude)).float()[:, None, :]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _token_rows(s):
    """For every new token: its sequence, its position there, its page and its slot."""
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    pos = s["kv_len"].long()[b] - s["cu_q"].long()[b + 1] + t
    page = s["pages"].long()[b, pos // s["case"]["page"]]
    return b, pos, page, pos % s["case"]["page"]


def _store(cache, scale, x, page, slot):
    """Writes x [tokens, heads, d] (32 bits) to its slots; 8-bit caches quantise it and grow the pages' scales."""
    if scale is None:
        cache[page, :, slot] = x.to(cache.dtype)
        return
    n_pages, size = cache.shape[0], cache.shape[2]
    finite = torch.where(x.isfinite(), x.abs(), 0.0).amax(dim=-1)
    amax = torch.zeros(scale.shape, device="cuda").scatter_reduce(0, page[:, None].expand_as(finite), finite, "amax")
    m, e = torch.frexp(amax / E4M3_MAX)
    need = torch.ldexp(torch.ones_like(m), torch.where(m > 0.5, e, e - 1).clamp_min(-100))
    first = torch.full((n_pages,), size, device="cuda").scatter_reduce(0, page, slot, "amin")
    touched = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
    touched[page] = True
    grown = torch.where((first > 0)[:, None], torch.maximum(scale, need), need)
    hit = touched.nonzero()[:, 0]
    ratio = (scale[hit] / grown[hit])[:, :, None, None]
    old = cache[hit].float()
    kept = (torch.arange(size, device="cuda")[None, :] < first[hit][:, None])[:, None, :, None]
    cache[hit] = torch.where(kept, old * ratio, old).to(cache.dtype)
    scale[hit] = grown[hit]
    cache[page, :, slot] = (x / scale[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(cache.dtype)


def _append(s):
    c = s["case"]
    _, pos, page, slot = _token_rows(s)
    turn = (pos, s["freqs"], s["magnitude"], c["interleaved"])
    _store(s["k"], s["k_scale"], _rotate(s["new_k"], *turn), page, slot)
    _store(s["v"], s["v_scale"], s["new_v"].float(), page, slot)
    return _rotate(s["q"], *turn).to(s["q"].dtype)


def _gathered(cache, scale, pages):
    """[batch, heads, keys, d] in 32 bits: the pages of each sequence in order."""
    x = cache[pages.long()].float()
    if scale is not None:
        x = x * scale[pages.long()][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attention(s):
    c = s["case"]
    B, H, n, d = c["batch"], c["heads"], s["max_new"], c["d"]
    G = c["heads_q"] // H
    cu, total = s["cu_q"].long(), s["kv_len"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device="cuda")
    row = (cu[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)              # [B, n]
    real = i < count[:, None]
    q = s["q"][row].float().view(B, n, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, d)
    k = _gathered(s["k"], s["k_scale"], s["pages"])
    score = (q @ k.transpose(-1, -2)).view(B, H, G, n, -1) * (1.0 / math.sqrt(d))
    del k
    j = torch.arange(score.shape[-1], device="cuda")
    p = (total - count)[:, None] + i                                         # [B, n]
    see = (j <= p[..., None]) & (j < total[:, None, None])
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top.isfinite(), top, 0.0)
    weight = (score - top).exp_()
    del score
    mass = weight.sum(dim=-1, keepdim=True)
    v = _gathered(s["v"], s["v_scale"], s["pages"])
    v = torch.where((j < total[:, None])[:, None, :, None], v, 0.0)
    o = (weight.view(B, H, G * n, -1) @ v).view(B, H, G, n, d) / torch.where(mass > 0, mass, 1.0)
    lse = (top + mass.log())[..., 0]
    at = row[real]
    out, out_lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], device="cuda")
    out[at] = o.permute(0, 3, 1, 2, 4)[real].reshape(-1, H * G, d).to(out.dtype)
    out_lse[at] = lse.permute(0, 3, 1, 2)[real].reshape(-1, H * G)
    return out, out_lse


# ------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        return _run_own(state)
    if c["op"] == "rope":
        turn = (state["positions"], state["freqs"], state["magnitude"], c["interleaved"])
        y = _rotate(state["x"], *turn).to(state["x"].dtype)
        if state["dy"] is None:
            return {"y": y}
        return {"y": y, "dx": _rotate(state["dy"], *turn, inverse=True).to(y.dtype)}
    if c["op"] == "append":
        q = _append(state)
        return _append_outputs(state, q)
    out, lse = _attention(state)
    return {"out": out, "lse": lse}


def _append_outputs(s, q):
    got = {"q": q, "k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        got.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return got


def _run_own(s):
    import comm_gemm_tile_gb300 as mk
    c = s["case"]
    if c["op"] == "rope":
        turn = dict(positions=s["positions"], magnitude=s["magnitude"], interleaved=c["interleaved"])
        y = mk.rope(s["x"], s["freqs"], **turn)
        if s["dy"] is None:
            return {"y": y}
        return {"y": y, "dx": mk.rope(s["dy"], s["freqs"], inverse=True, **turn)}
    cache = mk.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        q = mk.kv_append(cache, s["new_k"], s["new_v"], s["cu_q"], s["kv_len"], s["pages"], q=s["q"], freqs=s["freqs"],
                         magnitude=s["magnitude"], interleaved=c["interleaved"])
        return _append_outputs(s, q)
    out, lse = mk.paged_attention(s["q"], cache, s["cu_q"], s["kv_len"], s["pages"], window=c["window"],
                                  sinks=c["sinks"], max_q=s["max_new"], return_lse=True)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ what a pass cannot do without

def _visible(case, n, total):
    """(keys some new token sees, (token, key) pairs seen) of one sequence."""
    w, first, pairs = case["window"], total - n, 0
    if not w:
        return total, n * first + n * (n + 1) // 2
    for i in range(n):
        p = first + i
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(case["sinks"], lo)
    lo = max(0, first - w + 1)
    return total - lo + min(case["sinks"], lo), pairs


def work(case):
    size = 4 if case["type"] == "fp32" else 2
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["d"] * (2 if case["gradient"] else 1)
        return {"bytes": 2 * n * size + 8 * case["tokens"], "flops": 3 * n}
    new, total = _lengths(case)
    kv = 1 if case["cache"] == "e4m3" else size
    T = sum(new)
    if case["op"] == "append":
        rows_kv, rows_q = 2 * T * case["heads"] * case["d"], T * case["heads_q"] * case["d"]
        return {"bytes": rows_kv * (size + kv) + 2 * rows_q * size, "flops": 3 * (rows_q + rows_kv)}
    keys = pairs = 0
    for n, t in zip(new, total):
        k, p = _visible(case, n, t)
        keys, pairs = keys + k, pairs + p
    return {"bytes": 2 * keys * case["heads"] * case["d"] * kv + T * case["heads_q"] * (2 * case["d"] * size + 4),
            "flops": 4 * pairs * case["heads_q"] * case["d"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rotation(x, p, freqs, magnitude, interleaved, sign=1.0):
    """One token's heads [heads, d] at position p, or many tokens' with p a column, by complex products."""
    rot = 2 * freqs.numel()
    z = torch.polar(torch.full_like(p * freqs, magnitude), sign * p * freqs)
    x = x.double()
    head = x[..., :rot].unflatten(-1, (rot // 2, 2) if interleaved else (2, rot // 2))
    pair = torch.view_as_complex((head if interleaved else head.transpose(-1, -2)).contiguous())
    y = torch.view_as_real(pair * z)
    y = (y if interleaved else y.transpose(-1, -2)).flatten(-2)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _exact_append(s):
    c = s["case"]
    cu, total, size = s["cu_q"].tolist(), s["kv_len"].tolist(), c["page"]
    out = {"k": s["k"].double(), "v": s["v"].double()}
    scales = {"k": s["k_scale"], "v": s["v_scale"]}
    scales = {name: None if t is None else t.double() for name, t in scales.items()}
    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        start = total[b] - (cu[b + 1] - cu[b])
        p = torch.arange(start, total[b], dtype=torch.float64, device="cuda")[:, None, None]
        rows = slice(cu[b], cu[b + 1])
        turn = (p, s["freqs"], s["magnitude"], c["interleaved"])
        q[rows] = _exact_rotation(s["q"][rows], *turn)
        fresh = {"k": _exact_rotation(s["new_k"][rows], *turn), "v": s["new_v"][rows].double()}
        for which in range(start // size, -(-total[b] // size)):
            page = int(s["pages"][b, which])
            lo, hi = max(start, which * size), min(total[b], (which + 1) * size)
            for name in ("k", "v"):
                x = fresh[name][lo - start:hi - start].transpose(0, 1)                 # [heads, tokens, d]
                if scales[name] is None:
                    out[name][page, :, lo - which * size:hi - which * size] = x
                    continue
                need = torch.exp2(torch.ceil(torch.log2(x.abs().amax(dim=(1, 2)) / E4M3_MAX)).clamp_min(-100))
                if lo > which * size:
                    had = scales[name][page].clone()
                    need = torch.maximum(had, need)
                    out[name][page, :, :lo - which * size] *= (had / need)[:, None, None]
                scales[name][page] = need
                out[name][page, :, lo - which * size:hi - which * size] = x / need[:, None, None]
    got = {"q": q, "k": out["k"], "v": out["v"]}
    if scales["k"] is not None:
        got.update(k_scale=scales["k"], v_scale=scales["v"])
    return got


def _exact_attention(s):
    c = s["case"]
    cu, total, size = s["cu_q"].tolist(), s["kv_len"].tolist(), c["page"]
    G = c["heads_q"] // c["heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        n, L = cu[b + 1] - cu[b], total[b]
        if not n or not L:
            continue
        mine = s["pages"][b, :-(-L // size)].long()
        kv = []
        for t, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
            x = t[mine].double()
            if scale is not None:
                x = x * scale[mine].double()[..., None, None]
            kv.append(x.permute(1, 0, 2, 3).reshape(c["heads"], -1, c["d"])[:, :L])
        step = max(1, (1 << 28) // (L * c["heads_q"]))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            q = s["q"][cu[b] + lo:cu[b] + hi].double().view(hi - lo, c["heads"], G, c["d"])
            z = torch.einsum("nhgd,hkd->hgnk", q, kv[0]) / math.sqrt(c["d"])
            at = torch.arange(L - n + lo, L - n + hi, device="cuda")[:, None]
            key = torch.arange(L, device="cuda")[None, :]
            hidden = key > at
            if c["window"]:
                hidden |= (key <= at - c["window"]) & (key >= c["sinks"])
            z = z.masked_fill(hidden, -math.inf)
            lse[cu[b] + lo:cu[b] + hi] = torch.logsumexp(z, dim=-1).permute(2, 0, 1).flatten(1)
            o = torch.einsum("hgnk,hkd->nhgd", torch.softmax(z, dim=-1), kv[1])
            out[cu[b] + lo:cu[b] + hi] = o.flatten(1, 2)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        p = s["positions"].double()[:, None, None]
        turn = (p, s["freqs"], s["magnitude"], case["interleaved"])
        got = {"y": _exact_rotation(s["x"], *turn)}
        if s["dy"] is not None:
            got["dx"] = _exact_rotation(s["dy"], *turn, sign=-1.0)
        return got
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
