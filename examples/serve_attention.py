"""A tensor-parallel attention layer served from a paged cache: prompts of several sequences in one call, then decode
steps.  Every virtual rank has its share of the heads and a cache of its own; a call of the layer is

    projections -> kv_append (positions, rotation, the cache) -> paged_attention, for every rank -> gemm_ar

`python examples/serve_attention.py [--cache e4m3]` runs it on one GPU, compares each step with plain 64-bit attention
over everything the sequences have seen, and prints the largest error and the time of a decode step.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import comm_gemm_tile_gb300 as mk


class AttentionLayer:
    def __init__(self, ranks=2, hidden=512, heads_q=8, heads=4, d=64, window=0, sinks=0, pages=64, page=16, cache="bf16",
                 device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        draw = lambda *shape: (torch.randn(*shape, generator=g) * shape[0] ** -0.5).bfloat16().to(device)
        self.ranks, self.d, self.window, self.sinks = ranks, d, window, sinks
        self.hq, self.hk = heads_q // ranks, heads // ranks
        self.w_qkv = [draw(hidden, (self.hq + 2 * self.hk) * d) for _ in range(ranks)]
        self.w_o = [draw(self.hq * d, hidden) for _ in range(ranks)]
        self.freqs, self.magnitude = mk.rope_freqs(d, device=device)
        dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
        self.caches = [mk.KVCache.empty(pages, self.hk, page, d, dtype, device) for _ in range(ranks)]

    def __call__(self, x, cu_q, kv_len, pages, max_q):
        """x: [tokens x hidden], the new tokens of every sequence, which kv_len already counts."""
        heads = []
        for w, cache in zip(self.w_qkv, self.caches):
            q, k, v = (x @ w).view(x.shape[0], -1, self.d).split([self.hq, self.hk, self.hk], dim=1)
            q = mk.kv_append(cache, k, v, cu_q, kv_len, pages, q=q, freqs=self.freqs,
                             magnitude=self.magnitude)
            o = mk.paged_attention(q, cache, cu_q, kv_len, pages, window=self.window, sinks=self.sinks, max_q=max_q)
            heads.append(o.flatten(1))
        return mk.gemm_ar(heads, self.w_o)[0]


class Pages:
    """Hands pages to sequences as they grow."""

    def __init__(self, sequences, pages, page):
        self.free, self.page = list(range(pages)), page
        self.table = torch.full((sequences, pages), -1, dtype=torch.int32)
        self.length = [0] * sequences

    def grow(self, new):
        """(cu_q, kv_len, pages) on the GPU for a call that adds new[b] tokens to sequence b."""
        for b, n in enumerate(new):
            have, self.length[b] = -(-self.length[b] // self.page), self.length[b] + n
            for i in range(have, -(-self.length[b] // self.page)):
                self.table[b, i] = self.free.pop()
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0, dtype=torch.int32)
        return cu.cuda(), torch.tensor(self.length, dtype=torch.int32).cuda(), self.table.cuda()


def plain(layer, x):
    """The layer for one sequence with all its tokens x, in 64 bits."""
    n, out = x.shape[0], 0
    p = torch.arange(n, device=x.device)
    turn = p.double()[:, None, None] * layer.freqs.double()
    see = p[None, :] <= p[:, None]
    if layer.window:
        see &= (p[:, None] - p[None, :] < layer.window) | (p[None, :] < layer.sinks)

    def rotate(t):
        a, b = t.chunk(2, dim=-1)
        return torch.cat([a * turn.cos() - b * turn.sin(), b * turn.cos() + a * turn.sin()], dim=-1) * layer.magnitude

    for w_qkv, w_o in zip(layer.w_qkv, layer.w_o):
        qkv = (x @ w_qkv).double().view(n, -1, layer.d)
        q, k, v = qkv.split([layer.hq, layer.hk, layer.hk], dim=1)
        q, k = rotate(q), rotate(k)
        k, v = (t.repeat_interleave(layer.hq // layer.hk, dim=1) for t in (k, v))
        z = torch.einsum("ihd,jhd->hij", q, k) * layer.d ** -0.5
        o = torch.einsum("hij,jhd->ihd", z.masked_fill(~see, float("-inf")).softmax(dim=-1), v)
        out = out + o.flatten(1) @ w_o.double()
    return out


def run(prompts=(300, 77, 1), steps=20, cache="bf16", window=0, sinks=0, pages=64, page=16, hidden=512, seed=1):
    """(largest error of any step over the root mean square of the outputs, seconds of a decode step)."""
    layer = AttentionLayer(hidden=hidden, window=window, sinks=sinks, pages=pages, page=page, cache=cache)
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(n + steps, hidden, generator=g).bfloat16().cuda() for n in prompts]
    want = [plain(layer, t) for t in x]
    pool, at, worst = Pages(len(prompts), pages, page), [0] * len(prompts), 0.0
    calls, t0 = [list(prompts)] + [[1] * len(prompts)] * steps, 0.0
    for i, new in enumerate(calls):
        if i == len(calls) - steps // 2:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        batch = pool.grow(new)
        y = layer(torch.cat([t[a:a + n] for t, a, n in zip(x, at, new)]), *batch, max_q=max(new))
        at = [a + n for a, n in zip(at, new)]
        for t, a, n, part in zip(want, at, new, y.split(new)):
            worst = max(worst, float((part.double() - t[a - n:a]).abs().max() / t.square().mean().sqrt()))
    torch.cuda.synchronize()
    seconds = (time.perf_counter() - t0) / max(1, steps // 2)
    status, detail = mk.device_status()
    if status != mk.MK_OK:
        raise RuntimeError(f"device status {mk.status_string(status)} ({detail})")
    return worst, seconds


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    a = ap.parse_args()
    error, seconds = run(cache=a.cache, window=a.window, sinks=a.sinks)
    print(f"largest error / rms {error:.4f}, decode step {seconds * 1e3:.2f} ms (with the comparison)")
