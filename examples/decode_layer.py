"""A decoder layer in decode: attention and experts, with 4-bit projections.  A call of the layer is

    rms_norm (the residual stream goes on)
    -> w4_gemm (queries, keys, values) -> kv_append -> paged_attention -> w4_gemm
    -> rms_norm, which adds to the stream -> router logits -> moe_route -> moe_dispatch_gemm -> SiLU -> moe_combine
    -> rms_norm, which adds to the stream (that of the next layer)

for prompts of several sequences in one call, then decode steps.  Tokens are padded to whole ranks; the router leaves the
padding out.  `python examples/decode_layer.py` runs it on one GPU, compares each step with the layer in 64 bits (with the
experts that were chosen), and prints the largest error, the experts' load and the time of a decode step.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import comm_gemm_tile_gb300 as mk
from serve_attention import Pages


class DecoderLayer:
    def __init__(self, ranks=2, hidden=512, heads_q=8, heads=4, d=64, experts=8, topk=2, ffn=256, pages=64, page=16,
                 group=64, symmetric=True, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        draw = lambda *shape: torch.randn(*shape, generator=g) * shape[-1] ** -0.5   # noqa: E731
        self.ranks, self.hq, self.hk, self.d = ranks, heads_q, heads, d
        self.experts, self.topk = experts, topk
        pack = lambda w: mk.W4Weight.quantize(w.to(device), group=group, symmetric=symmetric)   # noqa: E731
        self.w_qkv, self.w_o = pack(draw((heads_q + 2 * heads) * d, hidden)), pack(draw(hidden, heads_q * d))
        self.norms = [(1.0 + 0.1 * torch.randn(hidden, generator=g)).to(device) for _ in range(3)]
        self.w_router = draw(experts, hidden).to(device)
        local = experts // ranks
        self.w_up = [(torch.randn(local, hidden, ffn, generator=g) * hidden ** -0.5).bfloat16().to(device) for _ in range(ranks)]
        self.w_down = [(torch.randn(local, ffn, hidden, generator=g) * ffn ** -0.5).bfloat16().to(device) for _ in range(ranks)]
        self.freqs, self.magnitude = mk.rope_freqs(d, device=device)
        self.cache = mk.KVCache.empty(pages, heads, page, d, torch.bfloat16, device)

    def __call__(self, x, stream, cu_q, kv_len, pages, max_q):
        """x: [tokens x hidden], what the layer before adds to the stream.  Returns (the next layer's
        normalised input, the stream, the route)."""
        n, stream = mk.rms_norm(x, self.norms[0], residual=stream)
        qkv = mk.w4_gemm(n, self.w_qkv).view(n.shape[0], -1, self.d)
        q, k, v = qkv.split([self.hq, self.hk, self.hk], dim=1)
        q = mk.kv_append(self.cache, k, v, cu_q, kv_len, pages, q=q, freqs=self.freqs, magnitude=self.magnitude)
        o = mk.paged_attention(q, self.cache, cu_q, kv_len, pages, max_q=max_q)
        n, stream = mk.rms_norm(mk.w4_gemm(o.flatten(1), self.w_o), self.norms[1], residual=stream, h_out=stream)
        y, route = self.experts_of(n)
        y, stream = mk.rms_norm(y, self.norms[2], residual=stream, h_out=stream)
        return y, stream, route

    def experts_of(self, n):
        R, tokens = self.ranks, n.shape[0]
        T = -(-tokens // R)
        padded = torch.zeros(R * T, n.shape[1], dtype=n.dtype, device=n.device)
        padded[:tokens] = n
        logits = padded.float() @ self.w_router.t()
        mask = torch.arange(R * T, device=n.device) < tokens
        route = mk.moe_route(logits, self.topk, mask=mask)
        # (clones: the shares of a rank start on whole 16-byte pieces)
        sent = mk.moe_dispatch_gemm(list(padded.view(R, T, -1)), [t.clone() for t in logits.view(R, T, -1)], self.w_up,
                                    E_loc=self.experts // R, topk=self.topk)
        h = [torch.nn.functional.silu(t) for t in sent["y"]]
        back = mk.moe_combine(h, self.w_down, [t.clone() for t in route["gates"].view(R, T, -1)], sent["recv_src"],
                              sent["counts"], E_loc=self.experts // R, topk=self.topk)
        return torch.cat(back["out"])[:tokens], route


def _norm(h, w):
    return h * (h.square().mean(dim=-1, keepdim=True) + 1e-6).rsqrt() * w.double()


def plain(layer, x, chosen):
    """(normalised output, stream) of one sequence with all its tokens x (the stream is empty before), in 64 bits, with
    the experts chosen [tokens x topk]."""
    n, d = x.shape[0], layer.d
    stream = x.double()
    turn = torch.arange(n, device=x.device).double()[:, None, None] * layer.freqs.double()

    def rotate(t):
        a, b = t.chunk(2, dim=-1)
        return torch.cat([a * turn.cos() - b * turn.sin(), b * turn.cos() + a * turn.sin()], dim=-1) * layer.magnitude

    qkv = (_norm(stream, layer.norms[0]) @ layer.w_qkv.dequantize(torch.float64).t()).view(n, -1, d)
    q, k, v = qkv.split([layer.hq, layer.hk, layer.hk], dim=1)
    q, k = rotate(q), rotate(k)
    k, v = (t.repeat_interleave(layer.hq // layer.hk, dim=1) for t in (k, v))
    z = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
    z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    o = torch.einsum("hij,jhd->ihd", z.softmax(dim=-1), v).flatten(1)
    stream = stream + o @ layer.w_o.dequantize(torch.float64).t()
    y = _norm(stream, layer.norms[1])
    gates = torch.softmax((y @ layer.w_router.double().t()).gather(1, chosen), dim=-1)
    up, down = torch.cat(layer.w_up).double(), torch.cat(layer.w_down).double()
    for s in range(layer.topk):
        e = chosen[:, s]
        h = torch.nn.functional.silu(torch.einsum("ti,tij->tj", y, up[e]))
        stream = stream + gates[:, s, None] * torch.einsum("tj,tji->ti", h, down[e])
    return _norm(stream, layer.norms[2]), stream


def run(prompts=(60, 33, 1), steps=8, symmetric=True, group=64, hidden=512, seed=1):
    """(largest error of any step's stream over its root mean square, tokens of each expert, seconds of a decode step)."""
    layer = DecoderLayer(hidden=hidden, symmetric=symmetric, group=group)
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(n + steps, hidden, generator=g).bfloat16().cuda() for n in prompts]
    pool, at = Pages(len(prompts), 64, 16), [0] * len(prompts)
    got, chosen, load = [[] for _ in prompts], [[] for _ in prompts], 0
    t0 = 0.0
    for i, new in enumerate([list(prompts)] + [[1] * len(prompts)] * steps):
        if i == 1 + steps // 2:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
        batch = pool.grow(new)
        now = torch.cat([t[a:a + n] for t, a, n in zip(x, at, new)])
        _, stream, route = layer(now, torch.zeros_like(now), *batch, max_q=max(new))
        at = [a + n for a, n in zip(at, new)]
        load = load + route["counts"]
        for b, (s, c) in enumerate(zip(stream.split(new), route["topk_idx"][:sum(new)].split(new))):
            got[b].append(s)
            chosen[b].append(c.long())
    torch.cuda.synchronize()
    seconds = (time.perf_counter() - t0) / max(1, steps - steps // 2)
    status, detail = mk.device_status()
    if status != mk.MK_OK:
        raise RuntimeError(f"device status {mk.status_string(status)} ({detail})")
    worst = 0.0
    for t, s, c in zip(x, got, chosen):
        _, want = plain(layer, t, torch.cat(c))
        worst = max(worst, float((torch.cat(s).double() - want).abs().max() / want.square().mean().sqrt()))
    return worst, load, seconds


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--zeros", action="store_true", help="4-bit weights with zero points")
    a = ap.parse_args()
    error, load, seconds = run(symmetric=not a.zeros)
    print(f"largest error / rms {error:.4f}, tokens of each expert {load.tolist()}, decode step {seconds * 1e3:.2f} ms")
