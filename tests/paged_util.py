"""Plain 64-bit implementations of the rotary, cache and paged attention operators, sequence by sequence, and the
inputs their tests share."""
import math

import torch

E4M3 = torch.float8_e4m3fn
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def rotate(x, positions, freqs, magnitude=1.0, interleaved=False, inverse=False):
    """x [tokens, heads, d] (any type) rotated, in float64 on the CPU."""
    x = x.detach().double().cpu()
    rot = 2 * freqs.numel()
    t = positions.double().cpu()[:, None, None] * freqs.double().cpu() * (-1.0 if inverse else 1.0)
    c, s = t.cos() * magnitude, t.sin() * magnitude
    y = x.clone()
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rotate_tolerance(x, positions, freqs, dtype, magnitude=1.0, interleaved=False, inverse=False):
    """Bound on |rope(x) - rotate(x)|: half a step of the output's type, and in the fp32 arithmetic the angle (half a
    step of a 24-bit fraction of a half turn: 2^-25 pi), sincospi (2 units in the last place), three roundings and
    the magnitude's two, each times the pair's magnitudes."""
    y = rotate(x, positions, freqs, magnitude, interleaved, inverse)
    size = rotate(x.abs(), torch.zeros_like(positions), freqs, abs(magnitude), interleaved)
    rot = 2 * freqs.numel()
    both = size.clone()
    if interleaved:
        pair = size[..., 0:rot:2] + size[..., 1:rot:2]
        both[..., 0:rot:2], both[..., 1:rot:2] = pair, pair
    else:
        pair = size[..., :rot // 2] + size[..., rot // 2:rot]
        both[..., :rot // 2], both[..., rot // 2:rot] = pair, pair
    fp32 = math.pi * 2.0 ** -25 + (4 + 5) * 2.0 ** -24
    tiny = torch.finfo(dtype).smallest_normal * 2.0 ** -8
    return y, HALF_STEP[dtype] * y.abs() + (1 + HALF_STEP[dtype]) * fp32 * both + tiny


class Batch:
    """Sequences with (new tokens, tokens in all) each, their pages in random order, as tensors on `device`."""

    def __init__(self, lengths, page, seed=0, device="cuda", spare=3, wide=1):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.page = lengths, page
        counts = [-(-max(t, 0) // page) for _, t in lengths]
        self.n_pages = sum(counts) + spare
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = []
        for c in counts:
            self.table.append(order[:c])
            order = order[c:]
        width = max(counts + [0]) + wide
        pages = torch.full((len(lengths), width), -7, dtype=torch.int32)   # entries past a sequence's end: nonsense
        for b, row in enumerate(self.table):
            pages[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        cu = [0]
        for n, _ in lengths:
            cu.append(cu[-1] + n)
        self.cu, self.tokens = cu, cu[-1]
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor([t for _, t in lengths], dtype=torch.int32, device=device)
        self.pages = pages.to(device)


def gather(cache, scale, table, length):
    """[heads, length, d] in float64: the tokens of one sequence out of a [pages, heads, slots, d] cache."""
    if length <= 0:
        return torch.zeros(cache.shape[1], 0, cache.shape[3], dtype=torch.float64)
    x = cache[table].detach().cpu().double() if cache.dtype != E4M3 else cache[table].detach().float().cpu().double()
    if scale is not None:
        x = x * scale[table].double().cpu()[:, :, None, None]
    return x.permute(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :length]


def attention(q, k, v, k_scale, v_scale, batch, scale=None, causal=True, window=0, sinks=0):
    """(out, lse, bound on |out error|, bound on |lse error|) in float64.

    The bounds count: half a step of q's type on the output and on every weight (relative, so 2^-b sum_j w_j |v_j|); the
    fp32 score, a sum of d products ((d + 8) 2^-24 sum |q k| scale, and the exponential's own few units), which moves
    each weight by that much, and the normalisation by as much again; and fp32 sums over the keys."""
    T, HQ, d = q.shape
    H = k.shape[1]
    G = HQ // H
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    step = HALF_STEP[q.dtype]
    out = torch.zeros(T, HQ, d, dtype=torch.float64)
    lse = torch.full((T, HQ), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros(T, HQ, dtype=torch.float64)
    qd = q.detach().double().cpu()
    for b, (n, length) in enumerate(batch.lengths):
        if n == 0 or length <= 0:
            continue
        rows = slice(batch.cu[b], batch.cu[b] + n)
        kk = gather(k, k_scale, batch.table[b], length)
        vv = gather(v, v_scale, batch.table[b], length)
        j = torch.arange(length)
        p = length - n + torch.arange(n)[:, None]
        see = (j <= p) if causal else torch.ones(n, length, dtype=torch.bool)
        if window:
            see = see & ((j > p - window) | (j < sinks))
        for h in range(HQ):
            K, V = kk[h // G], vv[h // G]
            z = (qd[rows, h] @ K.T) * scale
            e = ((qd[rows, h].abs() @ K.abs().T) * scale * (d + 8) * 2.0 ** -24 + z.abs() * 2.0 ** -22 + 2.0 ** -20)
            z = torch.where(see, z, -math.inf)
            e = torch.where(see, e, 0.0).amax(dim=1)
            some = see.any(dim=1)
            top = torch.where(some, z.amax(dim=1), 0.0)
            w = torch.where(see, (z - top[:, None]).exp(), 0.0)
            mass = w.sum(dim=1)
            w = w / torch.where(mass > 0, mass, 1.0)[:, None]
            # a token no row of the batch sees may hold NaN; one that some rows see is used where it is seen
            Vc = torch.where((see.any(dim=0))[:, None], V, 0.0)
            o = torch.where(some[:, None], w @ Vc, 0.0)
            size = w @ Vc.abs()
            out[rows, h] = o
            lse[rows, h] = torch.where(some, top + mass.log(), -math.inf)
            tol[rows, h] = step * o.abs() + size * (step + 2 * e[:, None] + length * 2.0 ** -24) * (1 + step) + 1e-30
            tol_lse[rows, h] = e + lse[rows, h].abs().nan_to_num(0, 0, 0) * 2.0 ** -22 + 2.0 ** -20
    return out, lse, tol, tol_lse


def random_cache(n_pages, heads, page, d, dtype, seed, order="heads", fill=float("nan"), device="cuda"):
    """(k, v, k_scale, v_scale) of random values, [pages, heads, slots, d] with the given memory order."""
    g = torch.Generator().manual_seed(seed)
    got = []
    for _ in range(2):
        x = torch.randn(n_pages, heads, page, d, generator=g)
        x = (x * 96).clamp(-448, 448).to(E4M3) if dtype == E4M3 else x.to(dtype)
        x = x.to(device)
        got.append(x.transpose(1, 2).contiguous().transpose(1, 2) if order == "tokens" else x)
    if dtype == E4M3:
        got += [torch.exp2(torch.randint(-9, -4, (n_pages, heads), generator=g).float()).to(device) for _ in range(2)]
    else:
        got += [None, None]
    return got


def poison(cache, scale, batch):
    """NaN in every slot that belongs to no token (the pages of no sequence, the slots past a sequence's end)."""
    held = torch.zeros(cache.shape[0], cache.shape[2], dtype=torch.bool)
    for table, (_, length) in zip(batch.table, batch.lengths):
        for i, page in enumerate(table):
            held[page, :max(0, min(batch.page, length - i * batch.page))] = True
    free = (~held)[:, None, :, None].expand(cache.shape).to(cache.device)
    if cache.dtype == E4M3:
        cache.view(torch.uint8).masked_fill_(free, 0x7f)
    else:
        cache.masked_fill_(free, float("nan"))
    if scale is not None:
        scale[(~held.any(dim=1)).to(scale.device)] = float("nan")


def e4m3_scale(amax):
    """The least power of two s >= 2^-100 with amax <= 448 s, by trying."""
    e = -100
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e
