"""Cases of the operators around a layer's products: the root-mean-square norm with its residual and 8-bit output, the
expert router with its losses, and products with 4-bit weights.

`listed()` gives fixed cases, `draw(rng)` one more of the same ranges, `prepare` the tensors a program holds before the
call, `run` one pass (the plain torch form, or the framework's calls where `own` is set), `work` the bytes and operations
of a pass, and `exact` the result in 64 bits.

Definitions.
  norm     h = x, or x + residual rounded to its type (the residual stream, an output); r = 1 / sqrt(mean(h^2) + eps);
           y = h r w.  8-bit output: a row's scale is max(amax / 448, 2^-100) and its codes are y / scale in e4m3.
           Gradient for dy (and dh, the stream's own): g = dy w, dx = r g - h r^3 mean(g h) + dh, dw = sum over rows dy h r
  route    p = softmax(logits); a token's experts are the top_k largest logits, ties to the lower number; its gates are
           scale * p of those (over their sum with normalize).  Masked tokens: experts -1, gates 0, counted nowhere.  With
           N other tokens: balance = experts * sum_e counts_e / (top_k N) * mean p_e, z = mean of logsumexp^2.  Gradient of
           sum(gates dgates) + db balance + dz z with respect to the logits (counts are constants)
  w4       y[m, n] = sum_k x[m, k] s[n, k / group] (code[n, k] - zero[n, k / group]); without zeros zero = 8.  Two codes a
           byte, the lower four bits first
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm before a layer of one decode step of 16 sequences: latency
        {"name": "norm step", "op": "norm", "rows": 16, "heads": 0, "n": 8192, "type": "bf16", "weight": "bf16",
         "residual": True, "out": "same", "gradient": False},
        # 8 shards of 1024 tokens, normalised into the 8-bit operand of an AllGather + GEMM with k = 8192
        {"name": "norm prompt e4m3", "op": "norm", "rows": 8192, "heads": 0, "n": 8192, "type": "bf16", "weight": "bf16",
         "residual": True, "out": "e4m3", "gradient": False},
        # a norm of every query and key head, out of a projection that holds the values too, with its gradient
        {"name": "norm heads", "op": "norm", "rows": 4099, "heads": 40, "n": 128, "type": "fp16", "weight": "fp16",
         "residual": False, "out": "same", "gradient": True},
        # a training step's 8 x 4096 tokens: the residual stream goes on and its gradient comes back
        {"name": "norm train", "op": "norm", "rows": 32768, "heads": 0, "n": 4096, "type": "bf16", "weight": "fp32",
         "residual": True, "out": "same", "gradient": True},
        # a decode step's tokens over 64 experts: latency
        {"name": "route step", "op": "route", "tokens": 16, "experts": 64, "top_k": 2, "type": "fp32", "normalize": True,
         "scale": 1.0, "mask": False, "gradient": False},
        # the 8 x 4096 tokens of the dispatch workload over its 64 experts, in training
        {"name": "route train", "op": "route", "tokens": 32768, "experts": 64, "top_k": 2, "type": "fp32",
         "normalize": True, "scale": 1.0, "mask": False, "gradient": True},
        # a padded batch of odd length with 16-bit logits (many ties) and gates that are not normalised
        {"name": "route padded", "op": "route", "tokens": 5003, "experts": 60, "top_k": 6, "type": "bf16",
         "normalize": False, "scale": 2.5, "mask": True, "gradient": False},
        # a long training batch over the most experts the dispatch takes
        {"name": "route many", "op": "route", "tokens": 131072, "experts": 256, "top_k": 8, "type": "fp32",
         "normalize": True, "scale": 2.5, "mask": True, "gradient": True},
        # one user's decode step: the up-projection of one rank's share of a layer (8192 to 3584)
        {"name": "w4 one", "op": "w4", "m": 1, "n": 3584, "k": 8192, "group": 128, "zeros": False, "type": "bf16"},
        # three users, small groups with zero points, odd sizes
        {"name": "w4 odd", "op": "w4", "m": 3, "n": 4097, "k": 1536, "group": 32, "zeros": True, "type": "fp16"},
        # a serving batch
        {"name": "w4 batch", "op": "w4", "m": 16, "n": 8192, "k": 8192, "group": 64, "zeros": True, "type": "bf16"},
        # the largest serving batch, a whole layer's projection
        {"name": "w4 many", "op": "w4", "m": 64, "n": 28672, "k": 8192, "group": 128, "zeros": False, "type": "fp16"},
    ]


def _between(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "w4"])
    if op == "norm":
        heads = rng.choice([0, 0, 0, rng.randint(1, 64)])
        if heads:
            n = rng.choice([64, 128, rng.randint(1, 256)])
            rows = _between(rng, 1, min(32768, (1 << 27) // (heads * n)))
        else:
            n = _between(rng, 1, 16384)
            if rng.random() < 0.6:
                n = max(64, n // 64 * 64)
            rows = _between(rng, 1, min(32768, (1 << 27) // n))
        kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        gradient = rng.random() < 0.5
        return {"op": op, "rows": rows if kind != "fp32" else max(1, rows // 2), "heads": heads, "n": n, "type": kind,
                "weight": rng.choice([kind, "fp32"]), "residual": rng.random() < 0.5,
                "out": "same" if gradient else rng.choice(["same", "e4m3"]), "gradient": gradient}
    if op == "route":
        experts = _between(rng, 2, 256)
        return {"op": op, "tokens": _between(rng, 1, 131072), "experts": experts,
                "top_k": rng.randint(1, min(8, experts)), "type": rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                "normalize": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]), "mask": rng.random() < 0.5,
                "gradient": rng.random() < 0.5}
    group = rng.choice([32, 64, 128])
    k = group * _between(rng, 1, 16384 // group)
    return {"op": op, "m": rng.choice([1, 1, rng.randint(2, 16), _between(rng, 1, 64)]), "n": _between(rng, 1, (1 << 27) // k)
            if k > 8192 else _between(rng, 1, 16384), "k": k, "group": group, "zeros": rng.random() < 0.5,
            "type": rng.choice(["bf16", "fp16"])}


# ------------------------------------------------------------------ inputs

def _normal(g, shape, dtype, size=1.0):
    return (torch.randn(shape, dtype=torch.float32, device="cuda", generator=g) * size).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]
    s = {"case": case}
    if case["op"] == "norm":
        n, heads = case["n"], case["heads"]
        if heads:                                   # the heads before the others of a projection's output
            s["x"] = _normal(g, (case["rows"], heads + 8, n), dtype, 2.0)[:, :heads]
        else:                                       # hidden states: channels of different sizes
            s["x"] = (torch.randn(case["rows"], n, device="cuda", generator=g)
                      * torch.exp(torch.randn(n, device="cuda", generator=g) * 0.5)).to(dtype)
        shape = s["x"].shape
        s["residual"] = _normal(g, shape, dtype, 3.0) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(n, device="cuda", generator=g)).to(TYPES[case["weight"]])
        if case["gradient"]:
            s["dy"] = _normal(g, shape, dtype)
            s["dh"] = _normal(g, shape, dtype) if case["residual"] else None
    elif case["op"] == "route":
        shape = (case["tokens"], case["experts"])
        bias = torch.randn(case["experts"], device="cuda", generator=g) * 0.5     # some experts are liked better
        s["logits"] = (torch.randn(shape, device="cuda", generator=g) * 1.5 + bias).to(dtype)
        s["mask"] = None
        if case["mask"]:                            # True: a real token; a tenth is padding
            s["mask"] = torch.rand(case["tokens"], device="cuda", generator=g) < 0.9
        if case["gradient"]:
            s["dgates"] = _normal(g, (case["tokens"], case["top_k"]), torch.float32)
            s["dbalance"] = torch.rand((), device="cuda", generator=g) * 0.02
            s["dz"] = torch.rand((), device="cuda", generator=g) * 0.002
    else:
        m, n, k, groups = case["m"], case["n"], case["k"], case["k"] // case["group"]
        s["x"] = _normal(g, (m, k), dtype)
        code = [(torch.randn((n, k // 2), device="cuda", generator=g) * 2.7 + 8.0).round_().clamp_(0, 15).to(torch.uint8)
                for _ in range(2)]
        s["codes"] = code[0] | (code[1] << 4)
        s["scales"] = ((0.5 + torch.rand((n, groups), device="cuda", generator=g)) * 0.3 * k ** -0.5).to(dtype)
        s["zeros"] = None
        if case["zeros"]:
            s["zeros"] = (8.0 + torch.randn((n, groups), device="cuda", generator=g)).to(dtype)
        if own:
            s["w"] = _handle(s)
    return s


def _handle(s):
    import comm_gemm_tile_gb300 as mk
    return mk.W4Weight(s["codes"], s["scales"], s["zeros"])


# ------------------------------------------------------------------ plain forms

def _norm(s):
    c = s["case"]
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(h.dtype)
    f = h.float()
    r = torch.rsqrt((f * f).mean(dim=-1, keepdim=True) + EPS)
    y = f * r * s["weight"].float()
    got = {}
    if c["out"] == "e4m3":
        scale = (y.abs().amax(dim=-1) / E4M3_MAX).clamp_min(2.0 ** -100)
        got["y"] = (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        got["scale"] = scale
    else:
        got["y"] = y.to(h.dtype)
    if s["residual"] is not None:
        got["h"] = h
    if c["gradient"]:
        dy = s["dy"].float()
        t = dy * f * r
        got["dw"] = t.flatten(0, -2).sum(dim=0, dtype=torch.float64).to(s["weight"].dtype)
        dot = (t * s["weight"].float()).mean(dim=-1, keepdim=True)
        dx = r * (dy * s["weight"].float() - f * r * dot)
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        got["dx"] = dx.to(h.dtype)
    return got


def _route(s):
    c = s["case"]
    E, K = c["experts"], c["top_k"]
    logits = s["logits"].float()
    idx = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :K]
    top = logits.amax(dim=-1, keepdim=True)
    e = (logits - top).exp()
    mass = e.sum(dim=-1, keepdim=True)
    p = e / mass
    lse = (top + mass.log())[:, 0]
    real = torch.ones(c["tokens"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    chosen = p.gather(1, idx)
    share = chosen / chosen.sum(dim=-1, keepdim=True) if c["normalize"] else chosen
    gates = torch.where(real[:, None], share * c["scale"], 0.0)
    N = real.sum().clamp_min(1)
    hit = torch.zeros(E, dtype=torch.int64, device="cuda")
    counts = hit.index_add(0, idx.flatten(), real[:, None].expand(-1, K).flatten().long())
    f = counts.double() / (K * N)
    mean_p = torch.where(real[:, None], p, 0.0).sum(dim=0, dtype=torch.float64) / N
    got = {"topk_idx": torch.where(real[:, None], idx, -1).int(), "gates": gates, "counts": counts.int(),
           "balance_loss": (E * (f * mean_p).sum()).float(),
           "z_loss": (torch.where(real, lse * lse, 0.0).sum(dtype=torch.float64) / N).float()}
    if c["gradient"]:
        dg = s["dgates"] * c["scale"]
        dot = (share * dg).sum(dim=-1, keepdim=True)
        if c["normalize"]:
            d = torch.zeros_like(p).scatter(1, idx, share * (dg - dot))
        else:
            d = torch.zeros_like(p).scatter(1, idx, chosen * dg) - p * dot
        ff = f.float()
        d = d + s["dbalance"] * (E / N) * p * (ff - (p * ff).sum(dim=-1, keepdim=True))
        d = d + s["dz"] * (2.0 / N) * lse[:, None] * p
        got["dlogits"] = torch.where(real[:, None], d, 0.0).to(s["logits"].dtype)
    return got


def _w4(s):
    c = s["case"]
    code = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=-1).view(c["n"], -1, c["group"]).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = ((code - zero) * s["scales"].float()[..., None]).flatten(1)
    return {"y": (s["x"].float() @ w.t()).to(s["x"].dtype)}


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "route": _route, "w4": _w4}[state["case"]["op"]](state)


def _run_own(s):
    import comm_gemm_tile_gb300 as mk
    c = s["case"]
    if c["op"] == "norm":
        got = {}
        made = mk.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS,
                           out_dtype=E4M3 if c["out"] == "e4m3" else None)
        names = ["y"] + ["scale"] * (c["out"] == "e4m3") + ["h"] * (s["residual"] is not None)
        got.update(zip(names, made if len(names) > 1 else (made,)))
        if c["gradient"]:
            dx, dw = mk.rms_norm_backward(s["dy"], got.get("h", s["x"]), s["weight"], dh=s["dh"], eps=EPS)
            got.update(dw=dw, dx=dx)
        return got
    if c["op"] == "route":
        how = dict(normalize=c["normalize"], scale=c["scale"])
        got = mk.moe_route(s["logits"], c["top_k"], mask=s["mask"], **how)
        out = {name: got[name] for name in ("topk_idx", "gates", "counts", "balance_loss", "z_loss")}
        if c["gradient"]:
            out["dlogits"] = mk.moe_route_backward(s["logits"], got, s["dgates"], s["dbalance"], s["dz"], **how)
        return out
    return {"y": mk.w4_gemm(s["x"], s["w"] if "w" in s else _handle(s))}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    size = 4 if case["type"] == "fp32" else 2
    if case["op"] == "norm":
        rows = case["rows"] * max(1, case["heads"])
        total = rows * case["n"]
        weight = case["n"] * (4 if case["weight"] == "fp32" else 2)
        b = total * (3 if case["residual"] else 1) * size + weight
        b += total + 4 * rows if case["out"] == "e4m3" else total * size
        if case["gradient"]:
            b += total * size * (3 if case["residual"] else 2) + weight
        return {"bytes": b, "flops": total * (16 if case["gradient"] else 5)}
    if case["op"] == "route":
        T, E, K = case["tokens"], case["experts"], case["top_k"]
        b = T * (E * size + 8 * K + (1 if case["mask"] else 0)) + 4 * E
        if case["gradient"]:
            b += T * (E * size + 4 * K)
        return {"bytes": b, "flops": T * E * (10 if case["gradient"] else 4)}
    m, n, k = case["m"], case["n"], case["k"]
    groups = n * (k // case["group"]) * (2 if case["zeros"] else 1)
    return {"bytes": n * k // 2 + 2 * groups + 2 * m * (n + k), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_norm(s):
    c = s["case"]
    h = s["x"].double()
    got = {}
    if s["residual"] is not None:
        h = (h + s["residual"].double()).to(s["x"].dtype).double()      # the stream holds values of its type
    w = s["weight"].double()
    size = (h.square().sum(dim=-1, keepdim=True) / c["n"] + EPS).sqrt()
    unit = h / size
    y = unit * w
    if c["out"] == "e4m3":
        got["scale"] = torch.maximum(y.abs().amax(dim=-1) / E4M3_MAX, torch.full((), 2.0 ** -100, device="cuda").double())
        y = y / got["scale"][..., None]
    got["y"] = y
    if s["residual"] is not None:
        got["h"] = h
    if c["gradient"]:
        # y_i = w_i h_i / size: dy_i/dh_j = w_i (delta_ij - unit_i unit_j / n) / size
        g = s["dy"].double() * w
        got["dx"] = (g - unit * (g * unit).sum(dim=-1, keepdim=True) / c["n"]) / size
        if s["dh"] is not None:
            got["dx"] = got["dx"] + s["dh"].double()
        got["dw"] = torch.einsum("ri,ri->i", s["dy"].double().flatten(0, -2), unit.flatten(0, -2))
    order = ["y"] + ["scale"] * (c["out"] == "e4m3") + ["h"] * (s["residual"] is not None)
    return {name: got[name] for name in order + ["dw", "dx"] * c["gradient"]}


def _exact_route(s):
    c = s["case"]
    T, E, K = c["tokens"], c["experts"], c["top_k"]
    z = s["logits"].double()
    real = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    rest, picks = z.clone(), []
    for _ in range(K):                              # the largest that is left, the first of equal ones
        best = rest.amax(dim=-1, keepdim=True)
        first = torch.where(rest == best, torch.arange(E, device="cuda"), E).amin(dim=-1, keepdim=True)
        picks.append(first)
        rest.scatter_(1, first, -math.inf)
    idx = torch.cat(picks, dim=1)
    lse = torch.logsumexp(z, dim=-1)
    p = torch.softmax(z, dim=-1)
    mine = z.gather(1, idx)
    share = torch.softmax(mine, dim=-1) if c["normalize"] else (mine - lse[:, None]).exp()
    counts = torch.bincount(idx[real].flatten(), minlength=E)
    N = max(1, int(real.sum()))
    f = counts.double() / (K * N)
    got = {"topk_idx": idx.masked_fill(~real[:, None], -1).int(), "gates": (share * c["scale"]).masked_fill(~real[:, None], 0.0),
           "counts": counts.int(), "balance_loss": E * (p[real] @ f).sum() / N, "z_loss": lse[real].square().sum() / N}
    if c["gradient"]:
        dp = (s["dbalance"].double() * E / N * f).expand(T, E).clone()     # with respect to p
        dl = torch.zeros_like(z)
        v = s["dgates"].double() * c["scale"]
        if c["normalize"]:                          # softmax over the chosen logits alone
            dl.scatter_add_(1, idx, share * (v - (share * v).sum(dim=-1, keepdim=True)))
        else:
            dp.scatter_add_(1, idx, v)
        dl += p * (dp - (p * dp).sum(dim=-1, keepdim=True))
        dl += s["dz"].double() * 2.0 / N * lse[:, None] * p
        got["dlogits"] = dl.masked_fill(~real[:, None], 0.0)
    return got


def _exact_w4(s):
    c = s["case"]
    y = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for g in range(c["k"] // c["group"]):           # group by group: (codes - zero) in whole numbers times the scale
        at = slice(g * c["group"], (g + 1) * c["group"])
        b = s["codes"][:, at.start // 2:at.stop // 2]
        part = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device="cuda")
        part += x[:, at][:, 0::2] @ (b % 16).double().t()
        part += x[:, at][:, 1::2] @ (b // 16).double().t()
        zero = 8.0 if s["zeros"] is None else s["zeros"][:, g].double()
        y += (part - x[:, at].sum(dim=-1, keepdim=True) * zero) * s["scales"][:, g].double()
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "w4": _exact_w4}[case["op"]](s)
