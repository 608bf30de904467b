"""The operators around the products and the logits, as cases to be measured.

Three kinds: layer norm over rows or heads (forward, and backward with the
gradients of weight and bias); rotary positions on queries and keys, forward
and backward; and the router of a mixture-of-experts layer (its choices, the
rows grouped by expert, the balance and z losses, and its gradient).

``run`` computes them in a plain form (elementary torch operations in 32 or
64 bits) unless ``own`` is true; then it calls the library.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6
BALANCE, Z = 1e-2, 1e-3  # coefficients of the two losses in the router's gradient

_library = None


def _lib():
    """The package and one handle for the process, as a program keeps them."""
    global _library
    if _library is None:
        import muon_step_02_amd as mu
        _library = (mu, mu.muon_init(0))
    return _library


# ------------------------------------------------------------------ cases ----

def _norm(name, op, tokens, heads, cols, pad, center, dtype, weight, add=False):
    """Rows of `cols` values: `heads` a token, `pad` values between two tokens'
    rows.  `center`: the mean is taken off, and there is a bias.  `weight`: the
    type of weight and bias and of their gradients; `add`: these accumulate."""
    return {"name": name, "op": op, "tokens": tokens, "heads": heads, "cols": cols, "pad": pad,
            "center": center, "dtype": dtype, "weight": weight, "add": add}


def _rotary(name, back, tokens, sequences, start, heads, kv_heads, head_dim, first, pairs, interleaved,
            scaling, dtype):
    """Queries and keys of `sequences` packed sequences, each from position
    `start` on; `pairs` pairs of every head from its element `first` on turn."""
    return {"name": name, "op": "rotary", "back": back, "tokens": tokens, "sequences": sequences,
            "start": start, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "first": first,
            "pairs": pairs, "interleaved": interleaved, "scaling": scaling, "dtype": dtype}


def _router(name, op, tokens, padded, experts, masked, top_k, renormalize, dtype):
    """`padded` of the tokens have no logits (all -inf); every other token is
    kept from `masked` of the experts."""
    return {"name": name, "op": op, "tokens": tokens, "padded": padded, "experts": experts,
            "masked": masked, "top_k": top_k, "renormalize": renormalize, "dtype": dtype}


def listed():
    return [
        # eight tokens at a time into the d=7168 layer: latency
        _norm("norm, 8 rows of 7168", "norm", 8, 1, 7168, 0, False, "bf16", "bf16"),
        # a training batch into a d=4096 layer
        _norm("norm, 16384 rows of 4096", "norm", 16384, 1, 4096, 0, True, "bf16", "f32"),
        # the query heads of a fused projection (32 heads, 8 key and 8 value heads)
        _norm("norm, 32 heads of 4099 tokens", "norm", 4099, 32, 128, 2048, False, "bf16", "bf16"),
        # a small fp32 layer of odd width on its way back
        _norm("norm grad, 777 rows of 1001", "norm_grad", 777, 1, 1001, 0, True, "f32", "f32"),
        # the d=7168 layer on its way back, gradients added up over micro-batches
        _norm("norm grad, 16384 rows of 7168", "norm_grad", 16384, 1, 7168, 0, True, "bf16", "f32", True),
        # 16 sequences that each get one token far into their context: latency
        _rotary("rotary, 16 tokens", False, 16, 16, 100000, 64, 8, 128, 0, 64, False, "parts", "bf16"),
        # a training batch of packed sequences with shared key heads
        _rotary("rotary, 32768 tokens", False, 32768, 16, 0, 32, 8, 128, 0, 64, False, "none", "bf16"),
        # the last third of each head in neighbouring pairs, on its way back
        _rotary("rotary back, part of 64 heads", True, 4099, 3, 0, 64, 64, 192, 128, 32, True, "linear", "f32"),
        # eight tokens of eight sequences at the router of the 64-expert layer
        _router("router, 64 tokens", "router", 64, 0, 64, 0, 8, False, "bf16"),
        # a padded training batch at a router of many experts
        _router("router, 32768 tokens", "router", 32768, 512, 256, 0, 8, True, "f32"),
        # a small router of an odd number of experts, some out of reach, on its way back
        _router("router grad, 4099 tokens", "router_grad", 4099, 99, 61, 7, 3, True, "f32"),
        # the 64-expert layer's router on its way back
        _router("router grad, 32768 tokens", "router_grad", 32768, 0, 64, 0, 8, False, "bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width: mostly a multiple of 8 (or 64), at times any number."""
    n = _log(rng, low, high)
    step = rng.choice((1, 8, 8, 64, 64, 64))
    return max(low, n // step * step)


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "rotary", "rotary", "router", "router_grad"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("norm", "norm_grad"):
        heads = rng.choice((1, 1, 8, 32))
        cols = _width(rng, 33, 16384) if heads == 1 else rng.choice((64, 80, 128, 192))
        most = (6e7 if dtype == "bf16" else 3e7) / (heads * cols)
        return {"op": op, "tokens": _log(rng, 1, max(2, min(65536, most))), "heads": heads, "cols": cols,
                "pad": rng.choice((0, 0, 8, 3, 1024)), "center": rng.random() < 0.6, "dtype": dtype,
                "weight": rng.choice(("f32", dtype)), "add": op == "norm_grad" and rng.random() < 0.3}
    if op == "rotary":
        heads = rng.choice(((8, 8), (16, 4), (32, 8), (24, 24), (64, 1)))
        dim, first, pairs = rng.choice(((64, 0, 32), (128, 0, 64), (128, 0, 32), (192, 128, 32), (80, 0, 40),
                                        (100, 3, 17)))
        most = (7e7 if dtype == "bf16" else 3e7) / (sum(heads) * dim)
        tokens = _log(rng, 1, min(32768, most))
        return {"op": op, "back": rng.random() < 0.5, "tokens": tokens,
                "sequences": _log(rng, 1, min(33, tokens)), "start": rng.choice((0, 0, 0, 5000, 1000000)),
                "heads": heads[0], "kv_heads": heads[1], "head_dim": dim, "first": first, "pairs": pairs,
                "interleaved": rng.random() < 0.5, "scaling": rng.choice(("none", "linear", "base", "parts")),
                "dtype": dtype}
    experts = _log(rng, 2, 512)
    masked = rng.choice((0, 0, 1, experts // 3))
    tokens = _log(rng, 1, min(32768, 8e6 / experts))
    return {"op": op, "tokens": tokens, "padded": rng.choice((0, 0, tokens // 7)), "experts": experts,
            "masked": masked, "top_k": rng.randint(1, min(12, experts)), "renormalize": rng.random() < 0.5,
            "dtype": dtype}


# ----------------------------------------------------------------- inputs ----

def _randn(gen, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype) * std


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device=DEV)


def _rows(gen, case, std):
    """(tokens, heads, cols) values with `pad` values behind every token's."""
    T, H, C = case["tokens"], case["heads"], case["cols"]
    flat = _randn(gen, T, H * C + case["pad"], dtype=DTYPES[case["dtype"]], std=std)
    return flat[:, :H * C].view(T, H, C)


def _prepare_norm(case, gen):
    T, H, C = case["tokens"], case["heads"], case["cols"]
    x, wide = _rows(gen, case, 1.0), DTYPES[case["weight"]]
    # rows differ in scale and offset, a few columns stand out
    x.mul_((0.2 + 3.0 * _uniform(gen, T, H, 1)).to(x.dtype)).add_(_randn(gen, T, H, 1, dtype=x.dtype, std=0.3))
    x[:, :, ::61] *= 6.0
    s = {"op": case["op"], "center": case["center"], "x": x, "add": case["add"],
         "w": (1.0 + 0.2 * _randn(gen, C)).to(wide), "b": (0.1 * _randn(gen, C)).to(wide) if case["center"] else None,
         "y": torch.zeros(T, H, C, device=DEV, dtype=x.dtype)}
    if case["op"] == "norm":
        s["mean"] = torch.zeros(T, H, device=DEV) if case["center"] else None
        s["rstd"] = torch.zeros(T, H, device=DEV)
    else:
        wide_x = x.double()
        mean = wide_x.mean(2, keepdim=True) if case["center"] else torch.zeros_like(wide_x[:, :, :1])
        s["rstd"] = ((wide_x - mean).square().mean(2) + EPS).rsqrt().float()
        s["mean"] = mean[:, :, 0].float() if case["center"] else None
        s["dy"] = _rows(gen, case, 1e-2)
        s["dw"] = torch.zeros(C, device=DEV, dtype=wide)
        s["db"] = torch.zeros(C, device=DEV, dtype=wide) if case["center"] else None
        if case["add"]:
            s["dw"].normal_(generator=gen).mul_(1e-2)
    if own and case["op"] == "norm_grad":
        mu, h = _lib()
        s["workspace"] = torch.empty(mu.muon_layernorm_workspace_size(h, x), dtype=torch.uint8, device=DEV)
    return s


def _lengths(case):
    """Lengths of the packed sequences: of the case alone, no two runs differ."""
    r = random.Random("%d %d" % (case["sequences"], case["tokens"]))
    w = [r.expovariate(1.0) + 0.05 for _ in range(case["sequences"])]
    left = case["tokens"] - case["sequences"]
    n = [1 + int(left * x / sum(w)) for x in w]
    n[0] += case["tokens"] - sum(n)
    return n


SCALING = {"none": {}, "linear": {"factor": 4.0}, "base": {"factor": 8.0},
           "parts": {"factor": 32.0, "context": 8192.0, "low": 1.0, "high": 32.0}}


def _frequencies(pairs, scaling):
    """Radians a position of every pair, scaled for contexts `factor` longer."""
    s = SCALING[scaling]
    base = 10000.0
    if scaling == "base":  # the last pair's frequency falls by the factor
        base *= s["factor"] ** (pairs / (pairs - 1.0))
    f = torch.tensor([base ** (-i / pairs) for i in range(pairs)], dtype=torch.float64)
    if scaling == "linear":
        f /= s["factor"]
    if scaling == "parts":  # by the turns a pair makes over the context
        keep = ((s["context"] * f / (2.0 * math.pi) - s["low"]) / (s["high"] - s["low"])).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / s["factor"])
    return f


def _prepare_rotary(case, gen):
    T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
    dtype = DTYPES[case["dtype"]]
    flat = _randn(gen, T, H + 2 * K, D, dtype=dtype)  # with the values that do not turn
    at = [case["start"] + i for n in _lengths(case) for i in range(n)]
    s = {"op": "rotary", "back": case["back"], "x": [flat[:, :H], flat[:, H:H + K]],
         "y": [torch.zeros(T, n, D, device=DEV, dtype=dtype) for n in (H, K)],
         "positions": torch.tensor(at, dtype=torch.int32, device=DEV),
         "first": case["first"], "pairs": case["pairs"], "interleaved": case["interleaved"],
         "scale": 0.1 * math.log(32.0) + 1.0 if case["scaling"] == "parts" else 1.0}
    if own:
        mu, _ = _lib()
        f = mu.muon_rotary_frequencies(case["pairs"], scaling=case["scaling"], **SCALING[case["scaling"]])
    else:
        f = _frequencies(case["pairs"], case["scaling"])
    s["frequencies"] = f.to(DEV)
    return s


def _prepare_router(case, gen, seed):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    # tokens have tastes in common: some experts are asked for more than others
    z = _randn(gen, T, E, std=1.5) + _randn(gen, E, std=0.7)
    r = random.Random(seed)
    z[:, r.sample(range(E), min(case["masked"], E - 1))] = -math.inf
    if case["padded"]:
        z[T - case["padded"]:] = -math.inf
    s = {"op": case["op"], "logits": z.to(DTYPES[case["dtype"]]), "top_k": k, "renormalize": case["renormalize"]}
    if case["op"] == "router_grad":
        chosen, _ = _choose(s["logits"].float(), k)
        s["chosen"] = chosen.int()
        s["counts"] = torch.bincount(chosen[chosen >= 0], minlength=E).int()
        s["live"] = torch.full((1,), T - case["padded"], dtype=torch.int32, device=DEV)
        s["dgates"] = _randn(gen, T, k, std=1e-3)
        s["dlogits"] = torch.zeros_like(s["logits"])
    elif own:
        mu, h = _lib()
        s["chosen"], s["rows"] = (torch.zeros(T, k, dtype=torch.int32, device=DEV) for _ in range(2))
        s["order"] = torch.zeros(T * k, dtype=torch.int32, device=DEV)
        s["gates"] = torch.zeros(T, k, device=DEV)
        s["counts"] = torch.zeros(E, dtype=torch.int32, device=DEV)
        s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        s["live"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["losses"] = torch.zeros(2, device=DEV)
        s["workspace"] = torch.empty(mu.muon_router_workspace_size(h, s["logits"], k), dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] in ("norm", "norm_grad"):
        return _prepare_norm(case, gen)
    if case["op"] == "rotary":
        return _prepare_rotary(case, gen)
    return _prepare_router(case, gen, seed)


# ---------------------------------------------------------------- one pass ----

def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(2, keepdim=True) if s["center"] else None
    if s["center"]:
        x = x - mean
    rstd = (x.square().mean(2, keepdim=True) + EPS).rsqrt()
    y = x * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    out = {"y": y.to(s["x"].dtype), "rstd": rstd[:, :, 0]}
    if s["center"]:
        out["mean"] = mean[:, :, 0]
    return out


def _plain_norm_grad(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, :, None]
    hat = (x - s["mean"][:, :, None]) * rstd if s["center"] else x * rstd
    dw = (dy * hat).sum((0, 1), dtype=torch.float64)
    g = dy * s["w"].float()
    dx = g - hat * (g * hat).mean(2, keepdim=True)
    if s["center"]:
        dx = dx - g.mean(2, keepdim=True)
    out = {"dx": (dx * rstd).to(s["x"].dtype),
           "dw": s["dw"].copy_(s["dw"].double() + dw if s["add"] else dw)}
    if s["center"]:
        db = dy.sum((0, 1), dtype=torch.float64)
        out["db"] = s["db"].copy_(s["db"].double() + db if s["add"] else db)
    return out


def _plain_rotary(s):
    a = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = (f.float()[:, None, :] * s["scale"] for f in (a.cos(), a.sin()))
    if s["back"]:
        sin = -sin
    n, first = s["pairs"], s["first"]
    if s["interleaved"]:
        one, two = slice(first, first + 2 * n, 2), slice(first + 1, first + 2 * n, 2)
    else:
        one, two = slice(first, first + n), slice(first + n, first + 2 * n)
    out = []
    for x in s["x"]:
        y, u, v = x.clone(), x[:, :, one].float(), x[:, :, two].float()
        y[:, :, one] = (u * cos - v * sin).to(x.dtype)
        y[:, :, two] = (v * cos + u * sin).to(x.dtype)
        out.append(y)
    return {"q": out[0], "k": out[1]}


def _choose(z, k):
    """The k largest logits of every row, the lowest index first where they are
    equal: (experts, logits); -1 where a row has no logit above -inf left."""
    top, at = torch.sort(z, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    return torch.where(top == -math.inf, -1, at), top


def _softmax(z):
    """(probabilities, logarithm of the sum of exponentials, whether there is any)."""
    m = z.amax(1, keepdim=True)
    live = m > -math.inf
    e = (z - torch.where(live, m, 0.0)).exp()
    total = e.sum(1, keepdim=True)
    p = torch.where(live, e / total, 0.0)
    return p, torch.where(live, m + total.log(), 0.0)[:, 0], live[:, 0]


def _plain_router(s):
    z, k = s["logits"].float(), s["top_k"]
    T, E = z.shape
    chosen, _ = _choose(z, k)
    none = chosen < 0
    p, lse, live = _softmax(z)
    gates = torch.where(none, 0.0, p.gather(1, chosen.clamp(min=0)))
    if s["renormalize"]:
        total = gates.sum(1, keepdim=True)
        gates = torch.where(none, 0.0, gates / torch.where(total > 0, total, 1.0))
    group = torch.where(none, E, chosen).view(-1)
    counts = torch.bincount(group, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    order = group.argsort(stable=True)
    rows = torch.empty_like(order)
    rows[order] = torch.arange(T * k, device=DEV)
    order = torch.where(torch.arange(T * k, device=DEV) < offsets[E], order, -1)
    n, share = live.sum().clamp(min=1), counts.double() / offsets[E].clamp(min=1)
    balance = E * (share * p.sum(0, dtype=torch.float64)).sum() / n
    return {"chosen": chosen.int(), "gates": gates, "rows": torch.where(none, -1, rows.view(T, k)).int(),
            "order": order.int(), "counts": counts.int(), "offsets": offsets.int(),
            "live": live.sum().int().view(1),
            "losses": torch.stack([balance, lse.double().square().sum() / n]).float()}


def _plain_router_grad(s):
    z, chosen = s["logits"].float(), s["chosen"].long()
    E, none = z.shape[1], chosen < 0
    p, lse, _ = _softmax(z)
    n = s["live"].clamp(min=1)
    g = (BALANCE * E / n * (s["counts"].double() / s["counts"].sum().clamp(min=1))).float().expand_as(z)
    d = torch.where(none, 0.0, s["dgates"])
    at = chosen.clamp(min=0)
    if s["renormalize"]:
        gates = torch.where(none, 0.0, p.gather(1, at))
        total = gates.sum(1, keepdim=True)
        gates = gates / torch.where(total > 0, total, 1.0)
        d = gates * (d - (gates * d).sum(1, keepdim=True))
        dz = p * (g - (p * g).sum(1, keepdim=True))
        dz = dz.scatter_add(1, at, d)
    else:
        g = g.scatter_add(1, at, d)
        dz = p * (g - (p * g).sum(1, keepdim=True))
    dz = dz + p * (2.0 * Z / n * lse[:, None])
    return {"dlogits": dz.to(s["logits"].dtype)}


def _own(s):
    mu, h = _lib()
    op = s["op"]
    if op == "norm":
        mu.muon_layernorm_forward(h, s["x"], s["y"], weight=s["w"], bias=s["b"], mean=s["mean"], rstd=s["rstd"],
                                  eps=EPS, center=s["center"])
        out = {"y": s["y"], "rstd": s["rstd"]}
        return dict(out, mean=s["mean"]) if s["center"] else out
    if op == "norm_grad":
        mu.muon_layernorm_grad(h, s["x"], s["dy"], s["rstd"], s["workspace"], mean=s["mean"], weight=s["w"],
                               dx=s["y"], dweight=s["dw"], dbias=s["db"], accumulate=s["add"], center=s["center"])
        out = {"dx": s["y"], "dw": s["dw"]}
        return dict(out, db=s["db"]) if s["center"] else out
    if op == "rotary":
        mu.muon_rotary(h, s["x"], s["y"], s["positions"], s["frequencies"], first=s["first"],
                       interleaved=s["interleaved"], scale=s["scale"], transpose=s["back"])
        return {"q": s["y"][0], "k": s["y"][1]}
    if op == "router":
        mu.muon_router_forward(h, s["logits"], s["chosen"], s["gates"], s["counts"], s["offsets"], s["workspace"],
                               rows=s["rows"], order=s["order"], live=s["live"], losses=s["losses"],
                               renormalize=s["renormalize"])
        return {n: s[n] for n in ("chosen", "gates", "rows", "order", "counts", "offsets", "live", "losses")}
    mu.muon_router_grad(h, s["logits"], s["chosen"], s["counts"], s["live"], s["dlogits"], dgates=s["dgates"],
                        balance=BALANCE, z=Z, renormalize=s["renormalize"])
    return {"dlogits": s["dlogits"]}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "rotary": _plain_rotary,
            "router": _plain_router, "router_grad": _plain_router_grad}[state["op"]](state)


# ------------------------------------------------------------------- work ----

def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_grad"):
        rows, side = case["tokens"] * case["heads"], 2 if case["center"] else 1
        n, w = rows * case["cols"], BYTES[case["weight"]] * case["cols"]
        if op == "norm":
            return {"bytes": 2 * b * n + side * (w + 4 * rows), "flops": (8 if case["center"] else 5) * n}
        return {"bytes": 3 * b * n + w + 4 * side * rows + (2 if case["add"] else 1) * side * w,
                "flops": (14 if case["center"] else 11) * n}
    T = case["tokens"]
    if op == "rotary":
        heads = case["heads"] + case["kv_heads"]
        return {"bytes": 2 * b * T * heads * case["head_dim"] + 4 * T + 8 * case["pairs"],
                "flops": 6 * T * heads * case["pairs"]}
    E, k = case["experts"], case["top_k"]
    if op == "router":
        return {"bytes": b * T * E + 4 * (4 * T * k + 2 * E + 4), "flops": (6 + k) * T * E}
    return {"bytes": 2 * b * T * E + 4 * (2 * T * k + E + 1), "flops": 10 * T * E}


# ------------------------------------------------------------- in 64 bits ----

def _exact_norm(case, s):
    x = s["x"].double()
    out = {}
    if case["op"] == "norm":
        mu = x.sum(2) / case["cols"] if case["center"] else torch.zeros_like(x[:, :, 0])
        centred = x - mu.unsqueeze(2)
        out["rstd"] = 1.0 / torch.sqrt((centred * centred).sum(2) / case["cols"] + EPS)
        out["y"] = centred * out["rstd"].unsqueeze(2) * s["w"].double()
        if case["center"]:
            out["y"] += s["b"].double()
            out["mean"] = mu
        return {n: out[n] for n in (("y", "rstd", "mean") if case["center"] else ("y", "rstd"))}
    # the derivative of y_i by x_j, term by term, with the statistics as given
    r, dy = s["rstd"].double().unsqueeze(2), s["dy"].double()
    hat = x.sub_(s["mean"].double().unsqueeze(2)).mul_(r) if case["center"] else x.mul_(r)
    out["dw"] = (dy * hat).sum(0).sum(0)
    if case["add"]:
        out["dw"] += s["dw"].double()
    if case["center"]:
        out["db"] = dy.sum(0).sum(0) + (s["db"].double() if case["add"] else 0.0)
    g = dy * s["w"].double()
    along = torch.linalg.vecdot(g, hat).unsqueeze(2) / case["cols"]
    mean = g.sum(2, keepdim=True) / case["cols"] if case["center"] else 0.0
    out["dx"] = g.sub_(mean).sub_(hat.mul_(along)).mul_(r)
    return {n: out[n] for n in (("dx", "dw", "db") if case["center"] else ("dx", "dw"))}


def _exact_rotary(case, s):
    n, first = case["pairs"], case["first"]
    f = _frequencies(n, case["scaling"]).to(DEV)
    turn = torch.polar(torch.full((case["tokens"], n), float(s["scale"]), dtype=torch.float64, device=DEV),
                       s["positions"].double().unsqueeze(1) * f * (-1.0 if case["back"] else 1.0)).unsqueeze(1)
    out = {}
    for name, x in zip("qk", s["x"]):
        y = x.double()
        part = y[..., first:first + 2 * n]
        shape = (*part.shape[:2], n, 2) if case["interleaved"] else (*part.shape[:2], 2, n)
        pair = part.reshape(shape)
        pair = pair if case["interleaved"] else pair.transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        y[..., first:first + 2 * n] = (z if case["interleaved"] else z.transpose(2, 3)).reshape(part.shape)
        out[name] = y
    return out


def _exact_router(case, s):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    z = s["logits"].double()
    live = z.amax(1) > -math.inf
    lse = torch.where(live, torch.logsumexp(z, 1), 0.0)
    p = torch.where(live.unsqueeze(1), torch.exp(z - lse.unsqueeze(1)), 0.0)
    n = max(1, int(live.sum()))
    if case["op"] == "router":
        # one choice after the other: the first of the largest logits left
        left, numbers, picks = z.clone(), torch.arange(E, device=DEV), []
        for _ in range(k):
            m = left.amax(1, keepdim=True)
            i = torch.where(left == m, numbers, E).amin(1, keepdim=True)
            picks.append(torch.where(m > -math.inf, i, -1))
            left.scatter_(1, i, -math.inf)
        chosen = torch.cat(picks, 1)
    else:
        chosen = s["chosen"].long()
    hit = chosen.unsqueeze(2) == torch.arange(E, device=DEV) if T * k * E <= 4e8 else None
    if hit is None:
        counts = torch.stack([(chosen == e).sum() for e in range(E)])
    else:
        counts = hit.sum((0, 1))
    share = counts.double() / max(1, int(counts.sum()))
    picked = torch.where(chosen >= 0, p.gather(1, chosen.clamp(min=0)), 0.0)
    gates = picked / picked.sum(1, keepdim=True).clamp(min=1e-300) if case["renormalize"] else picked
    if case["op"] == "router":
        offsets = torch.zeros(E + 1, dtype=torch.long, device=DEV)
        order, rows, at = torch.full((T * k,), -1, device=DEV), torch.full((T * k,), -1, device=DEV), 0
        for e in range(E):
            mine = (chosen.view(-1) == e).nonzero().view(-1)
            order[at:at + len(mine)] = mine
            rows[mine] = torch.arange(at, at + len(mine), device=DEV)
            at += len(mine)
            offsets[e + 1] = at
        losses = torch.stack([E * (share @ p.sum(0)) / n, (lse * lse).sum() / n])
        return {"chosen": chosen.int(), "gates": gates, "rows": rows.view(T, k).int(), "order": order.int(),
                "counts": counts.int(), "offsets": offsets.int(),
                "live": torch.tensor([int(live.sum())], dtype=torch.int32, device=DEV), "losses": losses}
    dp = (BALANCE * E / n * share).repeat(T, 1)
    d = torch.where(chosen >= 0, s["dgates"].double(), 0.0)
    if case["renormalize"]:
        # d gate_i / d p_j = (delta_ij - gate_i) / sum of the picked
        d = (d - (d * gates).sum(1, keepdim=True)) / picked.sum(1, keepdim=True).clamp(min=1e-300)
        d = torch.where(chosen >= 0, d, 0.0)
    dp.scatter_add_(1, chosen.clamp(min=0), d)
    return {"dlogits": p * (dp - (p * dp).sum(1, keepdim=True) + 2.0 * Z / n * lse.unsqueeze(1))}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(case, s)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    return _exact_router(case, s)
