"""The operators around the optimizer step, as cases to be measured.

Four kinds: the global gradient norm and the clip to it; the products of a
mixture-of-experts layer grouped by expert (forward, input gradient, weight
gradient); and the largest attention logit per head that QK-Clip reads.

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

_library = None


def _lib():
    """The package and one handle for the process, as a program keeps them."""
    global _library
    if _library is None:
        import muon_step_02_amd as mu
        _library = (mu, mu.muon_init(0))
    return _library


# ------------------------------------------------------------------ cases ----

def _grads(name, op, matrices, rows, cols, vectors, pad, dtype, out):
    """`matrices` gradients of rows x cols (row stride cols + pad) and
    `vectors` of cols values; `out`: the type of the clipped gradients."""
    return {"name": name, "op": op, "matrices": matrices, "rows": rows, "cols": cols,
            "vectors": vectors, "pad": pad, "dtype": dtype, "out": out}


def _experts(name, op, experts, active, tokens, spare, rows, cols, dtype, out, add):
    """`tokens` rows over `active` of `experts` experts, `spare` rows behind
    the last group, weights of rows x cols; `out`: the type of the result
    (`dtype` but for weight gradients); `add`: weight gradients accumulate."""
    return {"name": name, "op": op, "experts": experts, "active": active, "tokens": tokens,
            "spare": spare, "rows": rows, "cols": cols, "dtype": dtype, "out": out, "add": add}


def _smax(name, heads, kv_heads, head_dim, sequences, tokens, more, causal, dtype):
    """`sequences` packed sequences of `tokens` queries together; every
    sequence has `more` keys before its first query."""
    return {"name": name, "op": "smax", "heads": heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "sequences": sequences, "tokens": tokens, "more": more,
            "causal": causal, "dtype": dtype}


def listed():
    return [
        # the norm of the layer norms and biases of a d=1024 block: latency
        _grads("norm, vectors of a d=1024 block", "norm", 0, 0, 1024, 4, 0, "f32", "f32"),
        # the norm over all expert gradients of the 64-expert d=7168 layer
        _grads("norm, 64 experts", "norm", 192, 2048, 7168, 0, 0, "f32", "f32"),
        # every gradient of a d=1024 block clipped before a caller's own step
        _grads("clip, d=1024 block", "clip", 16, 1024, 1024, 4, 0, "f32", "f32"),
        # the bf16 gradients of a d=4096 layer clipped into fp32 ones, rows padded
        _grads("clip, d=4096 layer to fp32", "clip", 4, 14336, 4096, 2, 8, "bf16", "f32"),
        # eight tokens at a time through the layer (top 8 of 64 experts)
        _experts("forward, 64 rows of 64 experts", "forward", 64, 41, 64, 0, 2048, 7168, "bf16", "bf16", False),
        # a training batch of the layer's up projection, some experts empty
        _experts("forward, 32768 rows", "forward", 64, 61, 32768, 37, 2048, 7168, "bf16", "bf16", False),
        # a small layer of odd widths on its way back
        _experts("grad input, odd widths", "grad_input", 8, 8, 4099, 5, 1000, 2056, "bf16", "bf16", False),
        # the training batch on its way back through the down projection
        _experts("grad input, 16384 rows", "grad_input", 64, 60, 16384, 0, 7168, 2048, "bf16", "bf16", False),
        # a small fp32 layer's weight gradients
        _experts("grad weight, fp32", "grad_weight", 8, 7, 777, 3, 384, 250, "f32", "f32", False),
        # the layer's weight gradients added to fp32 ones (micro-batches)
        _experts("grad weight, 32768 rows", "grad_weight", 64, 61, 32768, 0, 2048, 7168, "bf16", "f32", True),
        # packed short sequences with shared key heads
        _smax("smax, 16 packed sequences", 32, 8, 128, 16, 4099, 0, True, "bf16"),
        # one long sequence of a 64-head layer
        _smax("smax, 8192 tokens", 64, 64, 128, 1, 8192, 0, True, "bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width: mostly a multiple of 8 (or 64), at times any number."""
    n = _log(rng, low, high)
    step = rng.choice((1, 8, 8, 64, 64, 64))
    return max(low, n // step * step)


def draw(rng):
    op = rng.choice(("norm", "clip", "forward", "grad_input", "grad_weight", "smax"))
    if op in ("norm", "clip"):
        cols, dtype = _width(rng, 33, 8192), rng.choice(("f32", "bf16"))
        rows = _width(rng, 1, 8192)
        most = int(min(256, max(1, 1.2e9 // (rows * cols))))
        return {"op": op, "matrices": _log(rng, 1, most), "rows": rows, "cols": cols,
                "vectors": rng.choice((0, 1, 5, 49)), "pad": rng.choice((0, 0, 8, 3)),
                "dtype": dtype, "out": rng.choice((dtype, "f32"))}
    if op == "smax":
        heads, dim = rng.choice(((8, 8), (16, 4), (32, 8), (24, 24), (64, 1))), rng.choice((64, 128, 128, 192, 80))
        sequences = _log(rng, 1, 33)
        tokens = max(sequences, _log(rng, 17, 6000))
        return {"op": op, "heads": heads[0], "kv_heads": heads[1], "head_dim": dim,
                "sequences": sequences, "tokens": tokens, "more": rng.choice((0, 0, 1, 130)),
                "causal": rng.random() < 0.8, "dtype": rng.choice(("bf16", "bf16", "bf16", "f32"))}
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    experts = _log(rng, 1, 128)
    active = rng.randint(max(1, experts * 3 // 4), experts)
    rows, cols = _width(rng, 64, 7168), _width(rng, 64, 7168)
    while experts * rows * cols > 6e8:
        rows, cols = max(64, rows // 16 * 8), max(64, cols // 16 * 8)
    most = min(32768, (4e11 if dtype == "bf16" else 4e10) / (2 * rows * cols))
    tokens = max(active, _log(rng, 1, max(2, most)))
    add = op == "grad_weight" and rng.random() < 0.5
    out = rng.choice(("f32", dtype)) if op == "grad_weight" else dtype
    return {"op": op, "experts": experts, "active": active, "tokens": tokens,
            "spare": rng.choice((0, 0, 1, 70)), "rows": rows, "cols": cols, "dtype": dtype,
            "out": out, "add": add}


# ----------------------------------------------------------------- inputs ----

def _randn(gen, *shape, dtype, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype) * std


def _lengths(case):
    """Lengths of the packed sequences: of the case alone, no two runs differ."""
    r = random.Random("%d %d" % (case["sequences"], case["tokens"]))
    w = [r.expovariate(1.0) + 0.05 for _ in range(case["sequences"])]
    left = case["tokens"] - case["sequences"]
    n = [1 + int(left * x / sum(w)) for x in w]
    n[0] += case["tokens"] - sum(n)
    return n


def _prefix(sizes):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return out


def _views(flat, case, pad):
    """The gradients of a case as views of one buffer: matrices, then vectors."""
    rows, cols, ld = case["rows"], case["cols"], case["cols"] + pad
    got = [flat[i * rows * ld:(i + 1) * rows * ld].view(rows, ld)[:, :cols]
           for i in range(case["matrices"])]
    at = case["matrices"] * rows * ld
    return got + [flat[at + i * cols:at + (i + 1) * cols] for i in range(case["vectors"])]


def _prepare_grads(case, gen):
    pad = case["pad"]
    total = case["matrices"] * case["rows"] * (case["cols"] + pad) + case["vectors"] * case["cols"]
    flat = _randn(gen, total, dtype=DTYPES[case["dtype"]])
    grads = _views(flat, case, pad)
    # layers differ in scale by orders of magnitude
    scale = 10.0 ** (torch.rand(len(grads), generator=gen, device=DEV) * 3 - 4)
    torch._foreach_mul_(grads, list(scale.to(flat.dtype).unbind()))
    s = {"op": case["op"], "grads": grads, "max_norm": 1.0}
    if case["op"] == "clip":
        dense = case["matrices"] * case["rows"] * case["cols"] + case["vectors"] * case["cols"]
        s["clipped"] = torch.zeros(dense, device=DEV, dtype=DTYPES[case["out"]])
        s["out"] = _views(s["clipped"], case, 0)
    # the norm of what is drawn lies over or under the bound, by the seed
    most = math.sqrt(total) * 10.0 ** -2.5
    s["max_norm"] = most * (0.25 if float(torch.rand(1, generator=gen, device=DEV)) < 0.75 else 4.0)
    if own:
        mu, h = _lib()
        s["h"], s["norm"] = h, torch.zeros((), device=DEV)
        s["plan"] = [mu.muon_grad(g, o) for g, o in zip(grads, s.get("out", [None] * len(grads)))]
        s["workspace"] = torch.empty(mu.muon_grad_workspace_size(h, s["plan"]), dtype=torch.uint8, device=DEV)
    return s


def _prepare_experts(case, gen, seed):
    E, T, N, K = case["experts"], case["tokens"], case["rows"], case["cols"]
    dtype, held = DTYPES[case["dtype"]], case["tokens"] + case["spare"]
    # a skewed router: which experts get rows, and how many, by the seed
    r = random.Random(seed)
    chosen = sorted(r.sample(range(E), case["active"]))
    w = [r.lognormvariate(0.0, 0.7) for _ in chosen]
    n = [1 + int((T - len(chosen)) * x / sum(w)) for x in w]
    n[r.randrange(len(n))] += T - sum(n)
    sizes = [0] * E
    for e, k in zip(chosen, n):
        sizes[e] = k
    at = _prefix(sizes)
    s = {"op": case["op"], "at": at, "offsets": torch.tensor(at, dtype=torch.int32, device=DEV)}
    if case["op"] == "grad_weight":
        s["x"] = _randn(gen, held, K, dtype=dtype)
        s["dy"] = _randn(gen, held, N, dtype=dtype, std=1e-2)
        s["add"] = case["add"]
        s["dw"] = torch.zeros(E, N, K, device=DEV, dtype=DTYPES[case["out"]])
        if case["add"]:
            s["dw"].normal_(generator=gen).mul_(1e-2)
    else:
        s["w"] = _randn(gen, E, N, K, dtype=dtype, std=0.02)
        wide, to = (K, N) if case["op"] == "forward" else (N, K)
        s["x"] = _randn(gen, held, wide, dtype=dtype)
        s["y"] = torch.full((held, to), 7.0, device=DEV, dtype=dtype)
    if own:
        mu, s["h"] = _lib()
        s["plan"] = mu.muon_experts(list((s["dw"] if case["op"] == "grad_weight" else s["w"]).unbind()))
    return s


def _prepare_smax(case, gen):
    n = _lengths(case)
    cu_q, cu_k = _prefix(n), _prefix([x + case["more"] for x in n])
    dtype, D = DTYPES[case["dtype"]], case["head_dim"]
    q = _randn(gen, cu_q[-1], case["heads"], D, dtype=dtype)
    k = _randn(gen, cu_k[-1], case["kv_heads"], D, dtype=dtype)
    # some heads have grown: their logits pass the threshold of the clip
    q *= (1.0 + 3.0 * torch.rand(case["heads"], 1, generator=gen, device=DEV)).to(dtype)
    s = {"op": "smax", "q": q, "k": k, "at_q": cu_q, "at_k": cu_k, "causal": case["causal"],
         "scale": D ** -0.5, "cu_q": torch.tensor(cu_q, dtype=torch.int32, device=DEV),
         "cu_k": torch.tensor(cu_k, dtype=torch.int32, device=DEV)}
    if own:
        mu, s["h"] = _lib()
        s["smax_q"] = torch.zeros(case["heads"], device=DEV)
        s["smax_k"] = torch.zeros(case["kv_heads"], device=DEV)
        s["workspace"] = torch.empty(mu.muon_qk_smax_workspace_size(s["h"], q, k, s["cu_q"]),
                                     dtype=torch.uint8, device=DEV)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] in ("norm", "clip"):
        return _prepare_grads(case, gen)
    if case["op"] == "smax":
        return _prepare_smax(case, gen)
    return _prepare_experts(case, gen, seed)


# ---------------------------------------------------------------- one pass ----

def _plain_norm(grads):
    return torch.stack([g.double().square().sum() for g in grads]).sum().sqrt()


def _plain_clip(s):
    norm = _plain_norm(s["grads"])
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float()
    [o.copy_(g.float() * scale) for g, o in zip(s["grads"], s["out"])]
    return {"norm": norm.float(), "clipped": s["clipped"]}


def _plain_rows(s, product):
    """product(rows of x, weight) of every group that has rows."""
    at, x, y = s["at"], s["x"], s["y"]
    [y[a:b].copy_(product(x[a:b].float(), s["w"][e].float()))
     for e, (a, b) in enumerate(zip(at, at[1:])) if b > a]
    return y


def _plain_grad_weight(s):
    at, x, dy, dw = s["at"], s["x"], s["dy"], s["dw"]
    groups = [(e, dy[a:b].float().t() @ x[a:b].float()) if b > a else (e, torch.zeros_like(dw[e], dtype=torch.float32))
              for e, (a, b) in enumerate(zip(at, at[1:]))]
    [dw[e].copy_(dw[e].float() + g if s["add"] else g) for e, g in groups]
    return dw


def _plain_logits(s, i):
    """The largest logit of every query head in sequence i."""
    (a, b), (c, d) = s["at_q"][i:i + 2], s["at_k"][i:i + 2]
    heads, kv, n, m = s["q"].shape[1], s["k"].shape[1], b - a, d - c
    q = s["q"][a:b].float().transpose(0, 1).reshape(kv, heads // kv * n, -1)
    k = s["k"][c:d].float().permute(1, 2, 0).contiguous()
    z = (torch.bmm(q, k) * s["scale"]).view(heads, n, m)
    if s["causal"]:
        row = torch.arange(n, device=DEV)[:, None] + m - n
        z = torch.where(torch.arange(m, device=DEV)[None, :] <= row, z, -math.inf)
    return z.amax(2).amax(1)


def _plain_smax(s):
    heads, kv = s["q"].shape[1], s["k"].shape[1]
    top = torch.stack([_plain_logits(s, i) for i in range(len(s["at_q"]) - 1)]).amax(0)
    return {"q": top, "k": top.view(kv, heads // kv).amax(1)}


def _own(s):
    mu, h = _lib()
    op = s["op"]
    if op == "norm":
        mu.muon_grad_norm(h, s["plan"], s["max_norm"], s["workspace"], norm_out=s["norm"])
        return {"norm": s["norm"]}
    if op == "clip":
        mu.muon_grad_clip(h, s["plan"], s["max_norm"], s["workspace"], norm_out=s["norm"])
        return {"norm": s["norm"], "clipped": s["clipped"]}
    if op == "forward":
        mu.muon_expert_forward(h, s["plan"], s["offsets"], s["x"], s["y"])
        return s["y"]
    if op == "grad_input":
        mu.muon_expert_grad_input(h, s["plan"], s["offsets"], s["x"], s["y"])
        return s["y"]
    if op == "grad_weight":
        mu.muon_expert_grad_weight(h, s["plan"], s["offsets"], s["x"], s["dy"], accumulate=s["add"])
        return s["dw"]
    mu.muon_qk_smax(h, s["q"], s["k"], s["cu_q"], s["cu_k"], s["smax_q"], s["workspace"],
                    smax_k=s["smax_k"], scale=s["scale"], causal=s["causal"])
    return {"q": s["smax_q"], "k": s["smax_k"]}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "norm":
        return {"norm": _plain_norm(state["grads"]).float()}
    if op == "clip":
        return _plain_clip(state)
    if op == "forward":
        return _plain_rows(state, lambda x, w: x @ w.t())
    if op == "grad_input":
        return _plain_rows(state, lambda x, w: x @ w)
    if op == "grad_weight":
        return _plain_grad_weight(state)
    return _plain_smax(state)


# ------------------------------------------------------------------- work ----

def _pairs(n, more, causal):
    """Unmasked (query, key) pairs of a sequence of n queries, n + more keys."""
    return n * more + n * (n + 1) // 2 if causal else n * (n + more)


def work(case):
    op = case["op"]
    if op in ("norm", "clip"):
        n = (case["matrices"] * case["rows"] + case["vectors"]) * case["cols"]
        wrote = n * BYTES[case["out"]] if op == "clip" else 0
        return {"bytes": n * BYTES[case["dtype"]] + wrote + 4, "flops": (2 if op == "norm" else 3) * n}
    b = BYTES[case["dtype"]]
    if op == "smax":
        n = _lengths(case)
        keys = case["tokens"] + case["sequences"] * case["more"]
        pairs = sum(_pairs(x, case["more"], case["causal"]) for x in n)
        return {"bytes": b * case["head_dim"] * (case["tokens"] * case["heads"] + keys * case["kv_heads"]),
                "flops": 2 * case["head_dim"] * case["heads"] * pairs}
    T, N, K = case["tokens"], case["rows"], case["cols"]
    flops = 2 * T * N * K
    if op == "grad_weight":
        o = BYTES[case["out"]]
        # where gradients are added, those of an expert without rows stay as they are
        held = 2 * case["active"] if case["add"] else case["experts"]
        return {"bytes": b * T * (N + K) + o * held * N * K, "flops": flops}
    return {"bytes": b * (T * (N + K) + case["active"] * N * K), "flops": flops}


# ------------------------------------------------------------- in 64 bits ----

def _exact_grads(case, s):
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for g in s["grads"]:
        total += torch.linalg.vector_norm(g, dtype=torch.float64) ** 2
    norm = total.sqrt()
    if case["op"] == "norm":
        return {"norm": norm}
    factor = min(1.0, s["max_norm"] / float(norm))
    out = torch.empty(s["clipped"].numel(), dtype=torch.float64, device=DEV)
    at = 0
    for g in s["grads"]:
        out[at:at + g.numel()] = (g.to(torch.float64) * factor).reshape(-1)
        at += g.numel()
    return {"norm": norm, "clipped": out}


def _exact_experts(case, s):
    if case["op"] == "grad_weight":
        out = s["dw"].double() if case["add"] else torch.zeros(s["dw"].shape, dtype=torch.float64, device=DEV)
    else:
        out = s["y"].double()
    first = 0
    for e, last in enumerate(s["at"][1:]):
        x = s["x"][first:last].double()
        if case["op"] == "grad_weight":
            out[e] += torch.mm(s["dy"][first:last].double().t().contiguous(), x)
        elif last > first:
            w = s["w"][e].double()
            out[first:last] = torch.mm(x, w.t().contiguous() if case["op"] == "forward" else w)
        first = last
    return out


def _exact_smax(case, s):
    q, k = s["q"].double(), s["k"].double()
    share = case["heads"] // case["kv_heads"]
    best = torch.full((case["heads"],), -math.inf, dtype=torch.float64, device=DEV)
    n = _lengths(case)
    a = c = 0
    for length in n:
        b, d = a + length, c + length + case["more"]
        for h in range(case["heads"]):
            z = torch.mm(q[a:b, h].contiguous(), k[c:d, h // share].t().contiguous())
            if case["causal"]:
                z = z.masked_fill(~torch.ones(z.shape, dtype=torch.bool, device=DEV).tril(case["more"]), -math.inf)
            best[h] = torch.maximum(best[h], z.max() * case["head_dim"] ** -0.5)
        a, c = b, d
    return {"q": best, "k": torch.stack([best[i * share:(i + 1) * share].max() for i in range(case["kv_heads"])])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        return _exact_grads(case, s)
    if case["op"] == "smax":
        return _exact_smax(case, s)
    return _exact_experts(case, s)
