"""The router against its formulas in 64 bits; choices, counts, rows and order
exactly.

Bounds, with u = 2^-24 and r the largest distance of a token's (finite) logits
from its top one: exp(z - top) is off by r u from the rounded difference, 4 u of
its own and what its argument is scaled with, 2 r u; the sum over the experts by
26 u (16 values of a lane, 6 steps over lanes); quotients by 2 u.  A probability
is off by (6 r + 64) u of itself, whatever the order.  Sums of probabilities: 64
more additions in fp32, then 64 bits."""

import numpy as np
import pytest
import torch

import muon_step_02_amd as mu
from harness import Handle

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
NEG, U = -float("inf"), 2.0 ** -24
INTS = ("chosen", "rows", "order", "counts", "offsets", "live")


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _logits(seed, tokens, experts, dtype, pad=0, shift=0, std=2.0):
    flat = torch.randn(tokens * (experts + pad) + shift, generator=_gen(seed), device=DEV) * std
    return flat.to(dtype)[shift:].view(tokens, experts + pad)[:, :experts]


def _route(z, k, renormalize=False, wanted=True, stream=None):
    T, E = z.shape
    h = Handle.get()

    def ints(*s):
        return torch.full(s, 77, dtype=torch.int32, device=DEV)

    out = dict(chosen=ints(T, k), gates=torch.full((T, k), 77.0, device=DEV), counts=ints(E), offsets=ints(E + 1))
    more = dict(rows=ints(T, k), order=ints(T * k), live=ints(1), losses=torch.full((2,), 77.0, device=DEV))
    ws = torch.full((mu.muon_router_workspace_size(h, z, k),), 255, dtype=torch.uint8, device=DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    mu.muon_router_forward(h, z, workspace=ws, renormalize=renormalize, stream=stream, **out, **(more if wanted else {}))
    return dict(out, **more)


def _reference(z, k, renormalize):
    """Everything in 64 bits on the host."""
    z = z.double().cpu().numpy()
    T, E = z.shape
    by = np.argsort(-z, axis=1, kind="stable")[:, :k]
    chosen = np.where(np.take_along_axis(z, by, 1) > NEG, by, -1)
    live = (z > NEG).any(1)
    top = np.where(live, z.max(1, initial=NEG), 0.0)
    e = np.exp(z - top[:, None])
    lse = np.where(live, top + np.log(np.where(live, e.sum(1), 1.0)), 0.0)
    p = np.where(live[:, None], np.exp(z - lse[:, None]), 0.0)
    gates = np.where(chosen >= 0, np.take_along_axis(p, np.maximum(chosen, 0), 1), 0.0)
    if renormalize:
        s = gates.sum(1, keepdims=True)
        gates = gates / np.where(s > 0, s, 1.0)
    flat = chosen.reshape(-1)
    counts = np.bincount(flat[flat >= 0], minlength=E)
    offsets = np.concatenate([[0], counts.cumsum()])
    order = np.full(T * k, -1)
    rows = np.full(T * k, -1)
    place = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:offsets[-1]]
    order[:offsets[-1]] = place
    rows[place] = np.arange(offsets[-1])
    n, total = max(1, live.sum()), max(1, offsets[-1])
    balance = E * (counts / total * p.sum(0)).sum() / n
    finite = np.where(z > NEG, z, top[:, None])
    # (beyond 110 both are zero but for what 1e-38 covers)
    spread = min(110.0, float((top[:, None] - finite).max(initial=0.0)))
    return dict(chosen=chosen, gates=gates, rows=rows.reshape(T, k), order=order, counts=counts, offsets=offsets,
                live=np.array([live.sum()]), losses=np.array([balance, (lse ** 2).sum() / n])), \
        (6 * spread + 64) * U, float((np.abs(lse) * (np.abs(top) + 64)).sum() / n * 4 * U)


def _check(z, k, renormalize=False):
    got = _route(z, k, renormalize)
    want, rel, lse = _reference(z, k, renormalize)
    for name in INTS:
        assert np.array_equal(got[name].cpu().numpy(), want[name]), name
    gates, losses = got["gates"].double().cpu().numpy(), got["losses"].double().cpu().numpy()
    # (a sum of gates is off as they are)
    assert (np.abs(gates - want["gates"]) <= (2 if renormalize else 1) * rel * want["gates"] + 1e-38).all()
    assert abs(losses[0] - want["losses"][0]) <= (rel + 130 * U) * want["losses"][0]
    if want["losses"][1] > torch.finfo(F32).max:      # the square of a logit near the lowest value: rounded to fp32
        assert losses[1] == float("inf")
    else:
        assert abs(losses[1] - want["losses"][1]) <= lse + U * want["losses"][1]
    return got


EXPERTS = [(1, 1), (2, 1), (2, 2), (3, 3), (7, 2), (8, 8), (9, 4), (16, 16), (17, 5), (32, 32), (33, 6), (61, 3), (64, 8),
           (65, 8), (127, 7), (128, 1), (129, 32), (200, 12), (256, 8), (257, 8), (500, 9), (512, 32), (513, 8),
           (1000, 31), (1024, 32)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("experts,k", EXPERTS)
def test_experts(experts, k, dtype):
    for tokens in (1, 33, 200):
        for renormalize in (False, True):
            _check(_logits(experts, tokens, experts, dtype), k, renormalize)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [1, 2, 63, 64, 65, 127, 128, 129, 1000, 4097, 20011])
def test_tokens(tokens, dtype):
    _check(_logits(tokens, tokens, 64, dtype), 8)
    _check(_logits(tokens, tokens, 10, dtype), 3, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_tokens(dtype):
    # more workgroups than the sums between them take at once
    _check(_logits(3, 300001, 5, dtype), 2, True)
    _check(_logits(4, 70001, 200, dtype), 8)


def test_tokens_far_apart():
    # 2^31 logits and more between the first token's and the last one's
    far = (1 << 30) + 8
    buf = torch.zeros(2 * far + 80, device=DEV, dtype=BF16)
    z = torch.as_strided(buf, (3, 80), (far, 1))
    small = _logits(5, 3, 80, BF16)
    z.copy_(small)
    want, got = _route(small, 8), _route(z, 8)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    d = torch.randn(3, 8, generator=_gen(1), device=DEV)
    ref = _grad(small, want, d, 0.1, 0.1, True)
    assert torch.equal(_grad(z, want, d, 0.1, 0.1, True), ref)
    wide = torch.as_strided(torch.zeros(2 * far + 80, device=DEV, dtype=BF16), (3, 80), (far, 1))
    assert torch.equal(_grad(small, want, d, 0.1, 0.1, True, out=wide), ref)


def test_logits_next_to_zero_keep_their_order():
    # values that have no normal fp32 form, of both signs, with ties
    z = torch.randint(-3, 4, (130, 30), generator=_gen(6), device=DEV).float() * 1e-42
    assert int((z != 0).sum()) > 0
    got = _route(z, 6)
    by = np.argsort(-z.double().cpu().numpy(), axis=1, kind="stable")[:, :6]
    assert np.array_equal(got["chosen"].cpu().numpy(), by)


def test_no_tokens():
    got = _route(_logits(1, 0, 64, F32), 8)
    for name in ("counts", "offsets", "live", "losses"):
        assert float(got[name].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (1, 5)])
def test_strides_and_alignments(pad, shift, dtype):
    for experts in (64, 61, 300):
        _check(_logits(2, 150, experts, dtype, pad, shift), 6)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("experts,k", [(8, 8), (61, 6), (64, 8), (300, 20), (1024, 32)])
def test_equal_logits_go_to_the_lowest_index(experts, k, dtype):
    gen = _gen(3)
    for values in (1, 2, 4):
        z = torch.randint(0, values, (130, experts), generator=gen, device=DEV).to(dtype)
        _check(z, k)
        # both zeros are equal
        z = torch.where(torch.randint(0, 2, z.shape, generator=gen, device=DEV) == 1, -z, z).to(dtype)
        _check(z, k)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_experts_out_of_reach_and_tokens_without_any(dtype):
    for tokens in (50, 300):
        z = _logits(4, tokens, 61, dtype)
        z[:, ::3] = NEG
        z[::7] = NEG                       # padding within the batch
        z[tokens - 20:] = NEG              # and behind it
        z[3, :59] = NEG                    # two experts left, fewer than the choices
        z[5, 1:] = NEG
        z[5, 0] = torch.finfo(dtype).min   # the lowest value is one to choose
        for renormalize in (False, True):
            got = _check(z, 6, renormalize)
            assert int((got["chosen"][3] >= 0).sum()) == (z[3] > NEG).sum()
            assert got["chosen"][5].tolist() == [0, -1, -1, -1, -1, -1] and float(got["gates"][5, 0]) == 1.0
        got = _check(torch.full_like(z, NEG), 6)
        assert float(got["losses"].abs().max()) == 0.0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("experts", [129, 256, 300, 512, 700, 1024])
def test_few_choices_of_many_experts(experts, dtype):
    # up to 8 choices are found at once, from up to 16 logits that reach a bound
    gen = _gen(experts)
    for k in (1, 3, 7, 8):
        for values in (30, 100, 250):       # some of the largest are equal
            _check(torch.randint(0, values, (90, experts), generator=gen, device=DEV).to(dtype), k)
        z = _logits(k, 90, experts, dtype)
        z[::3] = NEG                        # tokens without any, beside others
        z[1::6, 5:] = NEG                   # with fewer than the choices
        z[2::6, :experts - 17] = NEG        # with all of them close together
        z[4::6] = torch.where(torch.arange(experts, device=DEV) % 16 == 3, z[4::6], NEG)
        for renormalize in (False, True):
            _check(z, k, renormalize)
        want = _route(z, k)
        z[7, 100] = float("nan")
        got = _route(z, k)
        assert bool(torch.isnan(got["gates"][7]).all()) and not bool((got["chosen"][7] == 100).any())
        keep = torch.arange(90, device=DEV) != 7
        for n in ("chosen", "gates"):
            assert torch.equal(got[n][keep], want[n][keep])


def test_values_far_apart_and_infinite():
    z = torch.zeros(70, 20, device=DEV)
    z[:, 3], z[:, 5] = 3e38, -3e38
    got = _route(z, 3)
    assert bool((got["chosen"] == torch.tensor([3, 0, 1], device=DEV)).all())
    assert bool((got["gates"] == torch.tensor([1.0, 0.0, 0.0], device=DEV)).all())
    # a NaN or an infinity leaves its token without gates, and the losses without value
    for value in (float("nan"), float("inf")):
        z = _logits(5, 70, 20, F32)
        want = _route(z, 3)
        z[33, 4] = value
        for renormalize in (False, True):
            got = _route(z, 3, renormalize)
            assert bool(torch.isnan(got["gates"][33]).any()) and bool(torch.isnan(got["losses"]).all())
            keep = torch.arange(70, device=DEV) != 33
            assert torch.equal(got["chosen"][keep], want["chosen"][keep])
            if not renormalize:
                assert torch.equal(got["gates"][keep], want["gates"][keep])
            assert bool((got["chosen"][33] == 4).any()) == (value == float("inf"))
    got = _route(torch.full((70, 20), float("nan"), device=DEV), 3)
    assert bool((got["chosen"] == -1).all()) and int(got["live"]) == 70 and int(got["offsets"][-1]) == 0


def test_what_is_not_wanted_and_a_fixed_order():
    for tokens in (40, 3000):
        z = _logits(6, tokens, 100, BF16)
        a, b, c = _route(z, 8), _route(z, 8), _route(z, 8, wanted=False)
        for name in a:
            assert torch.equal(a[name], b[name]), name
        for name in ("chosen", "gates", "counts", "offsets"):
            assert torch.equal(a[name], c[name]), name


def test_outputs_end_where_they_should():
    h = Handle.get()
    for tokens in (5, 64, 65, 700):
        z, k = _logits(7, tokens, 33, F32), 3
        sizes = dict(chosen=tokens * k, gates=tokens * k, counts=33, offsets=34, rows=tokens * k, order=tokens * k, live=1,
                     losses=2)
        guard = {n: torch.full((s + 64,), 77, dtype=torch.float32 if n in ("gates", "losses") else torch.int32, device=DEV)
                 for n, s in sizes.items()}
        view = {n: guard[n][32:32 + s] for n, s in sizes.items()}
        for n in ("chosen", "gates", "rows"):
            view[n] = view[n].view(tokens, k)
        size = mu.muon_router_workspace_size(h, z, k)
        space = torch.full((size + 512,), 255, dtype=torch.uint8, device=DEV)
        mu.muon_router_forward(h, z, workspace=space[256:256 + size], **view)
        want = _route(z, k)
        for n, s in sizes.items():
            assert bool((guard[n][:32] == 77).all()) and bool((guard[n][32 + s:] == 77).all()), n
            assert torch.equal(view[n], want[n]), n
        assert bool((space[:256] == 255).all()) and bool((space[256 + size:] == 255).all())


# ---- gradient --------------------------------------------------------------------------

def _grad(z, got, dgates, balance, zc, renormalize, out=None, stream=None):
    d = torch.full(z.shape, 7.0, device=DEV, dtype=z.dtype) if out is None else out
    mu.muon_router_grad(Handle.get(), z, got["chosen"], got["counts"], got["live"], d, dgates=dgates, balance=balance,
                        z=zc, renormalize=renormalize, stream=stream)
    return d


def _loss(z, chosen, counts, dgates, balance, zc, renormalize):
    """What router_grad differentiates, in 64 bits (chosen and counts constant)."""
    live = z.amax(1) > NEG
    lse = torch.where(live, torch.logsumexp(torch.where(live[:, None], z, 0.0), 1), 0.0)
    p = torch.where(live[:, None], (z - lse[:, None]).exp(), 0.0)
    g = torch.where(chosen >= 0, p.gather(1, chosen.clamp(min=0).long()), 0.0)
    if renormalize:
        s = g.sum(1, keepdim=True)
        g = g / torch.where(s > 0, s, 1.0)
    n = live.sum().clamp(min=1)
    share = counts.double() / counts.sum().clamp(min=1)
    return (g * dgates).sum() + balance * z.shape[1] * (share * p.sum(0)).sum() / n + zc * lse.square().sum() / n


def _check_grad(z, k, renormalize, balance=0.3, zc=0.05, dgates=True):
    T, E = z.shape
    got = _route(z, k, renormalize)
    d = torch.randn(T, k, generator=_gen(T), device=DEV) if dgates else None
    dz = _grad(z, got, d, balance, zc, renormalize)
    # the formula, and what each of its terms may be off by
    x = z.double()
    live = x.amax(1) > NEG
    lse = torch.where(live, torch.logsumexp(torch.where(live[:, None], x, 0.0), 1), 0.0)
    p = torch.where(live[:, None], (x - lse[:, None]).exp(), 0.0)
    n = int(live.sum()) or 1
    bal = balance * E / n * got["counts"].double() / max(1, int(got["counts"].sum()))
    dd = torch.where(got["chosen"] >= 0, d if dgates else 0.0, 0.0).double()
    at = got["chosen"].clamp(min=0).long()
    picked = torch.where(got["chosen"] >= 0, p.gather(1, at), 0.0)
    g, add, add_abs = bal.expand(T, E).clone(), torch.zeros(T, E, device=DEV, dtype=torch.float64), \
        torch.zeros(T, E, device=DEV, dtype=torch.float64)
    g_abs = g.abs()
    if renormalize:
        s = picked.sum(1, keepdim=True)
        w = picked / torch.where(s > 0, s, 1.0)
        add.scatter_add_(1, at, w * (dd - (w * dd).sum(1, keepdim=True)))
        add_abs.scatter_add_(1, at, w * (dd.abs() + (w * dd.abs()).sum(1, keepdim=True)))
    else:
        g.scatter_add_(1, at, dd)
        g_abs = g_abs.scatter_add(1, at, dd.abs())
    zt = (2 * zc / n * lse)[:, None]
    want = p * (g - (p * g).sum(1, keepdim=True) + zt) + add
    spread = min(110.0, float(torch.where(x > NEG, x.amax(1, keepdim=True) - x, 0.0).max()))
    off = (12 * spread + 256) * U * (p * (g_abs + (p * g_abs).sum(1, keepdim=True) + zt.abs()
                                          + abs(2 * zc / n) * (x.amax(1, keepdim=True).abs() * live[:, None]).nan_to_num(0.0, 0.0, 0.0))
                                     + add_abs)
    half = torch.finfo(z.dtype).eps / 2
    assert bool(((dz.double() - want).abs() <= off + half * (want.abs() + off) + 1e-38).all())
    return got, d, dz


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("experts,k", EXPERTS)
def test_grad_experts(experts, k, dtype):
    for tokens in (1, 33, 200):
        for renormalize in (False, True):
            _check_grad(_logits(experts, tokens, experts, dtype), k, renormalize)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [2, 63, 64, 65, 1000, 4097, 70001])
def test_grad_tokens(tokens, dtype):
    _check_grad(_logits(tokens, tokens, 64, dtype), 8, False)
    _check_grad(_logits(tokens, tokens, 10, dtype), 3, True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 8), (1, 5)])
def test_grad_strides_masks_and_parts(pad, shift, dtype):
    for experts in (64, 61, 300):
        z = _logits(8, 150, experts, dtype, pad, shift)
        z[:, 1::5] = NEG
        z[100:120] = NEG
        z[7, 2:] = NEG
        for renormalize in (False, True):
            got, d, dz = _check_grad(z, 6, renormalize)
            assert float(dz[100:120].abs().max()) == 0.0 and float(dz[:, 1::5].abs().max()) == 0.0
            wide = torch.full((150, experts + 5), 7.0, device=DEV, dtype=dtype)
            assert torch.equal(_grad(z, got, d, 0.3, 0.05, renormalize, out=wide[:, 2:2 + experts]), dz)
            assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + experts:] == 7).all())
            _check_grad(z, 6, renormalize, balance=0.0, zc=0.0)
            _check_grad(z, 6, renormalize, dgates=False)
    none = _grad(z, got, None, 0.0, 0.0, False)
    assert float(none.abs().max()) == 0.0


def test_grad_of_choices_out_of_range_and_listed_twice():
    z = _logits(9, 90, 20, F32)
    got = _route(z, 4)
    d = torch.randn(90, 4, generator=_gen(1), device=DEV)
    want = _grad(z, got, d, 0.0, 0.0, False)
    # twice the same expert: half the gradient each
    twice = dict(got, chosen=torch.cat([got["chosen"], got["chosen"]], 1))
    assert torch.equal(_grad(z, twice, torch.cat([d / 2, d / 2], 1), 0.0, 0.0, False), want)
    # no expert at all: as if the gate's gradient were zero
    odd = got["chosen"].clone()
    odd[:, 2] = torch.tensor([20, 1 << 30, -2, -(1 << 31), 21], dtype=torch.int32, device=DEV).repeat(18)
    d0 = d.clone()
    d0[:, 2] = 0
    for renormalize in (False, True):
        a = _grad(z, dict(got, chosen=odd), d, 0.1, 0.1, renormalize)
        keep = torch.where(odd < 20, odd.clamp(min=-1), -1)
        assert torch.equal(a, _grad(z, dict(got, chosen=keep), d, 0.1, 0.1, renormalize))
        if not renormalize:
            assert torch.equal(a, _grad(z, got, d0, 0.1, 0.1, False))


@pytest.mark.parametrize("renormalize", [False, True])
def test_grad_against_differences_and_the_differentiated_formula(renormalize):
    z = _logits(10, 40, 24, F32)
    z[5] = NEG
    z[:, 7] = NEG
    z[9, 3:] = NEG
    got, d, dz = _check_grad(z, 5, renormalize)
    args = got["chosen"], got["counts"], d.double(), 0.3, 0.05, renormalize
    x = z.double().clone().requires_grad_(True)
    _loss(x, *args).backward()
    # the finite entries' derivatives; the bound of _check_grad holds dz to 64 bits already
    ok = z > NEG
    assert bool(((dz.double() - x.grad)[ok].abs() <= 1e-4 * x.grad[ok].abs() + 1e-6).all())
    v, t = torch.randn(z.shape, generator=_gen(2), device=DEV, dtype=torch.float64), 1e-5
    v = torch.where(ok, v, 0.0)
    ends = [float(_loss(z.double() + s * v, *args)) for s in (t, -t)]
    want = float(torch.where(ok, dz.double() * v, 0.0).sum())
    assert abs((ends[0] - ends[1]) / (2 * t) - want) <= 1e-5 * float((dz.double() * v).abs().sum())


def test_grad_of_a_token_that_is_not_finite_stays_alone():
    z = _logits(11, 90, 20, F32)
    got = _route(z, 4)
    d = torch.randn(90, 4, generator=_gen(3), device=DEV)
    want = _grad(z, got, d, 0.1, 0.1, False)
    z[40, 6] = float("nan")
    dz = _grad(z, got, d, 0.1, 0.1, False)
    keep = torch.arange(90, device=DEV) != 40
    assert torch.equal(dz[keep], want[keep]) and bool(torch.isnan(dz[40]).all())


def test_streams_and_a_captured_graph():
    h = Handle.get()
    z = _logits(12, 700, 64, BF16)
    d = torch.randn(700, 8, generator=_gen(4), device=DEV)
    want = _route(z, 8, True)
    got = _route(z, 8, True, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    ws = torch.empty(mu.muon_router_workspace_size(h, z, 8), dtype=torch.uint8, device=DEV)
    out = {n: torch.zeros_like(t) for n, t in want.items()}
    dz = torch.zeros_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mu.muon_router_forward(h, z, workspace=ws, renormalize=True, **out)
        mu.muon_router_grad(h, z, out["chosen"], out["counts"], out["live"], dz, dgates=d, balance=0.1, z=0.1,
                            renormalize=True)
    for seed in (30, 31, 32):
        z.copy_(_logits(seed, 700, 64, BF16))
        z[600 + seed:] = NEG
        [t.zero_() for t in out.values()]
        dz.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = _route(z, 8, True)
        for n in want:
            assert torch.equal(out[n], want[n]), n
        assert torch.equal(dz, _grad(z, want, d, 0.1, 0.1, True))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("experts,k", [(8, 3), (20, 6), (61, 12), (100, 8), (200, 8), (300, 32), (1024, 20)])
def test_grad_of_the_gates_of_absent_choices_is_not_looked_at(experts, k, dtype):
    # a caller who fills dgates by `order` leaves anything where there is no choice
    z = _logits(13, 150, experts, dtype)
    z[::3, 2:] = NEG                       # fewer experts left than choices
    z[1::9] = NEG                          # padding
    got = _route(z, k)
    got["chosen"][2::5, 1] = experts + 3   # and choices out of range
    none = (got["chosen"] < 0) | (got["chosen"] >= experts)
    d = torch.randn(150, k, generator=_gen(6), device=DEV)
    for renormalize in (False, True):
        want = _grad(z, got, torch.where(none, 0.0, d), 0.1, 0.1, renormalize)
        assert bool(torch.isfinite(want).all())
        for value in (float("nan"), float("inf"), -float("inf"), 3e38):
            assert torch.equal(_grad(z, got, torch.where(none, value, d), 0.1, 0.1, renormalize), want)
