"""A training step's end as a user runs it: the experts' products forward and
back, the weight gradients as Muon matrices, the largest logits for QK-Clip,
one gradient norm over Muon and AdamW tensors, and both steps with its scale.
Eager, and captured in a graph."""

import numpy as np
import pytest
import torch

import muon_step_02_amd as mu
import oracle
import synth
from harness import Handle, TOL_O_BF16, TOL_O_F32, TOL_STATE, f64, hp_from, oracle_kwargs, recipe_floor_output, relF

pytestmark = pytest.mark.gpu

DEV = "cuda"
E, N, K, T = 4, 256, 384, 500
HEADS, HEAD, D_MODEL = 4, 64, 256


class Step:
    """One layer: experts' weights (N x K) and a query projection on Muon, a
    norm weight on AdamW."""

    def __init__(self, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def rnd(*s, dtype=torch.float32, std=1.0):
            return (torch.randn(*s, generator=g, device=DEV) * std).to(dtype)

        self.h = Handle.get()
        self.W = rnd(E, N, K, std=0.02)                     # fp32 masters, bf16 for the products
        self.Wb = self.W.to(torch.bfloat16)
        self.G = torch.zeros(E, N, K, device=DEV)
        self.M = torch.zeros(E, N, K, device=DEV)
        self.wq, self.gq, self.mq = rnd(HEADS * HEAD, D_MODEL, std=0.02), rnd(HEADS * HEAD, D_MODEL), \
            torch.zeros(HEADS * HEAD, D_MODEL, device=DEV)
        self.p, self.gp = rnd(1000), rnd(1000, std=3.0)
        self.m, self.v = torch.zeros(1000, device=DEV), torch.zeros(1000, device=DEV)
        self.x, self.dy = rnd(T, K, dtype=torch.bfloat16), rnd(T, N, dtype=torch.bfloat16)
        self.y, self.dx = torch.zeros_like(self.dy), torch.zeros_like(self.x)
        self.offsets = torch.tensor([0, 130, 130, 400, T], dtype=torch.int32, device=DEV)
        self.q, self.k = (rnd(90, HEADS, HEAD, dtype=torch.bfloat16, std=4.0) for _ in range(2))
        self.cu = torch.tensor([0, 40, 90], dtype=torch.int32, device=DEV)
        self.smax = torch.zeros(HEADS, device=DEV)
        self.norm, self.scale = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
        self.experts, self.dw = mu.muon_experts(list(self.Wb)), mu.muon_experts(list(self.G))
        self.grads = [mu.muon_grad(t) for t in list(self.G) + [self.gq, self.gp]]
        self.O = torch.zeros(E, N, K, device=DEV)
        self.mats = [mu.muon_matrix(*t) for t in zip(self.W, self.G, self.M, self.O)]
        self.mats.append(mu.muon_matrix(self.wq, self.gq, self.mq, qk_smax=self.smax, qk_block_rows=HEAD))
        self.hp = hp_from(synth.MUON_DEFAULT)
        self.hp.qk_tau = 20.0
        self.ahp = mu.adamw_hparams(step=1, **synth.ADAMW_DEFAULT)
        self.ts = [mu.adamw_tensor(self.p, self.gp, self.m, self.v)]

        def space(n):
            return torch.empty(n, dtype=torch.uint8, device=DEV)

        self.ws = space(mu.muon_workspace_size(self.h, self.mats, self.hp))
        self.ws_g = space(mu.muon_grad_workspace_size(self.h, self.grads))
        self.ws_s = space(mu.muon_qk_smax_workspace_size(self.h, self.q, self.k, self.cu))

    def __call__(self):
        h = self.h
        mu.muon_expert_forward(h, self.experts, self.offsets, self.x, self.y)
        mu.muon_expert_grad_input(h, self.experts, self.offsets, self.dy, self.dx)
        mu.muon_expert_grad_weight(h, self.dw, self.offsets, self.x, self.dy)
        mu.muon_qk_smax(h, self.q, self.k, self.cu, self.cu, self.smax, self.ws_s, scale=1.0 / 8)
        mu.muon_grad_norm(h, self.grads, 1.0, self.ws_g, norm_out=self.norm, scale_out=self.scale)
        mu.muon_step_batched_scaled(h, self.mats, self.hp, self.scale, self.ws)
        mu.adamw_step_scaled(h, self.ts, self.ahp, self.scale)

    def state(self):
        return dict(W=self.W, M=self.M, G=self.G, wq=self.wq, mq=self.mq, p=self.p, m=self.m, v=self.v,
                    y=self.y, dx=self.dx, smax=self.smax, norm=self.norm, scale=self.scale)


def test_step_against_the_oracle():
    s = Step()
    W0, wq0, p0 = f64(s.W), f64(s.wq), f64(s.p)
    s()
    torch.cuda.synchronize()
    at = s.offsets.tolist()
    # the gradients: fp32 sums of at most 270 products each (as in the products' own test)
    x, dy = f64(s.x), f64(s.dy)
    G = [dy[a:b].T @ x[a:b] for a, b in zip(at, at[1:])]
    for e in range(E):
        assert relF(f64(s.G[e]), G[e]) <= 272 * 2.0 ** -23
    assert float(torch.count_nonzero(s.G[1])) == 0
    # one norm over all of it
    gs = [f64(g) for g in s.G] + [f64(s.gq), f64(s.gp)]
    clipped, norm = oracle.clip_by_global_norm(gs, 1.0)
    assert norm > 1.0 and abs(float(s.norm) - norm) <= (2.0 ** -24 + 1e-9) * norm
    kw = oracle_kwargs(synth.MUON_DEFAULT)
    for e in (0, 2, 3):
        W, M, O = oracle.muon_matrix_step(W0[e], clipped[e], np.zeros((N, K)), **kw)
        assert relF(f64(s.M[e]), M) <= TOL_STATE
        # A gradient of 100 or 130 tokens has rank 100 or 130 of 256: its other
        # singular values are zero, and a rounding of X_k (relative 2^-8 at
        # most, 2^-8 / sqrt(3) in the mean square) in their directions grows by
        # a = 3.4445 in every iteration left.  ||X_k|| <= a^k, so each of the
        # six X_k and five B_k adds up to a^5 2^-8 / sqrt(3) = 1.1, beside
        # ||O|| of about sqrt(rank) = 10: the usual 3e-2 is for gradients of
        # full rank.  A plain bf16 implementation of the method rounds all of
        # these and six more tensors an iteration: its error on the same input
        # is the bound.
        floor = relF(recipe_floor_output(clipped[e]), O)
        assert relF(f64(s.O[e]), O) <= max(TOL_O_BF16, floor), (e, floor)
    # the empty expert only decays
    assert relF(f64(s.W[1]), W0[1] * (1.0 - kw["lr"] * kw["weight_decay"])) <= 2.0 ** -22
    th, m, v = oracle.adamw_tensor_step(p0, clipped[-1], np.zeros(1000), np.zeros(1000), step=1,
                                        **synth.ADAMW_DEFAULT)
    assert relF(f64(s.m), m) <= TOL_STATE and relF(f64(s.v), v) <= TOL_STATE
    assert relF(f64(s.p), th) <= TOL_STATE
    # the logits the query projection's heads are clipped by
    q, k = f64(s.q), f64(s.k)
    top = np.full(HEADS, -np.inf)
    for a, b in ((0, 40), (40, 90)):
        for h in range(HEADS):
            z = q[a:b, h] @ k[a:b, h].T / 8
            top[h] = max(top[h], z[np.tril(np.ones_like(z, dtype=bool))].max())
    assert np.abs(f64(s.smax) - top).max() <= 65 * 2.0 ** -23 * np.abs(q).max() * np.abs(k).max() * 64 / 8
    assert top.max() > 20.0
    Wq, _, _ = oracle.muon_matrix_step(wq0, clipped[E], np.zeros_like(wq0), **kw)
    factor = np.sqrt(np.minimum(1.0, 20.0 / top)).repeat(HEAD)[:, None]
    # the update's own tolerance, on a step of lr * 0.2 * sqrt(256) * O
    step = kw["lr"] * 0.2 * 16.0 * np.sqrt(HEADS * HEAD)
    assert np.linalg.norm(f64(s.wq) - Wq * factor) <= TOL_O_BF16 * step + 2e-6 * np.linalg.norm(Wq)


def test_scaled_steps_equal_steps_on_clipped_gradients():
    """The fused clip against clipping first: fp32 gradients clipped to fp32
    hold the same products, so every bit agrees."""
    a, b = Step(3), Step(3)
    a()
    torch.cuda.synchronize()
    mu.muon_expert_grad_weight(b.h, b.dw, b.offsets, b.x, b.dy)
    mu.muon_qk_smax(b.h, b.q, b.k, b.cu, b.cu, b.smax, b.ws_s, scale=1.0 / 8)
    plan = [mu.muon_grad(t, t) for t in list(b.G) + [b.gq, b.gp]]
    mu.muon_grad_clip(b.h, plan, 1.0, b.ws_g, norm_out=b.norm, scale_out=b.scale)
    mu.muon_step_batched(b.h, b.mats, b.hp, b.ws)
    mu.adamw_step(b.h, b.ts, b.ahp)
    torch.cuda.synchronize()
    for name in ("W", "M", "wq", "mq", "p", "m", "v", "norm", "scale"):
        assert torch.equal(a.state()[name], b.state()[name]), name


def test_a_scale_of_one_changes_nothing():
    a, b = Step(4), Step(4)
    one = torch.ones(1, device=DEV)
    for s in (a, b):
        mu.muon_expert_grad_weight(s.h, s.dw, s.offsets, s.x, s.dy)
    mu.muon_step_batched_scaled(a.h, a.mats, a.hp, one, a.ws)
    mu.adamw_step_scaled(a.h, a.ts, a.ahp, one)
    mu.muon_step_batched(b.h, b.mats, b.hp, b.ws)
    mu.adamw_step(b.h, b.ts, b.ahp)
    torch.cuda.synchronize()
    for name in ("W", "M", "wq", "mq", "p", "m", "v"):
        assert torch.equal(a.state()[name], b.state()[name]), name


def test_captured_step_replays_as_the_eager_one():
    a, b = Step(5), Step(5)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        a()
    for r in range(4):
        g.replay()
        b()
        torch.cuda.synchronize()
        for name, t in a.state().items():
            assert torch.equal(t, b.state()[name]), (r, name)
        for s in (a, b):  # other tokens, groups and queries for the next one
            s.x.mul_(-0.5)
            s.q.add_(0.25)
            s.offsets.copy_(torch.tensor([0, 10 * r, 200, 200, T - r], dtype=torch.int32))
        torch.cuda.synchronize()


def test_two_handles_and_two_streams():
    a, b = Step(6), Step(6)
    b.h = mu.muon_init(0)
    try:
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            a()
        with torch.cuda.stream(s2):
            b()
        torch.cuda.synchronize()
        for name, t in a.state().items():
            assert torch.equal(t, b.state()[name]), name
    finally:
        mu.muon_destroy(b.h)


def test_a_scale_beside_what_the_steps_write():
    """Behind a parameter's last value, and in the padding of a momentum's rows:
    it belongs to no tensor there."""
    a, b = Step(7), Step(7)
    for s in (a, b):
        mu.muon_expert_grad_weight(s.h, s.dw, s.offsets, s.x, s.dy)
    scale = torch.full((1,), 0.25, device=DEV)
    p = torch.zeros(1001, device=DEV)
    p[:1000], p[1000] = a.p, 0.25
    mu.adamw_step_scaled(a.h, [mu.adamw_tensor(p[:1000], a.gp, a.m, a.v)], a.ahp, p[1000:])
    mom = torch.zeros(N, K + 4, device=DEV)
    mom[5, K + 1] = 0.25
    mats = [mu.muon_matrix(a.W[0], a.G[0], mom[:, :K], a.O[0])]
    mu.muon_step_batched_scaled(a.h, mats, a.hp, mom[5, K + 1:K + 2], a.ws)
    mu.adamw_step_scaled(b.h, b.ts, b.ahp, scale)
    mu.muon_step_batched_scaled(b.h, b.mats[:1], b.hp, scale, b.ws)
    torch.cuda.synchronize()
    assert torch.equal(p[:1000], b.p) and torch.equal(a.m, b.m) and torch.equal(a.v, b.v)
    assert torch.equal(a.W[0], b.W[0]) and torch.equal(mom[:, :K], b.M[0])
    assert float(mom[5, K + 1]) == 0.25 and float(p[1000]) == 0.25


@pytest.mark.parametrize("ns_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("grad_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("pad", [0, 4, 3])
def test_scaled_steps_of_every_layout(pad, grad_dtype, ns_dtype):
    """Wide and tall matrices, padded rows that vector accesses fit and that they
    do not: a scaled step against the oracle's step on scaled gradients."""
    g = torch.Generator(device=DEV).manual_seed(11)
    scale = torch.full((1,), 0.3, device=DEV)
    s64 = float(scale.double())
    hp = hp_from(synth.MUON_DEFAULT, ns_dtype=ns_dtype)
    shapes, mats, held = [(96, 200), (200, 96), (160, 416), (416, 160), (8, 24)], [], []

    def tensor(r, c, dtype=torch.float32, std=1.0):
        return (torch.randn(r, c + pad, generator=g, device=DEV) * std).to(dtype)[:, :c]

    for r, c in shapes:
        W, G, M = tensor(r, c, std=0.02), tensor(r, c, grad_dtype), tensor(r, c, std=0.1)
        O = torch.zeros(r, c, device=DEV)
        held.append((W, G, M, O, f64(W), f64(G), f64(M)))
        mats.append(mu.muon_matrix(W, G, M, O))
    h = Handle.get()
    ws = torch.empty(mu.muon_workspace_size(h, mats, hp), dtype=torch.uint8, device=DEV)
    mu.muon_step_batched_scaled(h, mats, hp, scale, ws)
    n = 4097 + pad
    p, pg = torch.randn(n + 1, generator=g, device=DEV)[1:], torch.randn(n + 1, generator=g, device=DEV).to(grad_dtype)[1:]
    p0 = f64(p)
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    mu.adamw_step_scaled(h, [mu.adamw_tensor(p, pg, m, v)], mu.adamw_hparams(step=1, **synth.ADAMW_DEFAULT), scale)
    torch.cuda.synchronize()
    kw = oracle_kwargs(synth.MUON_DEFAULT)
    for W, G, M, O, W0, G0, M0 in held:
        Wr, Mr, Or = oracle.muon_matrix_step(W0, G0 * s64, M0, **kw)
        # three roundings of 2^-24 beside the unscaled step's
        assert relF(f64(M), Mr) <= TOL_STATE, W.shape
        # 8 x 24 runs in fp32 in either mode
        assert relF(f64(O), Or) <= (TOL_O_F32 if ns_dtype == "fp32" else TOL_O_BF16), W.shape
    th, mr, vr = oracle.adamw_tensor_step(p0, f64(pg) * s64, np.zeros(n), np.zeros(n), step=1, **synth.ADAMW_DEFAULT)
    assert relF(f64(m), mr) <= TOL_STATE and relF(f64(v), vr) <= TOL_STATE and relF(f64(p), th) <= TOL_STATE
