"""Global gradient norm and clip against 64-bit sums.

Tolerances: the squares are formed and summed in 64 bits, so the norm is off by
its own rounding to fp32, 2^-24 relative, and 64-bit errors far below 1e-9.
A clipped value is g * scale: scale and the fp32 product are rounded once each
(2^-24 both), a bf16 output once more (2^-8).  Values below the smallest normal
number are off by at most half their smallest step."""

import pytest
import torch

import muon_step_02_amd as mu
from harness import Handle

pytestmark = pytest.mark.gpu

DEV = "cuda"
NORM_TOL = 2.0 ** -24 + 1e-9


def _out_tol(dtype):
    return 2.0 ** -23 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) + 1e-9


def _workspace(h, plan):
    # no byte of it has to start at zero
    return torch.full((mu.muon_grad_workspace_size(h, plan),), 255, dtype=torch.uint8, device=DEV)


def _reference(grads, max_norm):
    norm = sum(float(g.double().square().sum()) for g in grads) ** 0.5
    return norm, (max_norm / norm if norm > max_norm else 1.0)


def _check_norm(got, want):
    assert abs(float(got) - want) <= NORM_TOL * want, (float(got), want)


def _check_outs(grads, outs, scale):
    for i, (g, o) in enumerate(zip(grads, outs)):
        want = g.double() * scale
        small = 2.0 ** -134 if o.dtype == torch.bfloat16 else 2.0 ** -149
        bad = (o.double() - want).abs() > _out_tol(o.dtype) * want.abs() + small
        assert not bool(bad.any()), (i, int(bad.sum()))


# shapes: (rows, cols, padding of the row) or a vector's length
SETS = {
    "one value": [1],
    "vectors": [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 255, 1000, 4096],
    "empty among them": [0, (0, 7, 0), 5, (3, 0, 2)],
    "odd rows": [(1, 1, 0), (3, 5, 0), (7, 33, 3), (64, 1, 1), (513, 3, 2), (5, 1025, 7), (2, 4097, 1)],
    "long rows": [(3, 70001, 8), 300000],
    "many short rows": [(9001, 2, 1), (40000, 9, 0), (1000, 300, 1)],
    "several chunks": [(512, 512, 0), (100, 4096, 8)],
    "more tensors than a launch holds": [7] * 300 + [(5, 6, 1)] * 300,
    "more chunks than blocks": [(4096, 4096, 0), (999, 8192, 8), 5],
}


def _make(shapes, dtype, seed, spread=3.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    grads, buffers = [], []
    for s in shapes:
        rows, cols, pad = s if isinstance(s, tuple) else (None, s, 0)
        n = cols if rows is None else rows * (cols + pad)
        b = torch.randn(n, generator=gen, device=DEV)
        b *= 10.0 ** float(torch.rand(1, generator=gen, device=DEV) * spread - spread / 2)
        b = b.to(dtype)
        buffers.append(b)
        grads.append(b if rows is None else b.view(rows, cols + pad)[:, :cols])
    return grads, buffers


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shapes", SETS.values(), ids=list(SETS))
def test_norm_and_clip(shapes, dtype):
    h = Handle.get()
    grads, buffers = _make(shapes, dtype, 3)
    kept = [b.clone() for b in buffers]
    norm, _ = _reference(grads, 1.0)
    for max_norm in (0.3 * norm, 2.0 * norm):
        _, scale = _reference(grads, max_norm)
        plan = [mu.muon_grad(g) for g in grads]
        got, factor = torch.full((2, 1), -1.0, device=DEV)
        mu.muon_grad_norm(h, plan, max_norm, _workspace(h, plan), norm_out=got, scale_out=factor)
        _check_norm(got, norm)
        assert abs(float(factor) - scale) <= NORM_TOL * scale
        assert float(factor) == 1.0 if scale == 1.0 else float(factor) < 1.0
        for out_dtype in (torch.float32, torch.bfloat16):
            outs, obufs = _make(shapes, out_dtype, 4)
            okept = [b.clone() for b in obufs]
            plan = [mu.muon_grad(g, o) for g, o in zip(grads, outs)]
            again, factor2 = torch.full((2, 1), -1.0, device=DEV)
            mu.muon_grad_clip(h, plan, max_norm, _workspace(h, plan), norm_out=again, scale_out=factor2)
            _check_outs(grads, outs, scale)
            _check_norm(again, norm)
            assert torch.equal(factor, factor2)
            for o, b, k in zip(outs, obufs, okept):  # the padding of the rows stays
                if o.dim() == 2 and o.shape[0] and b.numel() > o.numel():
                    pad = b.view(o.shape[0], -1)[:, o.shape[1]:]
                    assert torch.equal(pad, k.view(o.shape[0], -1)[:, o.shape[1]:])
    for b, k in zip(buffers, kept):
        assert torch.equal(b, k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shapes", [SETS["odd rows"], SETS["several chunks"], SETS["vectors"]],
                         ids=["odd rows", "several chunks", "vectors"])
def test_clip_in_place_equals_clip_to_another_tensor(shapes, dtype):
    h = Handle.get()
    grads, buffers = _make(shapes, dtype, 5)
    outs = [torch.empty_like(b).view(g.shape[0], -1)[:, :g.shape[1]] if g.dim() == 2 else torch.empty_like(b)
            for g, b in zip(grads, buffers)]
    norm, _ = _reference(grads, 1.0)
    plan = [mu.muon_grad(g, o) for g, o in zip(grads, outs)]
    ws = _workspace(h, plan)
    mu.muon_grad_clip(h, plan, 0.5 * norm, ws)
    before = [g.clone() for g in grads]
    plan = [mu.muon_grad(g, g) for g in grads]
    mu.muon_grad_clip(h, plan, 2.0 * norm, ws)
    for g, k in zip(grads, before):
        assert torch.equal(g, k)      # under the bound: not touched
    mu.muon_grad_clip(h, plan, 0.5 * norm, ws)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)


def test_column_blocks_of_one_tensor_are_clipped_in_place():
    h = Handle.get()
    t = torch.randn(257, 96, device=DEV)
    want = t.double()
    parts = [t[:, :33], t[:, 33:64], t[:, 64:]]
    norm = float(want.norm())
    plan = [mu.muon_grad(p, p) for p in parts]
    mu.muon_grad_clip(h, plan, norm / 3, _workspace(h, plan))
    assert float((t.double() - want / 3).abs().max()) <= 2.0 ** -22 * float(want.abs().max())


@pytest.mark.parametrize("value", [1e30, 3e38, 1e-30, 1e-42])
def test_no_gradient_is_too_large_or_too_small_for_its_square(value):
    h = Handle.get()
    g = torch.full((1000,), value, device=DEV)
    exact = g.double()
    plan = [mu.muon_grad(g, torch.empty_like(g))]
    norm, scale = torch.zeros(2, 1, device=DEV)
    out = torch.empty_like(g)
    plan = [mu.muon_grad(g, out)]
    want = float(exact.norm())
    mu.muon_grad_clip(h, plan, 1e-3, _workspace(h, plan), norm_out=norm, scale_out=scale)
    if want < 3.4e38:
        assert abs(float(norm) - want) <= NORM_TOL * want + 2.0 ** -150
    else:
        assert float(norm) == float("inf")      # beyond fp32, as the value it is rounded to
    if want > 1e-3:
        # the scale itself may lie below the smallest normal number
        step = 2.0 ** -149 * float(exact[0])
        assert abs(float(out[0]) - 1e-3 / 1000 ** 0.5) <= 2.0 ** -22 * 1e-3 + step
    else:
        assert torch.equal(out, g)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_gradients(bad):
    h = Handle.get()
    g = torch.ones(5000, device=DEV)
    g[4321] = bad
    out = torch.empty_like(g)
    norm, scale = torch.zeros(2, 1, device=DEV)
    plan = [mu.muon_grad(g, out)]
    mu.muon_grad_clip(h, plan, 1.0, _workspace(h, plan), norm_out=norm, scale_out=scale)
    rest = torch.arange(5000, device=DEV) != 4321
    if bad != bad:
        assert torch.isnan(norm) and float(scale) == 1.0 and bool((out[rest] == 1.0).all())
    else:
        assert float(norm) == float("inf") and float(scale) == 0.0 and bool((out[rest] == 0.0).all())
    assert torch.isnan(out[4321])


def test_a_tensor_listed_twice_counts_twice():
    h = Handle.get()
    g = torch.randn(777, device=DEV)
    norm = torch.zeros(1, device=DEV)
    plan = [mu.muon_grad(g), mu.muon_grad(g)]
    mu.muon_grad_norm(h, plan, 1.0, _workspace(h, plan), norm_out=norm)
    _check_norm(norm, 2 ** 0.5 * float(g.double().norm()))


def test_runs_are_bitwise_repeatable_and_streams_do_not_matter():
    h = Handle.get()
    grads, _ = _make(SETS["more chunks than blocks"], torch.float32, 8)
    plan = [mu.muon_grad(g) for g in grads]
    got = torch.zeros(4, device=DEV)
    spaces = [_workspace(h, plan) for _ in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(4):
        mu.muon_grad_norm(h, plan, 1.0, spaces[i], norm_out=got[i:i + 1], stream=streams[i % 2])
    torch.cuda.synchronize()
    assert bool((got == got[0]).all())


def test_offsets_beyond_32_bits():
    # more than 2^32 elements of bf16 in one tensor
    h = Handle.get()
    n = (1 << 32) + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g[7], g[(1 << 31) + 3], g[-1] = 3.0, 4.0, 12.0
    norm = torch.zeros(1, device=DEV)
    plan = [mu.muon_grad(g, g)]
    mu.muon_grad_clip(h, plan, 6.5, _workspace(h, plan), norm_out=norm)
    assert float(norm) == 13.0
    assert [float(g[i]) for i in (7, (1 << 31) + 3, n - 1)] == [1.5, 2.0, 6.0]
    assert int(torch.count_nonzero(g)) == 3


def test_binding_refuses():
    h = Handle.get()
    g = torch.zeros(8, device=DEV)
    plan = [mu.muon_grad(g)]
    ws = _workspace(h, plan)
    for norm in (torch.zeros(2, device=DEV), torch.zeros(1, device=DEV, dtype=torch.float64)):
        with pytest.raises(ValueError):
            mu.muon_grad_norm(h, plan, 1.0, ws, norm_out=norm)
    with pytest.raises(ValueError):
        mu.muon_grad_norm(h, plan, 1.0, ws.cpu(), norm_out=torch.zeros(1, device=DEV))
    with pytest.raises(mu.MuonError) as e:
        mu.muon_grad_norm(h, plan, 1.0, ws)
    assert e.value.status == 1
    with pytest.raises(mu.MuonError) as e:
        mu.muon_grad_clip(h, plan, 1.0, ws)       # no output
    assert e.value.status == 1
    with pytest.raises(mu.MuonError) as e:
        mu.muon_grad_norm(h, plan, 1.0, ws[:128], norm_out=torch.zeros(1, device=DEV))
    assert e.value.status == 3


def test_scalars_between_the_rows_of_a_gradient():
    """Padding belongs to no tensor: norm and scale may lie in it."""
    h = Handle.get()
    buf = torch.randn(300, 136, device=DEV)
    g = buf[:, :128]
    before = g.clone()
    norm, scale = _reference([before], 2.0)
    assert norm > 2.0
    plan = [mu.muon_grad(g, g)]
    mu.muon_grad_clip(h, plan, 2.0, _workspace(h, plan), norm_out=buf[0, 128:129], scale_out=buf[7, 135:136])
    _check_norm(buf[0, 128], norm)
    assert abs(float(buf[7, 135]) - scale) <= NORM_TOL * scale
    _check_outs([before], [g], scale)


# More tensors than a launch holds and more chunks than there are blocks (fp32
# 23 + 17 + 16 chunks of 16 KB each hundred times, bf16 12 + 9 + 8): the blocks
# go to the launches in proportion, and so do their partial sums.
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tensors_of_many_chunks(dtype):
    test_norm_and_clip([(130, 700, 4), 65537, (64, 1024, 0)] * 100, dtype)


@pytest.mark.parametrize("shapes", [[1 << 23], [70000] * 257, [1] * 600, [(130, 700, 4), 65537] * 300],
                         ids=["one tensor", "257 tensors", "600 values", "600 tensors"])
def test_the_workspace_is_as_large_as_its_size_says(shapes):
    h = Handle.get()
    grads, _ = _make(shapes, torch.float32, 6)
    plan = [mu.muon_grad(g) for g in grads]
    need = mu.muon_grad_workspace_size(h, plan)
    buf = torch.full((need + (1 << 16),), 0xA5, dtype=torch.uint8, device=DEV)
    norm = torch.zeros(1, device=DEV)
    mu.muon_grad_norm(h, plan, 1.0, buf[:need], norm_out=norm)
    _check_norm(norm, _reference(grads, 1.0)[0])
    assert bool((buf[need:] == 0xA5).all())


def test_both_types_in_one_call():
    """fp32 and bf16 gradients, outputs of either type and in place."""
    h = Handle.get()
    F32, BF16 = torch.float32, torch.bfloat16
    shapes = SETS["odd rows"] + SETS["vectors"] + SETS["several chunks"]
    grads, outs = [], []
    for i, s in enumerate(shapes):
        grads += _make([s], (F32, BF16)[i % 2], i)[0]
        outs += _make([s], (F32, BF16)[i // 2 % 2], 100 + i)[0]
    outs = [g if i % 5 == 0 else o for i, (g, o) in enumerate(zip(grads, outs))]
    before = [g.clone() for g in grads]
    norm, _ = _reference(before, 1.0)
    plan = [mu.muon_grad(g, o) for g, o in zip(grads, outs)]
    got = torch.zeros(1, device=DEV)
    mu.muon_grad_clip(h, plan, 0.3 * norm, _workspace(h, plan), norm_out=got)
    _check_norm(got, norm)
    _check_outs(before, outs, 0.3)
