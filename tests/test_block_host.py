"""Operators around the products and the logits (layer norm, rotary positions,
router): what their entry points refuse, the layout of their structures, and
the rotary frequencies.  No GPU: every refusal comes before a call touches a
device, so a zeroed block of memory stands in for the handle."""

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import muon_step_02_amd as mu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, WORKSPACE, OVERLAP, UNALIGNED = 0, 1, 3, 4, 6
BUF = 1 << 24  # an address for tensors that no call gets to read, and the room between two of them


@pytest.fixture(scope="module")
def lib():
    return mu.load()


@pytest.fixture(scope="module")
def handle():
    return ctypes.cast(ctypes.create_string_buffer(4096), ctypes.c_void_p)


def test_structures_match_the_header(tmp_path):
    structs = {"muon_heads": mu.MuonHeads, "muon_layernorm": mu.MuonLayernorm, "muon_rotary_plan": mu.MuonRotaryPlan,
               "muon_positions": mu.MuonPositions, "muon_router": mu.MuonRouter, "muon_routing": mu.MuonRouting}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "muon.h"', "int main(void){"]
    for name, cls in structs.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f) for f, _ in cls._fields_]
    c, exe = tmp_path / "s.c", tmp_path / "s"
    c.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {k: int(v) for k, v in (line.split() for line in out.splitlines())}
    for name, cls in structs.items():
        assert got[name] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got["%s.%s" % (name, f)] == getattr(cls, f).offset, (name, f)


def _heads(at, token=64, head=16, heads=4):
    return mu.MuonHeads(at, token, head, heads)


# ---- layer norm ----------------------------------------------------------------

def _norm(**over):
    d = dict(weight=5 * BUF, bias=6 * BUF, tokens=10, cols=16, dtype=0, weight_dtype=0, center=1, eps=1e-5)
    d.update(over)
    return mu.MuonLayernorm(**d)


def _forward(lib, h, n=None, x=None, y=None, mean=7 * BUF, rstd=8 * BUF):
    return lib.muon_layernorm_forward(h, n or _norm(), x or _heads(BUF), y or _heads(2 * BUF), mean, rstd, None)


def _grad(lib, h, n=None, x=None, dy=None, dx=True, mean=7 * BUF, rstd=8 * BUF, dw=9 * BUF, db=10 * BUF, dtype=0,
          acc=0, ws=11 * BUF, nbytes=0):
    # (no workspace: a call that is refused for nothing else is refused for that)
    dx = _heads(3 * BUF) if dx is True else dx
    return lib.muon_layernorm_grad(h, n or _norm(), x or _heads(BUF), dy or _heads(2 * BUF), mean, rstd, dx, dw, db,
                                   dtype, acc, ws, nbytes, None)


SIZES = [dict(tokens=-1), dict(tokens=1 << 31), dict(cols=0), dict(cols=16385), dict(dtype=2), dict(weight_dtype=-1),
         dict(center=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))]


@pytest.mark.parametrize("over", SIZES)
def test_norm_sizes_refused(lib, handle, over):
    assert _forward(lib, handle, _norm(**over)) == INVALID
    assert _grad(lib, handle, _norm(**over)) == INVALID
    sz = ctypes.c_size_t()
    assert lib.muon_layernorm_workspace_size(handle, _norm(**over), 4, sz) == INVALID


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=-1), dict(token=-1), dict(head=-16), dict(token=1 << 41),
                                 dict(head=1 << 41), dict(token=1 << 39), dict(at=None)])
def test_norm_strides_refused(lib, handle, bad):
    x = _heads(**dict(dict(at=BUF), **bad))
    assert _forward(lib, handle, x=x) == INVALID
    assert _grad(lib, handle, x=x) == INVALID
    if "heads" not in bad:
        assert _forward(lib, handle, y=x) == INVALID
        assert _grad(lib, handle, dy=x) == INVALID
        assert _grad(lib, handle, dx=x) == INVALID


def test_norm_outputs_may_not_share_their_own_elements(lib, handle):
    for y in (_heads(2 * BUF, token=0), _heads(2 * BUF, token=63), _heads(2 * BUF, head=15), _heads(2 * BUF, head=0),
              _heads(2 * BUF, token=16, head=159), _heads(2 * BUF, token=15, head=160)):
        assert _forward(lib, handle, y=y) == INVALID
        assert _grad(lib, handle, dx=y) == INVALID
        assert _grad(lib, handle, dy=y) == WORKSPACE  # to read, they may
    # heads before tokens
    assert _grad(lib, handle, dx=_heads(3 * BUF, token=16, head=160)) == WORKSPACE


def test_norm_arguments_refused(lib, handle):
    assert _forward(lib, None) == INVALID and _grad(lib, None) == INVALID
    assert lib.muon_layernorm_forward(handle, None, _heads(BUF), _heads(2 * BUF), None, None, None) == INVALID
    assert lib.muon_layernorm_forward(handle, _norm(), None, _heads(2 * BUF), None, None, None) == INVALID
    assert lib.muon_layernorm_forward(handle, _norm(), _heads(BUF), None, None, None, None) == INVALID
    assert _forward(lib, handle, y=_heads(2 * BUF, heads=3)) == INVALID
    assert _grad(lib, handle, dy=_heads(2 * BUF, heads=3)) == INVALID
    assert _grad(lib, handle, dx=_heads(3 * BUF, heads=3)) == INVALID
    assert _grad(lib, handle, dx=None, dw=None, db=None) == INVALID
    assert _grad(lib, handle, rstd=None) == INVALID
    assert _grad(lib, handle, mean=None) == INVALID
    assert _grad(lib, handle, _norm(center=0), mean=None) == WORKSPACE
    assert _grad(lib, handle, dtype=2) == INVALID
    assert _grad(lib, handle, acc=2) == INVALID
    assert _grad(lib, handle, dx=None) == WORKSPACE
    assert _grad(lib, handle, nbytes=1 << 20, ws=None) == WORKSPACE
    assert _grad(lib, handle, nbytes=1 << 20, ws=11 * BUF + 128) == WORKSPACE


def test_norm_alignment_refused(lib, handle):
    for kw in (dict(x=_heads(BUF + 2)), dict(y=_heads(2 * BUF + 1)), dict(mean=7 * BUF + 2), dict(rstd=8 * BUF + 1),
               dict(n=_norm(weight=5 * BUF + 2)), dict(n=_norm(bias=6 * BUF + 1, weight_dtype=1))):
        assert _forward(lib, handle, **kw) == UNALIGNED
    for kw in (dict(x=_heads(BUF + 2)), dict(dy=_heads(2 * BUF + 1)), dict(dx=_heads(3 * BUF + 2)),
               dict(mean=7 * BUF + 2), dict(rstd=8 * BUF + 1), dict(dw=9 * BUF + 2), dict(db=10 * BUF + 1, dtype=1)):
        assert _grad(lib, handle, **kw) == UNALIGNED


def test_norm_overlaps_refused(lib, handle):
    bytes_ = 10 * 64 * 4
    for kw in (dict(y=_heads(BUF + 64)), dict(y=_heads(BUF, token=80)), dict(y=_heads(5 * BUF)), dict(y=_heads(6 * BUF)),
               dict(y=_heads(7 * BUF)), dict(mean=BUF + bytes_ - 4), dict(rstd=7 * BUF + 4), dict(rstd=5 * BUF)):
        assert _forward(lib, handle, **kw) == OVERLAP, kw
    size = 1 << 20
    for kw in (dict(dx=_heads(BUF + 64)), dict(dx=_heads(2 * BUF + 64)), dict(dx=_heads(5 * BUF)), dict(dw=10 * BUF),
               dict(dw=5 * BUF), dict(db=8 * BUF), dict(ws=BUF), dict(ws=9 * BUF), dict(dw=BUF), dict(dx=_heads(8 * BUF)),
               # x in place, but dy elsewhere within it
               dict(dx=_heads(BUF), dy=_heads(BUF + 64))):
        assert _grad(lib, handle, nbytes=size, **kw) == OVERLAP, kw
    # without center the mean is not read
    assert _grad(lib, handle, _norm(center=0), dx=_heads(7 * BUF), dw=7 * BUF, nbytes=size) == OVERLAP


def test_norm_without_rows_is_done(lib, handle):
    assert _forward(lib, handle, _norm(tokens=0), x=_heads(None), y=_heads(None)) == OK


@pytest.mark.parametrize("tokens,heads", [(100000, 1), (2, 1), (1, 4000), (50, 40)])
def test_norm_rows_that_are_one_take_the_bytes_of_one(lib, handle, tokens, heads):
    # (a handle of zeroes has no compute units: a call that is not refused launches no workgroup)
    n, row, need = _norm(tokens=tokens, weight=None, bias=None), 64 * BUF, ctypes.c_size_t()
    assert lib.muon_layernorm_workspace_size(handle, n, heads, need) == OK
    out = tokens * heads * 16 * 4

    def one(at):
        return mu.MuonHeads(at, 0, 16 if heads == 1 else 0, heads)

    def many(at):
        return mu.MuonHeads(at, heads * 16, 16, heads)

    def forward(at):
        return lib.muon_layernorm_forward(handle, n, one(row), many(at), None, None, None) == OVERLAP

    def back(at):
        # x is one row, and dy another one 64 bytes behind it
        return lib.muon_layernorm_grad(handle, n, one(row), one(row + 64), BUF, BUF, many(at), None, None, 0, 0, 2 * BUF,
                                       need.value, None) == OVERLAP

    assert not forward(row + 64) and not forward(row + 256) and not forward(row - out)
    assert forward(row) and forward(row + 60) and forward(row - out + 4)
    assert not back(row + 128) and not back(row + 1024) and not back(row - out)
    assert back(row) and back(row + 64) and back(row + 124) and back(row - out + 4)


# ---- rotary positions -------------------------------------------------------------

def _turn(**over):
    d = dict(positions=8 * BUF, frequencies=9 * BUF, tokens=10, head_dim=16, first=0, pairs=8, interleaved=0, dtype=0,
             scale=1.0)
    d.update(over)
    return mu.MuonPositions(**d)


def _rotary(lib, h, p=None, x=None, y=None, transpose=0, n=None):
    x, y = x or [_heads(BUF)], y or [_heads(2 * BUF)]
    a = mu.MuonHeads * max(len(x), 1)
    return lib.muon_rotary(h, p or _turn(), a(*x), a(*y), len(x) if n is None else n, transpose, None)


@pytest.mark.parametrize("over", [dict(tokens=-1), dict(tokens=1 << 31), dict(head_dim=0), dict(head_dim=65537),
                                  dict(pairs=0), dict(pairs=-1), dict(pairs=9), dict(first=1), dict(first=-1),
                                  dict(first=2, pairs=8), dict(dtype=2), dict(interleaved=2), dict(positions=None),
                                  dict(frequencies=None), dict(scale=float("nan")), dict(scale=float("inf")),
                                  dict(head_dim=8192, pairs=2049)])
def test_rotary_sizes_refused(lib, handle, over):
    assert _rotary(lib, handle, _turn(**over)) == INVALID


def test_rotary_arguments_refused(lib, handle):
    assert _rotary(lib, None) == INVALID
    assert lib.muon_rotary(handle, None, _heads(BUF), _heads(2 * BUF), 1, 0, None) == INVALID
    assert lib.muon_rotary(handle, _turn(), None, _heads(2 * BUF), 1, 0, None) == INVALID
    assert lib.muon_rotary(handle, _turn(), _heads(BUF), None, 1, 0, None) == INVALID
    assert _rotary(lib, handle, n=0) == INVALID
    assert _rotary(lib, handle, x=[_heads(BUF)] * 5, y=[_heads(2 * BUF)] * 5) == INVALID
    assert _rotary(lib, handle, transpose=2) == INVALID
    assert _rotary(lib, handle, y=[_heads(2 * BUF, heads=3)]) == INVALID
    assert _rotary(lib, handle, x=[_heads(BUF, heads=65537)], y=[_heads(2 * BUF, heads=65537, token=1 << 21)]) == INVALID
    for bad in (_heads(None), _heads(2 * BUF, token=63), _heads(2 * BUF, head=15), _heads(2 * BUF, heads=0)):
        assert _rotary(lib, handle, y=[bad]) == INVALID
    assert _rotary(lib, handle, x=[_heads(BUF + 2)]) == UNALIGNED
    assert _rotary(lib, handle, y=[_heads(2 * BUF + 2)]) == UNALIGNED
    assert _rotary(lib, handle, _turn(positions=8 * BUF + 2)) == UNALIGNED
    assert _rotary(lib, handle, _turn(frequencies=9 * BUF + 4)) == UNALIGNED
    assert _rotary(lib, handle, _turn(tokens=0, positions=None), x=[_heads(None)], y=[_heads(None)]) == OK


def test_rotary_overlaps_refused(lib, handle):
    for y in (_heads(BUF + 64), _heads(BUF, token=80), _heads(8 * BUF), _heads(9 * BUF)):
        assert _rotary(lib, handle, y=[y]) == OVERLAP
    # one tensor into another's input, or two into one
    assert _rotary(lib, handle, x=[_heads(BUF), _heads(3 * BUF)], y=[_heads(3 * BUF), _heads(4 * BUF)]) == OVERLAP
    assert _rotary(lib, handle, x=[_heads(BUF), _heads(3 * BUF)], y=[_heads(2 * BUF), _heads(2 * BUF)]) == OVERLAP
    assert _rotary(lib, handle, x=[_heads(BUF), _heads(BUF)], y=[_heads(BUF), _heads(BUF)]) == OVERLAP
    # a call whose grid no launch holds: nothing else is wrong with it
    wide = 65536
    big = _turn(tokens=1 << 16, head_dim=64, pairs=32)
    x, y = (_heads(at, token=wide * 64, head=64, heads=wide) for at in (1 << 42, 1 << 44))
    assert _rotary(lib, handle, big, x=[x], y=[y]) == INVALID


def test_rotary_heads_that_are_one_take_the_bytes_of_one(lib, handle):
    # a call whose grid no launch holds is refused for that, behind the check for overlaps
    wide, row = 65536, 1 << 42
    p = _turn(tokens=1 << 20, head_dim=wide, pairs=8)

    def turn(at):
        return _rotary(lib, handle, p, x=[mu.MuonHeads(row, 0, wide, 1)], y=[mu.MuonHeads(at, wide, wide, 1)])

    assert turn(row + 4 * wide) == INVALID and turn(row - (4 * wide << 20)) == INVALID
    for at in (row, row + 4 * wide - 4, row - (4 * wide << 20) + 4):
        assert turn(at) == OVERLAP


def test_frequencies_against_their_formulas():
    for n in (1, 17, 64):
        i = np.arange(n) / n
        np.testing.assert_allclose(mu.muon_rotary_frequencies(n).numpy(), 10000.0 ** -i, rtol=1e-14)
        np.testing.assert_allclose(mu.muon_rotary_frequencies(n, base=5e5, scaling="linear", factor=4.0).numpy(),
                                   5e5 ** -i / 4.0, rtol=1e-14)
        f = mu.muon_rotary_frequencies(n, scaling="parts", factor=8.0, context=4096.0, low=1.0, high=4.0).numpy()
        turns = 4096.0 * 10000.0 ** -i / (2.0 * math.pi)
        for t, got, plain in zip(turns, f, 10000.0 ** -i):
            if t >= 4.0:
                assert got == pytest.approx(plain, rel=1e-14)
            elif t <= 1.0:
                assert got == pytest.approx(plain / 8.0, rel=1e-14)
            else:
                assert plain / 8.0 <= got <= plain
                k = (t - 1.0) / 3.0
                assert got == pytest.approx(plain * (k + (1.0 - k) / 8.0), rel=1e-13)
    f = mu.muon_rotary_frequencies(64, scaling="base", factor=8.0).numpy()
    assert f[0] == 1.0 and f[-1] == pytest.approx(10000.0 ** (-63 / 64) / 8.0, rel=1e-13)


@pytest.mark.parametrize("kw", [dict(pairs=0), dict(pairs=2049), dict(base=0.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.0), dict(scaling="base", pairs=1, factor=2.0),
                                dict(scaling="parts", factor=2.0, context=0.0),
                                dict(scaling="parts", factor=2.0, context=9.0, low=4.0, high=4.0),
                                dict(scaling="parts", factor=2.0, context=9.0, high=float("inf"))])
def test_frequencies_refused(kw):
    kw = dict(dict(pairs=8), **kw)
    with pytest.raises(mu.MuonError) as e:
        mu.muon_rotary_frequencies(kw.pop("pairs"), **kw)
    assert e.value.status == INVALID


# ---- router --------------------------------------------------------------------------

def _router(**over):
    d = dict(logits=BUF, tokens=10, ld=16, experts=16, top_k=4, dtype=0, renormalize=0)
    d.update(over)
    return mu.MuonRouter(**d)


def _route(lib, h, r=None, ws=12 * BUF, nbytes=1 << 20, **over):
    d = dict(chosen=2 * BUF, gates=3 * BUF, counts=4 * BUF, offsets=5 * BUF, rows=6 * BUF, order=7 * BUF, live=8 * BUF,
             losses=9 * BUF)
    d.update(over)
    return lib.muon_router_forward(h, r or _router(), mu.MuonRouting(**d), ws, nbytes, None)


def _route_grad(lib, h, r=None, chosen=2 * BUF, counts=4 * BUF, live=8 * BUF, dgates=9 * BUF, balance=0.0, z=0.0,
                dlogits=10 * BUF, ld=16):
    return lib.muon_router_grad(h, r or _router(), chosen, counts, live, dgates, balance, z, dlogits, ld, None)


@pytest.mark.parametrize("over", [dict(tokens=-1), dict(tokens=(1 << 28) + 1), dict(experts=0), dict(experts=1025, ld=1025),
                                  dict(top_k=0), dict(top_k=17), dict(experts=64, ld=64, top_k=33), dict(ld=15),
                                  dict(ld=1 << 41), dict(tokens=1 << 20, ld=1 << 30), dict(dtype=2), dict(renormalize=2)])
def test_router_sizes_refused(lib, handle, over):
    assert _route(lib, handle, _router(**over)) == INVALID
    assert _route_grad(lib, handle, _router(**over)) == INVALID
    sz = ctypes.c_size_t()
    assert lib.muon_router_workspace_size(handle, _router(**over), sz) == INVALID


def test_router_arguments_refused(lib, handle):
    assert _route(lib, None) == INVALID and _route_grad(lib, None) == INVALID
    assert lib.muon_router_forward(handle, _router(), None, 12 * BUF, 1 << 20, None) == INVALID
    assert lib.muon_router_forward(handle, None, mu.MuonRouting(), 12 * BUF, 1 << 20, None) == INVALID
    for name in ("chosen", "gates", "counts", "offsets"):
        assert _route(lib, handle, **{name: None}) == INVALID
    assert _route(lib, handle, _router(logits=None)) == INVALID
    for name in ("chosen", "gates", "counts", "offsets", "rows", "order", "live", "losses"):
        assert _route(lib, handle, **{name: 2 * BUF + 2}) == UNALIGNED
    assert _route(lib, handle, _router(logits=BUF + 2)) == UNALIGNED
    assert _route(lib, handle, ws=None) == WORKSPACE
    assert _route(lib, handle, ws=12 * BUF + 64) == WORKSPACE
    assert _route(lib, handle, nbytes=100) == WORKSPACE
    # what is not wanted is not looked at
    assert _route(lib, handle, rows=None, order=None, live=None, losses=None, nbytes=100) == WORKSPACE
    for kw in (dict(chosen=None), dict(counts=None), dict(live=None), dict(dlogits=None), dict(ld=15), dict(ld=1 << 41),
               dict(balance=float("nan")), dict(z=float("inf"))):
        assert _route_grad(lib, handle, **kw) == INVALID
    for kw in (dict(chosen=2 * BUF + 1), dict(counts=4 * BUF + 2), dict(live=8 * BUF + 2), dict(dgates=9 * BUF + 2),
               dict(dlogits=10 * BUF + 2)):
        assert _route_grad(lib, handle, **kw) == UNALIGNED
    assert _route_grad(lib, handle, _router(tokens=0), chosen=None, counts=None, live=None, dlogits=None) == OK


def test_router_overlaps_refused(lib, handle):
    names = ("chosen", "gates", "counts", "offsets", "rows", "order", "live", "losses")
    for a in names:
        assert _route(lib, handle, **{a: BUF}) == OVERLAP                      # the logits
        assert _route(lib, handle, **{a: 12 * BUF}) == OVERLAP                 # the workspace
        for i, b in enumerate(names):
            if b != a:
                assert _route(lib, handle, **{a: (2 + i) * BUF}) == OVERLAP    # another output
    assert _route(lib, handle, ws=BUF) == OVERLAP
    for at in (BUF, BUF + 64, 2 * BUF, 4 * BUF, 8 * BUF, 9 * BUF):
        assert _route_grad(lib, handle, dlogits=at) == OVERLAP
    # behind the experts of a padded row nothing is shared, but there is no room for 16
    assert _route_grad(lib, handle, _router(ld=24), dlogits=BUF + 64, ld=24) == OVERLAP


def test_workspace_sizes_grow_with_the_sizes(lib, handle):
    def need(**over):
        sz = ctypes.c_size_t()
        assert lib.muon_router_workspace_size(handle, _router(**over), sz) == OK
        assert sz.value % 256 == 0
        return sz.value
    assert need(tokens=65) >= 2 * 16 * (1 + 4 + 4) + 16 * 8 + 2 * 12
    assert need(tokens=1 << 20) >= (1 << 14) * 16 * 9
    assert need(tokens=0) > 0


# ---- the binding -----------------------------------------------------------------------

def test_binding_refuses_tensors_on_the_host():
    h = ctypes.c_void_p()
    h.device = 0
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mu.muon_layernorm_forward(h, x, x)
    with pytest.raises(ValueError):
        mu.muon_rotary(h, x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        mu.muon_router_grad(h, x, x, x, x, x)


def test_binding_takes_a_handle_that_does_not_name_its_device():
    # as the step's calls do; the tensors are looked at all the same
    x = torch.zeros(4, 8)
    for call in (lambda h: mu.muon_layernorm_forward(h, x, x),
                 lambda h: mu.muon_rotary(h, x, x, torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.float64)),
                 lambda h: mu.muon_router_grad(h, x, x, x, x, x)):
        with pytest.raises(ValueError):
            call(ctypes.c_void_p())


def test_binding_describes_tensors():
    from muon_step_02_amd import _lib

    def heads(t):
        return _lib._heads(t, t.shape, "x")

    t = torch.zeros(6, 4, 10)
    d = heads(t[:, 1:3, 2:8])
    assert (d.token, d.head, d.heads, d.data) == (40, 10, 2, t.data_ptr() + 4 * 12)
    d = heads(t[:, 0])
    assert (d.token, d.head, d.heads) == (40, 10, 1)
    d = heads(t[:1])
    assert (d.token, d.head, d.heads) == (40, 10, 4)
    d = heads(t.transpose(0, 1))
    assert (d.token, d.head, d.heads) == (10, 40, 6)
    with pytest.raises(ValueError):
        heads(t.transpose(1, 2))
    with pytest.raises(ValueError):
        heads(t[0, 0])
    for bad in (t[:, 0, 0], torch.zeros(5), torch.zeros(6, dtype=torch.float64)):
        with pytest.raises(ValueError):
            _lib._vector(bad, 6, torch.float32, "w")
    with pytest.raises(ValueError):
        _lib._router(t[0].t(), 1, _lib._torch_parts()[3], False)


class _Recorder:
    """In the library's place: the descriptors that a binding hands it."""

    def __init__(self):
        self.x, self.y = [], []

    def muon_rotary(self, h, p, x, y, n, transpose, stream):
        def row(t):
            return t.data, t.token, t.head, t.heads
        self.x, self.y = [row(x[i]) for i in range(n)], [row(y[i]) for i in range(n)]
        return 0


@pytest.fixture
def recorder(monkeypatch):
    """What the bindings describe, without a device: tensors of the host count as the handle's."""
    from muon_step_02_amd import _lib
    stub = _Recorder()
    monkeypatch.setattr(_lib, "_torch", _lib._torch_parts()[:4] + (lambda device: 0,))
    monkeypatch.setattr(_lib, "_lib", stub)
    return stub


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("names", ["q", "qk", "kq", "qkq", "kqk", "qkqk", "kqqk", "qqk", "qkkq"])
def test_binding_describes_every_tensor_of_a_turn(recorder, names, tokens):
    # the same input may be listed again: it is only read
    h = ctypes.c_void_p()
    h.device = torch.zeros(0).get_device()
    given = {"q": torch.zeros(tokens, 16, 8), "k": torch.zeros(tokens, 2, 8)}
    xs = [given[n] for n in names]
    ys = [torch.zeros_like(t) for t in xs]
    mu.muon_rotary(h, xs, ys, torch.zeros(tokens, dtype=torch.int32), torch.zeros(4, dtype=torch.float64))
    for tensors, rows in ((xs, recorder.x), (ys, recorder.y)):
        assert rows == [(t.data_ptr(), t.shape[1] * 8, 8, t.shape[1]) for t in tensors]
