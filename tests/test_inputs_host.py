"""Operators on the step's inputs (gradient norm and clip, expert products,
largest attention logits): what their entry points refuse, and the layout of
their structures.  No GPU: every refusal comes before a call touches a
device, so a zeroed block of memory stands in for the handle."""

import ctypes
import os
import subprocess

import pytest
import torch

import muon_step_02_amd as mu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, WORKSPACE, OVERLAP, UNALIGNED = 1, 3, 4, 6
BUF = 1 << 20  # an address for tensors that no call gets to read


@pytest.fixture(scope="module")
def lib():
    return mu.load()


@pytest.fixture(scope="module")
def handle():
    return ctypes.cast(ctypes.create_string_buffer(4096), ctypes.c_void_p)


def test_structures_match_the_header(tmp_path):
    structs = {"muon_grad": mu.MuonGrad, "muon_experts": mu.MuonExperts, "muon_qk": mu.MuonQk}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "muon.h"', "int main(void){"]
    for name, cls in structs.items():
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        lines += ['printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f)
                  for f, _ in cls._fields_]
    c, exe = tmp_path / "s.c", tmp_path / "s"
    c.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = {k: int(v) for k, v in (line.split() for line in out.splitlines())}
    for name, cls in structs.items():
        assert got[name] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got["%s.%s" % (name, f)] == getattr(cls, f).offset, (name, f)


# ---- gradient norm and clip ------------------------------------------------

def _grad(**over):
    d = dict(grad=BUF, out=BUF, rows=4, cols=8, ld_grad=8, ld_out=8, grad_dtype=0, out_dtype=0)
    d.update(over)
    return mu.MuonGrad(**d)


def _grad_call(lib, h, grads, clip=True, max_norm=1.0, norm=4 * BUF, scale=None, ws=8 * BUF,
               nbytes=1 << 20):
    arr = (mu.MuonGrad * max(len(grads), 1))(*grads)
    fn = lib.muon_grad_clip if clip else lib.muon_grad_norm
    return fn(h, arr, len(grads), max_norm, norm, scale, ws, nbytes, None)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("over", [dict(rows=-1), dict(cols=-1), dict(ld_grad=7), dict(grad_dtype=2),
                                  dict(grad=None), dict(rows=1 << 41), dict(cols=1 << 41),
                                  dict(rows=1 << 39, cols=1 << 39, ld_grad=1 << 39),
                                  dict(rows=1 << 20, ld_grad=1 << 39)])
def test_grad_sizes_refused(lib, handle, clip, over):
    assert _grad_call(lib, handle, [_grad(**over)], clip) == INVALID


@pytest.mark.parametrize("over", [dict(out=None), dict(out_dtype=5), dict(ld_out=7)])
def test_grad_outputs_refused(lib, handle, over):
    assert _grad_call(lib, handle, [_grad(**over)]) == INVALID


@pytest.mark.parametrize("clip", [False, True])
def test_grad_arguments_refused(lib, handle, clip):
    g = [_grad()]
    assert _grad_call(lib, handle, [], clip) == INVALID
    assert _grad_call(lib, None, g, clip) == INVALID
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert _grad_call(lib, handle, g, clip, max_norm=bad) == INVALID
    assert _grad_call(lib, handle, g, clip, ws=None) == WORKSPACE
    assert _grad_call(lib, handle, g, clip, ws=8 * BUF + 128) == WORKSPACE
    assert _grad_call(lib, handle, g, clip, nbytes=64) == WORKSPACE
    assert _grad_call(lib, handle, g, clip, norm=BUF + 2) == UNALIGNED
    assert _grad_call(lib, handle, [_grad(grad=BUF + 2, out=BUF + 2)], clip) == UNALIGNED
    if not clip:
        assert _grad_call(lib, handle, g, False, norm=None, scale=None) == INVALID


def test_clip_outputs_that_share_memory_are_refused(lib, handle):
    def both(a, b):
        return _grad_call(lib, handle, [a, b], nbytes=0)  # refused for its workspace, if at all

    far = _grad(grad=2 * BUF, out=2 * BUF)
    assert both(_grad(), far) == WORKSPACE
    assert both(_grad(), _grad()) == OVERLAP                              # one tensor twice
    assert both(_grad(), _grad(grad=2 * BUF, out=BUF + 64)) == OVERLAP    # into another's gradient
    assert both(_grad(out=3 * BUF), _grad(grad=2 * BUF, out=3 * BUF)) == OVERLAP
    assert both(_grad(out=3 * BUF), _grad(out=4 * BUF)) == WORKSPACE      # one gradient read twice
    # its own gradient, but not exactly in place
    assert both(_grad(out=BUF + 32), far) == OVERLAP
    assert both(_grad(grad_dtype=1), far) == OVERLAP
    assert both(_grad(ld_out=16), far) == OVERLAP
    # column blocks of one buffer interleave without sharing
    left, right = (_grad(grad=BUF + o, out=BUF + o, ld_grad=16, ld_out=16) for o in (0, 32))
    assert both(left, right) == WORKSPACE
    assert both(left, _grad(grad=BUF + 28, out=BUF + 28, ld_grad=16, ld_out=16)) == OVERLAP
    assert both(left, _grad(grad=BUF + 36, out=BUF + 36, ld_grad=16, ld_out=16)) == OVERLAP


def test_grad_workspace_size(lib, handle):
    for n in (1, 16, 17, 257, 5000):
        sz = ctypes.c_size_t()
        arr = (mu.MuonGrad * n)(*[_grad()] * n)
        assert lib.muon_grad_workspace_size(handle, arr, n, ctypes.byref(sz)) == 0
        assert sz.value % 256 == 0 and sz.value >= 8 * 2048
    assert lib.muon_grad_workspace_size(handle, arr, 0, ctypes.byref(sz)) == INVALID


def test_the_handles_device_has_to_be_the_tensors():
    from muon_step_02_amd import _lib
    h = ctypes.c_void_p()
    h.device = 0
    with pytest.raises(ValueError):
        _lib._stream_on(None, torch.device("cuda:1"), h)
    with pytest.raises(ValueError):
        _lib._same_device(torch.zeros(1), None)
    with pytest.raises(ValueError):
        _lib._same_device(None)


def test_scaled_steps_need_a_scale(lib, handle):
    mats, hp = (mu.MuonMatrix * 1)(), mu.muon_hparams(lr=1e-3)
    assert lib.muon_step_batched_scaled(handle, mats, 1, ctypes.byref(hp), None, BUF, 1 << 20, None) == INVALID
    assert lib.muon_step_batched_scaled(handle, mats, 1, ctypes.byref(hp), BUF + 1, BUF, 1 << 20, None) == UNALIGNED
    ts, ahp = (mu.AdamwTensor * 1)(), mu.adamw_hparams(1e-3, 1)
    assert lib.adamw_step_scaled(handle, ts, 1, ctypes.byref(ahp), None, None) == INVALID
    assert lib.adamw_step_scaled(handle, ts, 1, ctypes.byref(ahp), BUF + 2, None) == UNALIGNED
    m = mu.MuonMatrix(param=2 * BUF, grad=3 * BUF, momentum=4 * BUF, rows=64, cols=64, ld_param=64,
                      ld_grad=64, ld_mom=64)
    mats = (mu.MuonMatrix * 1)(m)
    assert lib.muon_step_batched_scaled(handle, mats, 1, ctypes.byref(hp), 8 * BUF + 4, 8 * BUF,
                                        1 << 30, None) == OVERLAP


def test_grad_descriptors():
    t = torch.zeros(6, 10)
    g = mu.muon_grad(t[:, 2:7])
    assert (g.rows, g.cols, g.ld_grad, g.grad, g.out) == (6, 5, 10, t.data_ptr() + 8, None)
    g = mu.muon_grad(t.view(3, 2, 10))
    assert (g.rows, g.cols, g.ld_grad) == (1, 60, 60)
    g = mu.muon_grad(torch.zeros(5, dtype=torch.bfloat16), torch.zeros(5))
    assert (g.rows, g.cols, g.grad_dtype, g.out_dtype) == (1, 5, 1, 0)
    g = mu.muon_grad(torch.zeros(()))
    assert (g.rows, g.cols) == (1, 1)
    g = mu.muon_grad(torch.zeros(0, 7))
    assert g.rows * g.cols == 0
    for bad in (t.t(), t[:, ::2], t[:1].expand(6, 10), t.view(3, 2, 10)[:, :, :4]):
        with pytest.raises(ValueError):
            mu.muon_grad(bad)
    with pytest.raises(ValueError):
        mu.muon_grad(t, torch.zeros(10, 6))
    with pytest.raises(TypeError):
        mu.muon_grad(t.half())


# ---- expert products ---------------------------------------------------------

def _experts(n=3, at=BUF, step=1 << 14, **over):
    ptrs = (ctypes.c_void_p * max(n, 1))(*[at + i * step for i in range(n)])
    d = dict(weights=ptrs, rows=16, cols=32, ld=32, experts=n, dtype=1)
    d.update(over)
    ex = mu.MuonExperts(**d)
    ex._keep = ptrs
    return ex


def _rows_call(lib, h, ex, name="muon_expert_forward", offsets=9 * BUF, x=4 * BUF, ld_x=32, y=6 * BUF,
               ld_y=32, tokens=10):
    return getattr(lib, name)(h, ctypes.byref(ex), offsets, x, ld_x, y, ld_y, tokens, None)


def _weight_call(lib, h, ex, offsets=9 * BUF, x=4 * BUF, ld_x=32, dy=6 * BUF, ld_dy=16, tokens=10,
                 dtype=1, accumulate=0):
    return lib.muon_expert_grad_weight(h, ctypes.byref(ex), offsets, x, ld_x, dy, ld_dy, tokens, dtype,
                                       accumulate, None)


@pytest.mark.parametrize("over", [dict(experts=0), dict(experts=1025), dict(rows=0), dict(cols=0),
                                  dict(ld=31), dict(dtype=2), dict(rows=(1 << 20) + 1),
                                  dict(weights=None)])
def test_experts_refused(lib, handle, over):
    ex = _experts(**over)
    for name in ("muon_expert_forward", "muon_expert_grad_input"):
        assert _rows_call(lib, handle, ex, name) == INVALID
    assert _weight_call(lib, handle, ex) == INVALID


def test_expert_pointers_refused(lib, handle):
    ex = _experts()
    ex.weights[1] = None
    assert _rows_call(lib, handle, ex) == INVALID and _weight_call(lib, handle, ex) == INVALID
    ex = _experts(at=BUF + 1)
    assert _rows_call(lib, handle, ex) == UNALIGNED and _weight_call(lib, handle, ex) == UNALIGNED


@pytest.mark.parametrize("over,status", [
    (dict(offsets=None), INVALID), (dict(offsets=9 * BUF + 2), UNALIGNED), (dict(x=None), INVALID),
    (dict(ld_x=15), INVALID), (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), INVALID),
    (dict(x=4 * BUF + 1), UNALIGNED)])
def test_expert_tokens_refused(lib, handle, over, status):
    ex = _experts()
    assert _rows_call(lib, handle, ex, **over) == status
    assert _weight_call(lib, handle, ex, **over) == status


def test_expert_outputs_refused(lib, handle):
    ex = _experts()
    assert _rows_call(lib, handle, ex, y=None) == INVALID
    assert _rows_call(lib, handle, ex, ld_y=15) == INVALID
    assert _rows_call(lib, handle, ex, "muon_expert_grad_input", ld_y=31) == INVALID
    assert _rows_call(lib, handle, ex, y=4 * BUF + 64) == OVERLAP      # onto x
    assert _rows_call(lib, handle, ex, y=BUF + 512) == OVERLAP         # onto a weight
    assert _rows_call(lib, handle, ex, y=9 * BUF - 64) == OVERLAP      # onto the offsets
    assert _rows_call(lib, None, ex) == INVALID
    assert _rows_call(lib, handle, ex, tokens=0, x=None, y=None) == 0  # nothing to do


def test_expert_weight_gradients_refused(lib, handle):
    assert _weight_call(lib, handle, _experts(step=0)) == OVERLAP      # one gradient for two experts
    assert _weight_call(lib, handle, _experts(step=64)) == OVERLAP
    assert _weight_call(lib, handle, _experts(), x=BUF + 512) == OVERLAP
    assert _weight_call(lib, handle, _experts(), dy=BUF + 512) == OVERLAP
    assert _weight_call(lib, handle, _experts(), accumulate=2) == INVALID
    assert _weight_call(lib, handle, _experts(), dtype=3) == INVALID
    assert _weight_call(lib, handle, _experts(), dtype=0) == INVALID   # fp32 tokens, bf16 gradients
    assert _weight_call(lib, handle, _experts(rows=1 << 20, cols=1 << 20, ld=1 << 20, n=1024),
                        ld_x=1 << 20, ld_dy=1 << 20) == INVALID        # more tiles than a launch holds


def test_expert_binding_refuses(monkeypatch):
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        mu.muon_experts([cpu])      # not on a GPU
    with pytest.raises(ValueError):
        mu.muon_experts([])


# ---- largest attention logits -------------------------------------------------

def _qk(**over):
    d = dict(q=BUF, k=2 * BUF, tokens_q=10, tokens_k=12, q_token=128, q_head=32, k_token=64, k_head=32,
             cu_q=3 * BUF, cu_k=3 * BUF + 64, sequences=2, heads_q=4, heads_k=2, head_dim=32, dtype=1,
             causal=1, scale=0.5)
    d.update(over)
    return mu.MuonQk(**d)


def _smax_call(lib, h, qk, q=4 * BUF, k=5 * BUF, accumulate=0, ws=6 * BUF, nbytes=1 << 20):
    return lib.muon_qk_smax(h, ctypes.byref(qk), q, k, accumulate, ws, nbytes, None)


@pytest.mark.parametrize("over", [
    dict(heads_q=0), dict(heads_k=0), dict(heads_q=3), dict(head_dim=0), dict(sequences=0),
    dict(dtype=2), dict(causal=2), dict(tokens_q=-1), dict(tokens_k=-1), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_token=-1),
    dict(k_head=-1), dict(q=None), dict(k=None), dict(cu_q=None), dict(cu_k=None)])
def test_smax_refused(lib, handle, over):
    assert _smax_call(lib, handle, _qk(**over)) == INVALID


def test_smax_arguments_refused(lib, handle):
    assert _smax_call(lib, None, _qk()) == INVALID
    assert _smax_call(lib, handle, _qk(), q=None, k=None) == INVALID
    assert _smax_call(lib, handle, _qk(), accumulate=2) == INVALID
    assert _smax_call(lib, handle, _qk(), ws=None) == WORKSPACE
    assert _smax_call(lib, handle, _qk(), ws=6 * BUF + 64) == WORKSPACE
    assert _smax_call(lib, handle, _qk(), nbytes=16) == WORKSPACE
    for over in (dict(q=BUF + 1), dict(k=BUF + 1), dict(cu_q=BUF + 2), dict(cu_k=BUF + 2)):
        assert _smax_call(lib, handle, _qk(**over)) == UNALIGNED
    assert _smax_call(lib, handle, _qk(), q=BUF + 2) == UNALIGNED


def test_smax_workspace_holds_every_partial(lib, handle):
    sz = ctypes.c_size_t()
    for tq, seqs, heads in ((1, 1, 1), (10, 2, 4), (5000, 33, 64), (0, 1, 2)):
        qk = _qk(tokens_q=tq, sequences=seqs, heads_q=heads, heads_k=1)
        assert lib.muon_qk_smax_workspace_size(handle, ctypes.byref(qk), ctypes.byref(sz)) == 0
        assert sz.value % 256 == 0 and sz.value >= 4 * heads * (tq // 256)


# ---- the binding without a GPU ------------------------------------------------

class _On:
    """Stands in for a tensor on a device that this machine need not have."""

    def __init__(self, device, *shape, dtype=torch.float32, stride=None):
        self._t = torch.zeros(shape, dtype=dtype)
        if stride is not None:
            self._t = torch.zeros(1024, dtype=dtype).as_strided(shape, stride)
        self.device = torch.device(device)

    def get_device(self):
        return -1 if self.device.index is None else self.device.index

    def __getattr__(self, name):
        return getattr(self._t, name)


class _NoCalls:
    """Stands in for the library: any entry point that is reached fails."""

    def __getattr__(self, name):
        def called(*args):
            raise AssertionError("%s was called" % name)
        return called


@pytest.fixture
def bound(monkeypatch):
    """A handle of device 0, with a library that nothing may call."""
    from muon_step_02_amd import _lib
    monkeypatch.setattr(_lib, "load", _NoCalls)
    h = ctypes.c_void_p(BUF)
    h.device = 0
    return h


@pytest.mark.parametrize("device", ["cpu", "cuda:1"])
@pytest.mark.parametrize("call", [mu.muon_grad_norm, mu.muon_grad_clip])
def test_gradients_of_another_device_are_refused(bound, call, device):
    ws, norm = _On("cuda:0", 64, dtype=torch.uint8), _On("cuda:0", 1)
    here, there = _On("cuda:0", 4, 8), _On(device, 4, 8)
    for plan in ([mu.muon_grad(there, there)], [mu.muon_grad(here, here), mu.muon_grad(there, there)]):
        with pytest.raises(ValueError):
            call(bound, plan, 1.0, ws, norm_out=norm, stream=0)
    with pytest.raises(AssertionError):  # the same call with every tensor in place gets through
        call(bound, [mu.muon_grad(here, here)], 1.0, ws, norm_out=norm, stream=0)


def test_an_output_on_another_device_than_its_gradient_is_refused():
    for device in ("cpu", "cuda:1"):
        with pytest.raises(ValueError):
            mu.muon_grad(_On("cuda:0", 8), _On(device, 8))


def test_gradient_descriptors_keep_their_tensors():
    import gc
    import weakref
    g, o = torch.zeros(4, 8), torch.zeros(4, 8)
    alive = [weakref.ref(t) for t in (g, o)]
    plan = [mu.muon_grad(g, o)]
    del g, o
    gc.collect()
    assert all(r() is not None for r in alive)
    del plan
    gc.collect()
    assert all(r() is None for r in alive)


def test_one_row_experts_with_a_column_stride_are_refused():
    """One row has no leading dimension, but its columns still have to follow
    each other."""
    apart = _On("cuda:0", 1, 8, stride=(16, 2))
    with pytest.raises(ValueError):
        mu.muon_experts([apart])
    with pytest.raises(ValueError):
        mu.muon_experts([_On("cuda:0", 1, 8), apart])
    ex = mu.muon_experts([_On("cuda:0", 1, 8), _On("cuda:0", 1, 8, stride=(16, 1))])
    assert (ex.rows, ex.cols, ex.ld) == (1, 8, 8)
    # a column of one value a row
    ex = mu.muon_experts([_On("cuda:0", 1, 1, stride=(1, 5))])
    assert (ex.rows, ex.cols, ex.ld) == (1, 1, 1)


def test_a_stream_of_another_device_is_refused(bound):
    class Stream:
        cuda_stream = 0

        def __init__(self, device):
            self.device = torch.device(device)

    ws, norm, g = _On("cuda:0", 64, dtype=torch.uint8), _On("cuda:0", 1), _On("cuda:0", 8)
    with pytest.raises(ValueError):
        mu.muon_grad_norm(bound, [mu.muon_grad(g)], 1.0, ws, norm_out=norm, stream=Stream("cuda:1"))
    with pytest.raises(AssertionError):  # gets through
        mu.muon_grad_norm(bound, [mu.muon_grad(g)], 1.0, ws, norm_out=norm, stream=Stream("cuda:0"))


# ---- ranges that a call writes ------------------------------------------------

@pytest.mark.parametrize("clip", [False, True])
def test_grad_scalars_that_share_memory_are_refused(lib, handle, clip):
    ws = 8 * BUF
    need = ctypes.c_size_t()
    g = _grad(out=2 * BUF)          # 128 bytes at BUF and at 2 BUF
    assert lib.muon_grad_workspace_size(handle, ctypes.byref(g), 1, ctypes.byref(need)) == 0

    def call(**kw):
        return _grad_call(lib, handle, [_grad(grad=3 * BUF, out=3 * BUF), g], clip, **kw)

    far = 6 * BUF
    for at in (ws, ws + 256, ws + need.value - 4, BUF, BUF + 64, BUF + 124):
        assert call(norm=at) == OVERLAP
        assert call(norm=far, scale=at) == OVERLAP
    assert call(norm=far, scale=far) == OVERLAP         # on each other
    if clip:
        for at in (2 * BUF, 2 * BUF + 124, 3 * BUF):
            assert call(norm=at) == OVERLAP
            assert call(norm=far, scale=at) == OVERLAP


@pytest.mark.parametrize("clip", [False, True])
def test_gradients_in_the_workspace_are_refused(lib, handle, clip):
    for at in (8 * BUF, 8 * BUF + 1024, 8 * BUF - 64):
        assert _grad_call(lib, handle, [_grad(out=3 * BUF), _grad(grad=at, out=2 * BUF)], clip, norm=6 * BUF) == OVERLAP
    if clip:
        assert _grad_call(lib, handle, [_grad(out=8 * BUF + 64)], norm=6 * BUF) == OVERLAP


@pytest.mark.parametrize("tokens_q,dtype", [(10, 1), (3000, 0)])
def test_smax_outputs_and_workspace_that_share_memory_are_refused(lib, handle, tokens_q, dtype):
    far = dict(q=40 * BUF, k=50 * BUF, ws=60 * BUF)
    qk = _qk(q=10 * BUF, k=20 * BUF, cu_q=30 * BUF, cu_k=30 * BUF + 64, tokens_q=tokens_q, dtype=dtype)
    last_q, last_k = 10 * BUF + ((tokens_q - 1) * 128 + 127) * (2, 4)[1 - dtype], 20 * BUF + (11 * 64 + 63) * (2, 4)[1 - dtype]
    need = ctypes.c_size_t()
    assert lib.muon_qk_smax_workspace_size(handle, ctypes.byref(qk), ctypes.byref(need)) == 0
    inputs = [10 * BUF, last_q // 4 * 4, 20 * BUF, last_k // 4 * 4, 30 * BUF, 30 * BUF + 8, 30 * BUF + 64, 30 * BUF + 72]
    for at in inputs + [60 * BUF, 60 * BUF + need.value - 4]:
        for name in ("q", "k"):
            assert _smax_call(lib, handle, qk, **{**far, name: at}) == OVERLAP, (name, at)
            assert _smax_call(lib, handle, qk, **{**far, "q": None, "k": None, name: at}) == OVERLAP
    assert _smax_call(lib, handle, qk, **{**far, "q": 50 * BUF + 4}) == OVERLAP     # on the other output
    for at in inputs:
        assert _smax_call(lib, handle, qk, **{**far, "ws": at // 256 * 256}) == OVERLAP, at


def test_smax_spans_that_no_memory_holds_are_refused(lib, handle):
    for over in (dict(q_token=1 << 40, tokens_q=1 << 30), dict(k_token=1 << 40, tokens_k=1 << 30),
                 dict(q_head=1 << 40, heads_q=65536)):
        sz = ctypes.c_size_t()
        assert _smax_call(lib, handle, _qk(**over), nbytes=1 << 40) == INVALID
        assert lib.muon_qk_smax_workspace_size(handle, ctypes.byref(_qk(**over)), ctypes.byref(sz)) == INVALID


def test_a_scale_in_what_a_step_writes_is_refused(lib, handle):
    """4 x 8 weights, their momentum and outputs; AdamW tensors of 32 values."""
    hp, ahp = mu.muon_hparams(lr=1e-3), mu.adamw_hparams(1e-3, 1)
    m = mu.MuonMatrix(param=2 * BUF, grad=3 * BUF, momentum=4 * BUF, update_out=5 * BUF, norm_out=6 * BUF,
                      rows=4, cols=8, ld_param=8, ld_grad=8, ld_mom=8)
    other = mu.MuonMatrix(param=12 * BUF, grad=13 * BUF, momentum=14 * BUF, rows=4, cols=8, ld_param=8,
                          ld_grad=8, ld_mom=8, param_dtype=1)
    for mats in ((m, other), (other, m)):
        arr = (mu.MuonMatrix * 2)(*mats)
        for at in (2 * BUF, 2 * BUF + 124, 4 * BUF, 4 * BUF + 60, 5 * BUF + 4, 6 * BUF, 12 * BUF + 60, 14 * BUF + 124):
            assert lib.muon_step_batched_scaled(handle, arr, 2, ctypes.byref(hp), at, 32 * BUF, 1 << 24,
                                                None) == OVERLAP, at
    t = mu.AdamwTensor(param=2 * BUF, grad=3 * BUF, exp_avg=4 * BUF, exp_avg_sq=5 * BUF, numel=32)
    bf = mu.AdamwTensor(param=12 * BUF, grad=13 * BUF, exp_avg=14 * BUF, exp_avg_sq=15 * BUF, numel=32, param_dtype=1)
    for ts in ((t, bf), (bf, t)):
        arr = (mu.AdamwTensor * 2)(*ts)
        for at in (2 * BUF, 2 * BUF + 124, 4 * BUF + 8, 5 * BUF + 64, 12 * BUF + 60, 14 * BUF, 15 * BUF + 124):
            assert lib.adamw_step_scaled(handle, arr, 2, ctypes.byref(ahp), at, None) == OVERLAP, at


def test_more_threads_than_a_launch_holds_are_refused(lib, handle):
    """A launch takes fewer than 2^32 threads: ragged tiles of many groups over
    very wide outputs pass that within the sizes each argument may have."""
    wide = 1 << 20
    for over, tokens in ((dict(cols=8, ld=8, dtype=1), 32768), (dict(cols=8, ld=9, dtype=1), 1 << 17),
                         (dict(cols=1, ld=1, dtype=0), 1024)):
        ex = _experts(n=1024, at=1 << 40, step=1 << 25, rows=wide, **over)
        assert _rows_call(lib, handle, ex, x=BUF, ld_x=8, offsets=8 * BUF, y=1 << 44, ld_y=wide, tokens=tokens) == INVALID
    qk = _qk(q=1 << 40, k=1 << 44, heads_q=128, q_token=128 * 32, tokens_q=1 << 20, tokens_k=1 << 20,
             sequences=1 << 20, cu_q=8 * BUF, cu_k=16 * BUF)
    sz = ctypes.c_size_t()
    assert lib.muon_qk_smax_workspace_size(handle, ctypes.byref(qk), ctypes.byref(sz)) == INVALID
    assert _smax_call(lib, handle, qk, q=32 * BUF, k=33 * BUF, ws=1 << 46, nbytes=1 << 40) == INVALID


# ---- workspaces -----------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 16, 17, 256, 257, 512, 513, 5000])
def test_grad_workspace_holds_a_sum_per_block(lib, handle, n):
    """2048 blocks in proportion to the chunks, and one more for every launch of
    256 tensors at most: a 64-bit sum each."""
    sz = ctypes.c_size_t()
    arr = (mu.MuonGrad * n)(*[_grad()] * n)
    assert lib.muon_grad_workspace_size(handle, arr, n, ctypes.byref(sz)) == 0
    assert sz.value >= 8 * (2048 + (n + 255) // 256)


@pytest.mark.parametrize("tq,seqs", [(1, 1), (63, 2), (64, 1), (65, 65), (5000, 33), (9000, 3), (40, 1000), (0, 5)])
@pytest.mark.parametrize("heads", [1, 12, 64])
@pytest.mark.parametrize("dtype,dim", [(1, 32), (1, 33), (0, 32)])
def test_smax_workspace_holds_a_maximum_per_tile(lib, handle, tq, seqs, heads, dtype, dim):
    """Every sequence may end in a ragged tile, of 64 queries in the kernel for
    any type and of 128 or 256 in the others; with alignment the kernel may
    change while the size does not."""
    sz = ctypes.c_size_t()
    qk = _qk(tokens_q=tq, sequences=seqs, heads_q=heads, heads_k=1, head_dim=dim, q_head=dim, k_head=dim,
             q_token=heads * dim, k_token=dim, dtype=dtype)
    assert lib.muon_qk_smax_workspace_size(handle, ctypes.byref(qk), ctypes.byref(sz)) == 0
    assert sz.value >= 4 * heads * (tq // 64 + min(seqs, tq))
