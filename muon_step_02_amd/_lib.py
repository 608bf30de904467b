"""ctypes binding of libmuon.so: structures mirror include/muon.h exactly."""

import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmuon.so")

MUON_F32 = 0
MUON_BF16 = 1
SCALE_MODES = {"moonlight": 0, "jordan": 1, "bernstein": 2, "none": 3}

STATUS = {
    0: "MUON_OK",
    1: "MUON_ERR_INVALID_ARG",
    2: "MUON_ERR_UNSUPPORTED_DEVICE",
    3: "MUON_ERR_WORKSPACE",
    4: "MUON_ERR_OVERLAP",
    5: "MUON_ERR_HIP",
    6: "MUON_ERR_UNALIGNED",
    7: "MUON_ERR_SCRATCH",
}

# every entry point include/muon.h declares
SYMBOLS = (
    "muon_init",
    "muon_destroy",
    "muon_workspace_size",
    "muon_step_batched",
    "adamw_step",
    "muon_status_str",
    "muon_test_gram_bf16",
    "muon_test_poly_bf16",
    "muon_test_update_bf16",
    "muon_profile_enable",
    "muon_profile_collect",
    "adamw_workspace_size",
    "adamw_step_clipped",
    "muon_test_split_matrices",
    "adamw_step_clipped_noalloc",
    "muon_step_batched_scaled",
    "adamw_step_scaled",
    "muon_grad_workspace_size",
    "muon_grad_norm",
    "muon_grad_clip",
    "muon_expert_forward",
    "muon_expert_grad_input",
    "muon_expert_grad_weight",
    "muon_qk_smax_workspace_size",
    "muon_qk_smax",
)

NUM_PHASES = 7
PHASES = ("momentum", "norm", "gram", "poly", "update", "apply", "adamw")


class MuonError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s: %s" % (what, STATUS.get(status, "status %d" % status)))


class MuonMatrix(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("momentum", ctypes.c_void_p),
        ("update_out", ctypes.c_void_p),
        ("norm_out", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld_param", ctypes.c_int64),
        ("ld_grad", ctypes.c_int64),
        ("ld_mom", ctypes.c_int64),
        ("param_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
        ("qk_smax", ctypes.c_void_p),
        ("qk_block_rows", ctypes.c_int64),
    ]


class MuonHparams(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("momentum", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("extra_scale", ctypes.c_float),
        ("nesterov", ctypes.c_int32),
        ("ns_steps", ctypes.c_int32),
        ("ns_dtype", ctypes.c_int32),
        ("scale_mode", ctypes.c_int32),
        ("coeffs", ctypes.POINTER(ctypes.c_float)),
        ("qk_tau", ctypes.c_float),
    ]


class AdamwTensor(ctypes.Structure):
    _fields_ = [
        ("param", ctypes.c_void_p),
        ("grad", ctypes.c_void_p),
        ("exp_avg", ctypes.c_void_p),
        ("exp_avg_sq", ctypes.c_void_p),
        ("numel", ctypes.c_int64),
        ("param_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
    ]


class PhaseTimes(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_float * 7), ("launches", ctypes.c_int32 * 7)]


class AdamwHparams(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("step", ctypes.c_int64),
    ]


class MuonGrad(ctypes.Structure):
    _fields_ = [
        ("grad", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld_grad", ctypes.c_int64),
        ("ld_out", ctypes.c_int64),
        ("grad_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
    ]
    _index = None  # device of the tensors it was made of (muon_grad; -1: no GPU)


class MuonExperts(ctypes.Structure):
    _fields_ = [
        ("weights", ctypes.POINTER(ctypes.c_void_p)),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("experts", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class MuonQk(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("tokens_q", ctypes.c_int64),
        ("tokens_k", ctypes.c_int64),
        ("q_token", ctypes.c_int64),
        ("q_head", ctypes.c_int64),
        ("k_token", ctypes.c_int64),
        ("k_head", ctypes.c_int64),
        ("cu_q", ctypes.c_void_p),
        ("cu_k", ctypes.c_void_p),
        ("sequences", ctypes.c_int32),
        ("heads_q", ctypes.c_int32),
        ("heads_k", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


_lib = None


def load():
    """Load libmuon.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libmuon.so not built: run `python -m muon_step_02_amd.build` "
                           "(expected at %s)" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.muon_init.argtypes = [i32, ctypes.POINTER(vp)]
    lib.muon_destroy.argtypes = [vp]
    lib.muon_workspace_size.argtypes = [vp, ctypes.POINTER(MuonMatrix), i32,
                                        ctypes.POINTER(MuonHparams), ctypes.POINTER(ctypes.c_size_t)]
    lib.muon_step_batched.argtypes = [vp, ctypes.POINTER(MuonMatrix), i32,
                                      ctypes.POINTER(MuonHparams), vp, ctypes.c_size_t, vp]
    lib.adamw_step.argtypes = [vp, ctypes.POINTER(AdamwTensor), i32, ctypes.POINTER(AdamwHparams), vp]
    lib.muon_status_str.argtypes = [i32]
    lib.muon_status_str.restype = ctypes.c_char_p
    lib.muon_test_gram_bf16.argtypes = [vp, vp, vp, i64, i64, i64, i64, f32, vp]
    lib.muon_test_poly_bf16.argtypes = [vp, vp, vp, i64, i64, f32, f32, f32, vp]
    lib.muon_test_update_bf16.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, f32, vp]
    lib.adamw_workspace_size.argtypes = [vp, ctypes.POINTER(AdamwTensor), i32,
                                         ctypes.POINTER(ctypes.c_size_t)]
    lib.adamw_step_clipped.argtypes = [vp, ctypes.POINTER(AdamwTensor), i32,
                                       ctypes.POINTER(AdamwHparams), f32, vp, vp, ctypes.c_size_t, vp]
    lib.muon_test_split_matrices.argtypes = [vp, ctypes.POINTER(MuonMatrix), i32,
                                             ctypes.POINTER(MuonHparams),
                                             ctypes.POINTER(ctypes.c_int32), i32,
                                             ctypes.POINTER(ctypes.c_int)]
    lib.adamw_step_clipped_noalloc.argtypes = [vp, ctypes.POINTER(AdamwTensor), i32,
                                               ctypes.POINTER(AdamwHparams), f32, vp, vp]
    sz = ctypes.c_size_t
    lib.muon_step_batched_scaled.argtypes = [vp, ctypes.POINTER(MuonMatrix), i32,
                                             ctypes.POINTER(MuonHparams), vp, vp, sz, vp]
    lib.adamw_step_scaled.argtypes = [vp, ctypes.POINTER(AdamwTensor), i32,
                                      ctypes.POINTER(AdamwHparams), vp, vp]
    lib.muon_grad_workspace_size.argtypes = [vp, ctypes.POINTER(MuonGrad), i32, ctypes.POINTER(sz)]
    for name in ("muon_grad_norm", "muon_grad_clip"):
        getattr(lib, name).argtypes = [vp, ctypes.POINTER(MuonGrad), i32, f32, vp, vp, vp, sz, vp]
    for name in ("muon_expert_forward", "muon_expert_grad_input"):
        getattr(lib, name).argtypes = [vp, ctypes.POINTER(MuonExperts), vp, vp, i64, vp, i64, i64, vp]
    lib.muon_expert_grad_weight.argtypes = [vp, ctypes.POINTER(MuonExperts), vp, vp, i64, vp, i64,
                                            i64, ctypes.c_int32, i32, vp]
    lib.muon_qk_smax_workspace_size.argtypes = [vp, ctypes.POINTER(MuonQk), ctypes.POINTER(sz)]
    lib.muon_qk_smax.argtypes = [vp, ctypes.POINTER(MuonQk), vp, vp, i32, vp, sz, vp]
    lib.muon_profile_enable.argtypes = [vp, i32]
    lib.muon_profile_collect.argtypes = [vp, ctypes.POINTER(PhaseTimes)]
    for name in ("muon_init", "muon_destroy", "muon_workspace_size", "muon_step_batched",
                 "adamw_step", "muon_test_gram_bf16", "muon_test_poly_bf16",
                 "muon_test_update_bf16", "muon_profile_enable", "muon_profile_collect",
                 "adamw_workspace_size", "adamw_step_clipped", "muon_test_split_matrices",
                 "adamw_step_clipped_noalloc", "muon_step_batched_scaled", "adamw_step_scaled",
                 "muon_grad_workspace_size", "muon_grad_norm", "muon_grad_clip",
                 "muon_expert_forward", "muon_expert_grad_input", "muon_expert_grad_weight",
                 "muon_qk_smax_workspace_size", "muon_qk_smax"):
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def exported_symbols():
    """Names of SYMBOLS that the loaded library actually exports."""
    lib = load()
    out = []
    for s in SYMBOLS:
        try:
            getattr(lib, s)
            out.append(s)
        except AttributeError:
            pass
    return out


def _check(status, what):
    if status != 0:
        raise MuonError(status, what)


def _stream_ptr(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(stream)


def _dt(t):
    import torch
    if t.dtype == torch.float32:
        return MUON_F32
    if t.dtype == torch.bfloat16:
        return MUON_BF16
    raise TypeError("only float32 and bfloat16 tensors are supported, got %s" % t.dtype)


def _ld(t):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2D row-major tensor (stride(1) == 1)")
    return t.stride(0)


def muon_matrix(param, grad, momentum, update_out=None, norm_out=None, qk_smax=None,
                qk_block_rows=0):
    """Descriptor of one Muon matrix from 2D tensors (row blocks are fine).
    ``qk_smax``: optional float32 device tensor of per-head max logits for
    QK-Clip, one per ``qk_block_rows`` rows."""
    import torch
    if momentum.dtype != torch.float32:
        raise TypeError("momentum must be float32")
    if grad.shape != param.shape or momentum.shape != param.shape:
        raise ValueError("param, grad and momentum shapes differ")
    rows, cols = param.shape
    if update_out is not None:
        if update_out.dtype != torch.float32 or not update_out.is_contiguous() or \
                tuple(update_out.shape) != (rows, cols):
            raise ValueError("update_out must be a contiguous float32 (rows, cols) tensor")
    if norm_out is not None and norm_out.dtype != torch.float32:
        raise ValueError("norm_out must be float32")
    if qk_smax is not None:
        if qk_smax.dtype != torch.float32 or not qk_smax.is_contiguous():
            raise ValueError("qk_smax must be a contiguous float32 tensor")
        if qk_block_rows < 1 or qk_smax.numel() * qk_block_rows < rows:
            raise ValueError("qk_smax needs one value per qk_block_rows rows")
    return MuonMatrix(
        param=param.data_ptr(), grad=grad.data_ptr(), momentum=momentum.data_ptr(),
        update_out=update_out.data_ptr() if update_out is not None else None,
        norm_out=norm_out.data_ptr() if norm_out is not None else None,
        rows=rows, cols=cols, ld_param=_ld(param), ld_grad=_ld(grad), ld_mom=_ld(momentum),
        param_dtype=_dt(param), grad_dtype=_dt(grad),
        qk_smax=qk_smax.data_ptr() if qk_smax is not None else None,
        qk_block_rows=qk_block_rows if qk_smax is not None else 0)


def muon_hparams(lr, momentum=0.95, weight_decay=0.1, eps=1e-7, extra_scale=1.0, nesterov=True,
                 ns_steps=5, ns_dtype="bf16", scale_mode="moonlight", coeffs=None, qk_tau=100.0):
    """Hyperparameters; ``coeffs`` is None or a flat list of 3*ns_steps floats."""
    hp = MuonHparams(lr=lr, momentum=momentum, weight_decay=weight_decay, eps=eps,
                     extra_scale=extra_scale, nesterov=1 if nesterov else 0, ns_steps=ns_steps,
                     ns_dtype=MUON_BF16 if ns_dtype == "bf16" else MUON_F32,
                     scale_mode=SCALE_MODES[scale_mode], qk_tau=qk_tau)
    if coeffs is not None:
        arr = (ctypes.c_float * len(coeffs))(*[float(c) for c in coeffs])
        hp._coeff_keepalive = arr
        hp.coeffs = ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
    return hp


def adamw_tensor(param, grad, exp_avg, exp_avg_sq):
    import torch
    for t in (param, grad, exp_avg, exp_avg_sq):
        if not t.is_contiguous():
            raise ValueError("AdamW tensors must be contiguous")
    if exp_avg.dtype != torch.float32 or exp_avg_sq.dtype != torch.float32:
        raise TypeError("AdamW state must be float32")
    n = param.numel()
    if grad.numel() != n or exp_avg.numel() != n or exp_avg_sq.numel() != n:
        raise ValueError("AdamW tensor sizes differ")
    return AdamwTensor(param=param.data_ptr(), grad=grad.data_ptr(), exp_avg=exp_avg.data_ptr(),
                       exp_avg_sq=exp_avg_sq.data_ptr(), numel=n, param_dtype=_dt(param),
                       grad_dtype=_dt(grad))


def adamw_hparams(lr, step, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1):
    return AdamwHparams(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
                        step=step)


def muon_init(device=0):
    lib = load()
    h = ctypes.c_void_p()
    _check(lib.muon_init(int(device), ctypes.byref(h)), "muon_init")
    h.device = int(device)
    return h


def muon_destroy(h):
    _check(load().muon_destroy(h), "muon_destroy")


def _array(mats):
    arr = (MuonMatrix * len(mats))(*mats)
    return arr


def muon_workspace_size(h, mats, hp):
    sz = ctypes.c_size_t()
    arr = _array(mats)
    _check(load().muon_workspace_size(h, arr, len(mats), ctypes.byref(hp), ctypes.byref(sz)),
           "muon_workspace_size")
    return sz.value


def muon_step_batched(h, mats, hp, workspace, stream=None):
    """``workspace``: a uint8 CUDA tensor of at least muon_workspace_size bytes."""
    arr = _array(mats)
    _check(load().muon_step_batched(h, arr, len(mats), ctypes.byref(hp),
                                    ctypes.c_void_p(workspace.data_ptr()),
                                    workspace.numel() * workspace.element_size(),
                                    _stream_ptr(stream)),
           "muon_step_batched")


def adamw_step(h, tensors, hp, stream=None):
    arr = (AdamwTensor * len(tensors))(*tensors)
    _check(load().adamw_step(h, arr, len(tensors), ctypes.byref(hp), _stream_ptr(stream)),
           "adamw_step")


def adamw_workspace_size(h, tensors):
    arr = (AdamwTensor * len(tensors))(*tensors)
    sz = ctypes.c_size_t()
    _check(load().adamw_workspace_size(h, arr, len(tensors), ctypes.byref(sz)), "adamw_workspace_size")
    return sz.value


def adamw_step_clipped(h, tensors, hp, max_norm, workspace, norm_out=None, stream=None):
    """AdamW with the gradients clipped together to global norm ``max_norm``.
    ``workspace``: uint8 CUDA tensor of at least adamw_workspace_size bytes;
    ``norm_out``: optional float32 CUDA tensor receiving the norm."""
    arr = (AdamwTensor * len(tensors))(*tensors)
    _check(load().adamw_step_clipped(h, arr, len(tensors), ctypes.byref(hp), float(max_norm),
                                     ctypes.c_void_p(norm_out.data_ptr() if norm_out is not None else 0),
                                     ctypes.c_void_p(workspace.data_ptr()),
                                     workspace.numel() * workspace.element_size(),
                                     _stream_ptr(stream)),
           "adamw_step_clipped")


def adamw_step_clipped_noalloc(h, tensors, hp, max_norm, norm_out=None, stream=None):
    """adamw_step_clipped without a workspace: the library's fixed per-device
    scratch holds the partial sums (at most 2^18 chunks of 4096 elements)."""
    arr = (AdamwTensor * len(tensors))(*tensors)
    _check(load().adamw_step_clipped_noalloc(
        h, arr, len(tensors), ctypes.byref(hp), float(max_norm),
        ctypes.c_void_p(norm_out.data_ptr() if norm_out is not None else 0), _stream_ptr(stream)),
        "adamw_step_clipped_noalloc")


def _same_device(*tensors):
    """The one CUDA device of the tensors (None among them: not given)."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("expected tensors on one device, got %s and %s" % (dev, t.device))
    if dev is None or dev.type != "cuda":
        raise ValueError("expected tensors on a CUDA device, got %s" % dev)
    return dev


def _stream_on(stream, device, h):
    """`stream`, or the current stream of the tensors' device, which has to be
    the handle's."""
    if device.index != getattr(h, "device", device.index):
        raise ValueError("the tensors are on %s, the handle is bound to device %d" % (device, h.device))
    if stream is None:
        import torch
        return torch.cuda.current_stream(device.index).cuda_stream
    if getattr(stream, "device", device) != device:
        raise ValueError("the tensors are on %s, the stream on %s" % (device, stream.device))
    return _stream_ptr(stream)


def _scalar(t, what):
    if t is None:
        return None
    import torch
    if t.dtype != torch.float32 or t.numel() != 1:
        raise ValueError("%s must be one float32" % what)
    return t.data_ptr()


def _nbytes(workspace):
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.nbytes


def _int32(t, what):
    import torch
    if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous 1D int32 tensor" % what)
    return t.data_ptr()


def muon_step_batched_scaled(h, mats, hp, grad_scale, workspace, stream=None):
    """:func:`muon_step_batched` with every gradient multiplied by the one-element
    float32 CUDA tensor ``grad_scale`` (:func:`muon_grad_norm`'s ``scale_out``)."""
    arr = _array(mats)
    dev = _same_device(grad_scale, workspace)
    _check(load().muon_step_batched_scaled(h, arr, len(mats), ctypes.byref(hp),
                                           _scalar(grad_scale, "grad_scale"), workspace.data_ptr(),
                                           _nbytes(workspace), _stream_on(stream, dev, h)),
           "muon_step_batched_scaled")


def adamw_step_scaled(h, tensors, hp, grad_scale, stream=None):
    """:func:`adamw_step` with every gradient multiplied by ``grad_scale``."""
    arr = (AdamwTensor * len(tensors))(*tensors)
    dev = _same_device(grad_scale)
    _check(load().adamw_step_scaled(h, arr, len(tensors), ctypes.byref(hp),
                                    _scalar(grad_scale, "grad_scale"), _stream_on(stream, dev, h)),
           "adamw_step_scaled")


def _rows_of(t):
    """(rows, cols, leading dimension) of a vector, of a matrix with unit
    column stride, or of a contiguous tensor of any shape."""
    if t.dim() == 2 and t.numel() and (t.stride(1) == 1 or t.shape[1] == 1) and \
            (t.stride(0) >= t.shape[1] or t.shape[0] == 1):
        return t.shape[0], t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor, or a 2D one with stride(1) == 1")
    return 1, t.numel(), t.numel()


def muon_grad(grad, out=None):
    """Descriptor of one gradient for :func:`muon_grad_norm` and, with ``out``
    (the gradient itself clips in place), :func:`muon_grad_clip`.  It keeps both
    tensors alive."""
    if out is not None and out.device != grad.device:
        raise ValueError("the gradient is on %s, its output on %s" % (grad.device, out.device))
    rows, cols, ld = _rows_of(grad)
    g = MuonGrad(grad=grad.data_ptr(), rows=rows, cols=cols, ld_grad=ld, grad_dtype=_dt(grad))
    if out is not None:
        if out.shape != grad.shape:
            raise ValueError("grad and out shapes differ")
        orows, ocols, old = _rows_of(out)
        if (orows, ocols) != (rows, cols):
            # one of the two is seen as one row: both are then
            if not (grad.is_contiguous() and out.is_contiguous()):
                raise ValueError("grad and out layouts differ")
            g.rows, g.cols, g.ld_grad, old = 1, grad.numel(), grad.numel(), grad.numel()
        g.out, g.ld_out, g.out_dtype = out.data_ptr(), old, _dt(out)
    g._index = grad.get_device()
    g._keepalive = (grad, out)
    return g


def muon_grad_workspace_size(h, grads):
    arr = (MuonGrad * len(grads))(*grads)
    sz = ctypes.c_size_t()
    _check(load().muon_grad_workspace_size(h, arr, len(grads), ctypes.byref(sz)),
           "muon_grad_workspace_size")
    return sz.value


def _grad_call(name, h, grads, max_norm, workspace, norm_out, scale_out, stream):
    dev = _same_device(workspace, norm_out, scale_out)
    arr = grads
    if not isinstance(grads, ctypes.Array):  # (whose structures have lost their tensors)
        here = dev.index
        for g in grads:
            if g._index != here and g._index is not None:
                raise ValueError("a gradient is on %s, the workspace on %s" % (g._keepalive[0].device, dev))
        arr = (MuonGrad * len(grads))(*grads)
    _check(getattr(load(), name)(h, arr, len(arr), float(max_norm), _scalar(norm_out, "norm_out"),
                                 _scalar(scale_out, "scale_out"), workspace.data_ptr(),
                                 _nbytes(workspace), _stream_on(stream, dev, h)), name)


def muon_grad_norm(h, grads, max_norm, workspace, norm_out=None, scale_out=None, stream=None):
    """Global norm of all ``grads`` (:func:`muon_grad` descriptors) and the clip
    scale for ``max_norm``, into one-element float32 CUDA tensors."""
    _grad_call("muon_grad_norm", h, grads, max_norm, workspace, norm_out, scale_out, stream)


def muon_grad_clip(h, grads, max_norm, workspace, norm_out=None, scale_out=None, stream=None):
    """:func:`muon_grad_norm`, then every descriptor's ``out`` = ``grad`` * scale."""
    _grad_call("muon_grad_clip", h, grads, max_norm, workspace, norm_out, scale_out, stream)


def muon_experts(weights):
    """Descriptor of a layer's expert matrices (or their gradients): equally
    shaped 2D tensors of one type and leading dimension."""
    if not weights:
        raise ValueError("no experts")
    w0 = weights[0]
    dev = _same_device(*weights)
    ld = _ld(w0) if w0.shape[0] > 1 else w0.shape[1]
    for w in weights:
        if w.shape != w0.shape or w.dtype != w0.dtype or (w.shape[0] > 1 and _ld(w) != ld):
            raise ValueError("the experts' shapes, types or leading dimensions differ")
        if w.shape[1] > 1 and w.stride(1) != 1:
            raise ValueError("expected 2D row-major tensors (stride(1) == 1)")
    ptrs = (ctypes.c_void_p * len(weights))(*[w.data_ptr() for w in weights])
    ex = MuonExperts(weights=ptrs, rows=w0.shape[0], cols=w0.shape[1], ld=ld, experts=len(weights),
                     dtype=_dt(w0))
    ex._keepalive = (ptrs, list(weights))
    ex._device = dev
    return ex


def _tokens(t, width, what):
    """Pointer and leading dimension of a token tensor of `width` columns."""
    if t.dim() != 2 or t.shape[1] != width or (width > 1 and t.stride(1) != 1):
        raise ValueError("%s must be 2D with %d columns and unit column stride" % (what, width))
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else width


def _offsets(ex, offsets, *tensors):
    if offsets.numel() != ex.experts + 1:
        raise ValueError("offsets must hold experts + 1 values")
    dev = _same_device(offsets, *tensors)
    if dev != ex._device:
        raise ValueError("the experts are on %s, the tokens on %s" % (ex._device, dev))
    return _int32(offsets, "offsets"), dev


def _expert_rows(name, h, ex, offsets, x, y, wx, wy, stream):
    po, dev = _offsets(ex, offsets, x, y)
    if _dt(x) != ex.dtype or _dt(y) != ex.dtype:
        raise TypeError("tokens and weights differ in type")
    if x.shape[0] != y.shape[0]:
        raise ValueError("the token tensors differ in rows")
    px, lx = _tokens(x, wx, "the input")
    py, ly = _tokens(y, wy, "the output")
    _check(getattr(load(), name)(h, ctypes.byref(ex), po, px, lx, py, ly, x.shape[0],
                                 _stream_on(stream, dev, h)), name)


def muon_expert_forward(h, ex, offsets, x, y, stream=None):
    """y[t] = W_e x[t] for the rows t of every group e: ``offsets`` (experts + 1
    int32, CUDA) bounds the groups; other rows of ``y`` stay as they are."""
    _expert_rows("muon_expert_forward", h, ex, offsets, x, y, ex.cols, ex.rows, stream)


def muon_expert_grad_input(h, ex, offsets, dy, dx, stream=None):
    """dx[t] = W_e^T dy[t], the input gradient of :func:`muon_expert_forward`."""
    _expert_rows("muon_expert_grad_input", h, ex, offsets, dy, dx, ex.rows, ex.cols, stream)


def muon_expert_grad_weight(h, grads, offsets, x, dy, accumulate=False, stream=None):
    """dW_e = sum of dy[t] x[t]^T over the rows of group e, or += with
    ``accumulate``; ``grads``: :func:`muon_experts` of the gradient tensors."""
    po, dev = _offsets(grads, offsets, x, dy)
    if _dt(x) != _dt(dy):
        raise TypeError("x and dy differ in type")
    if x.shape[0] != dy.shape[0]:
        raise ValueError("the token tensors differ in rows")
    px, lx = _tokens(x, grads.cols, "x")
    pd, ldd = _tokens(dy, grads.rows, "dy")
    _check(load().muon_expert_grad_weight(h, ctypes.byref(grads), po, px, lx, pd, ldd, x.shape[0],
                                          _dt(x), 1 if accumulate else 0, _stream_on(stream, dev, h)),
           "muon_expert_grad_weight")


def _qk(q, k, cu_q, cu_k, scale, causal):
    if q.dim() != 3 or k.dim() != 3 or q.shape[2] != k.shape[2]:
        raise ValueError("q and k must be (tokens, heads, head_dim) with equal head_dim")
    if q.shape[2] > 1 and (q.stride(2) != 1 or k.stride(2) != 1):
        raise ValueError("q and k need unit stride in their last dimension")
    if _dt(q) != _dt(k):
        raise TypeError("q and k differ in type")
    if cu_q is not None and cu_k is not None and cu_q.numel() != cu_k.numel():
        raise ValueError("cu_q and cu_k differ in length")
    if cu_q.numel() < 2:
        raise ValueError("cu_q must hold sequences + 1 values")
    return MuonQk(q=q.data_ptr(), k=k.data_ptr(), tokens_q=q.shape[0], tokens_k=k.shape[0],
                  q_token=q.stride(0), q_head=q.stride(1), k_token=k.stride(0), k_head=k.stride(1),
                  cu_q=_int32(cu_q, "cu_q"), cu_k=_int32(cu_k, "cu_k") if cu_k is not None else None,
                  sequences=cu_q.numel() - 1, heads_q=q.shape[1], heads_k=k.shape[1],
                  head_dim=q.shape[2], dtype=_dt(q), causal=1 if causal else 0,
                  scale=q.shape[2] ** -0.5 if scale is None else float(scale))


def muon_qk_smax_workspace_size(h, q, k, cu_q):
    """Workspace bytes of :func:`muon_qk_smax` for tensors of these shapes."""
    sz = ctypes.c_size_t()
    qk = _qk(q, k, cu_q, None, None, True)
    _check(load().muon_qk_smax_workspace_size(h, ctypes.byref(qk), ctypes.byref(sz)),
           "muon_qk_smax_workspace_size")
    return sz.value


def muon_qk_smax(h, q, k, cu_q, cu_k, smax_q, workspace, smax_k=None, scale=None, causal=True,
                 accumulate=False, stream=None):
    """Largest logit scale * <q_i, k_j> per head over packed sequences: ``q``
    (tokens, heads, head_dim), ``k`` (tokens, key heads, head_dim), ``cu_q`` and
    ``cu_k`` the sequences' bounds (int32, CUDA).  ``smax_q`` and ``smax_k``
    (float32, one value per head; either may be None) are what
    :func:`muon_matrix` takes as ``qk_smax`` for the query and the key
    projection.  ``scale`` defaults to head_dim ** -0.5."""
    import torch
    dev = _same_device(q, k, cu_q, cu_k, smax_q, smax_k, workspace)
    for t, n in ((smax_q, q.shape[1]), (smax_k, k.shape[1])):
        if t is not None and (t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous()):
            raise ValueError("smax outputs must be contiguous float32, one value per head")
    qk = _qk(q, k, cu_q, cu_k, scale, causal)
    _check(load().muon_qk_smax(h, ctypes.byref(qk), smax_q.data_ptr() if smax_q is not None else None,
                               smax_k.data_ptr() if smax_k is not None else None,
                               1 if accumulate else 0, workspace.data_ptr(), _nbytes(workspace),
                               _stream_on(stream, dev, h)), "muon_qk_smax")


def muon_test_gram_bf16(h, X, A, m, n, ldx, lda, s2=1.0, stream=None):
    _check(load().muon_test_gram_bf16(h, X.data_ptr(), A.data_ptr(), m, n, ldx, lda, s2,
                                      _stream_ptr(stream)), "muon_test_gram_bf16")


def muon_test_poly_bf16(h, A, B, m, lda, a, b, c, stream=None):
    """B = a I + b A + c A A (bf16, m x m, leading dimension lda)."""
    _check(load().muon_test_poly_bf16(h, A.data_ptr(), B.data_ptr(), m, lda, a, b, c,
                                      _stream_ptr(stream)), "muon_test_poly_bf16")


def muon_test_update_bf16(h, X, B, Xo, m, n, ldx, ldb, s=1.0, stream=None):
    """Xo = s B X (bf16; X, Xo m x n with leading dimension ldx, B m x m)."""
    _check(load().muon_test_update_bf16(h, X.data_ptr(), B.data_ptr(), Xo.data_ptr(), m, n, ldx,
                                        ldb, s, _stream_ptr(stream)), "muon_test_update_bf16")


def muon_test_split_matrices(h, mats, hp):
    """Indices of the matrices whose tiles sit where the grouped GEMM
    launches' per-XCD tile ranges start or end, or that hold quarter tiles."""
    arr = _array(mats)
    cnt = ctypes.c_int()
    _check(load().muon_test_split_matrices(h, arr, len(mats), ctypes.byref(hp), None, 0,
                                           ctypes.byref(cnt)), "muon_test_split_matrices")
    out = (ctypes.c_int32 * max(cnt.value, 1))()
    _check(load().muon_test_split_matrices(h, arr, len(mats), ctypes.byref(hp), out, cnt.value,
                                           ctypes.byref(cnt)), "muon_test_split_matrices")
    return list(out[:cnt.value])


def muon_profile_enable(h, enable=True):
    _check(load().muon_profile_enable(h, 1 if enable else 0), "muon_profile_enable")


def muon_profile_collect(h):
    """{phase: (total_ms, launches)} since the previous collect."""
    pt = PhaseTimes()
    _check(load().muon_profile_collect(h, ctypes.byref(pt)), "muon_profile_collect")
    return {PHASES[i]: (pt.ms[i], pt.launches[i]) for i in range(NUM_PHASES)}
