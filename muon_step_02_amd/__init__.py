"""MI355X (gfx950) Muon optimizer step: Python binding of libmuon.

The binding only marshals arguments: every step of the optimizer runs in the
HIP kernels of ``libmuon.so`` (built from ``csrc/`` by ``build.py``).  There
is no fallback: if the library is missing, :func:`load` raises.

Names follow the C ABI in ``include/muon.h``:

* :func:`muon_init` / :func:`muon_destroy`
* :func:`muon_workspace_size`
* :func:`muon_step_batched`
* :func:`adamw_step`
* :func:`muon_grad_norm`, :func:`muon_grad_clip` and the steps that take their
  scale, :func:`muon_step_batched_scaled`, :func:`adamw_step_scaled`
* :func:`muon_expert_forward`, :func:`muon_expert_grad_input`,
  :func:`muon_expert_grad_weight`
* :func:`muon_qk_smax`
* :func:`muon_layernorm_forward`, :func:`muon_layernorm_grad`
* :func:`muon_rotary`, :func:`muon_rotary_frequencies`
* :func:`muon_router_forward`, :func:`muon_router_grad`

plus helpers that build the C descriptors from PyTorch tensors
(:func:`muon_matrix`, :func:`muon_hparams`, :func:`adamw_tensor`,
:func:`adamw_hparams`, :func:`muon_grad`, :func:`muon_experts`).
"""

from ._lib import (  # noqa: F401
    LIB_PATH,
    MUON_BF16,
    MUON_F32,
    SCALE_MODES,
    MuonError,
    MuonExperts,
    MuonGrad,
    MuonHeads,
    MuonLayernorm,
    MuonPositions,
    MuonQk,
    MuonRotaryPlan,
    MuonRouter,
    MuonRouting,
    AdamwHparams,
    AdamwTensor,
    MuonHparams,
    MuonMatrix,
    adamw_hparams,
    adamw_step,
    adamw_step_clipped,
    adamw_step_clipped_noalloc,
    adamw_step_scaled,
    adamw_workspace_size,
    adamw_tensor,
    exported_symbols,
    load,
    muon_destroy,
    muon_expert_forward,
    muon_expert_grad_input,
    muon_expert_grad_weight,
    muon_experts,
    muon_grad,
    muon_grad_clip,
    muon_grad_norm,
    muon_grad_workspace_size,
    muon_hparams,
    muon_init,
    muon_layernorm_forward,
    muon_layernorm_grad,
    muon_layernorm_workspace_size,
    muon_matrix,
    muon_profile_collect,
    muon_profile_enable,
    PhaseTimes,
    PHASES,
    muon_qk_smax,
    muon_qk_smax_workspace_size,
    muon_rotary,
    muon_rotary_frequencies,
    muon_router_forward,
    muon_router_grad,
    muon_router_workspace_size,
    muon_step_batched,
    muon_step_batched_scaled,
    muon_test_gram_bf16,
    muon_test_poly_bf16,
    muon_test_update_bf16,
    muon_test_split_matrices,
    muon_workspace_size,
)
from .route import route_parameters  # noqa: F401
