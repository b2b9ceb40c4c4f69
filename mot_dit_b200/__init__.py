"""mot_dit_b200 -- B200 (sm_100a) MoT world-action-model forward behind a C ABI.

The package is a thin ctypes binding over ``libmotdit.so`` (built in-tree by
``mot_dit_b200.build``): every step of the forward runs in the library's CUDA
kernels; this module only marshals arguments (device pointers of torch
tensors, CUDA stream handles, host arrays).  Importing works without a GPU;
calling anything that needs the library raises if it is missing -- there is
no CPU fallback.
"""
from ._binding import (  # noqa: F401
    ACTS,
    BF16,
    CEWP,
    FP32,
    PROF_CLASSES,
    SEQUENTIAL,
    TRACE_KINDS,
    Wam,
    WamConfig,
    WamError,
    lib,
    library_path,
    op_attention,
    op_attention_noalloc,
    op_linear,
    op_linear_tiled,
    op_linear_act,
    op_linear_act_backward,
    op_linear_act_workspace,
    op_gated,
    op_gated_backward,
    op_gated_workspace,
    op_residual_norm,
    op_residual_norm_backward,
    op_residual_norm_workspace,
    ops_check_status,
    op_attention_joint,
    op_norm_mod,
    patchify,
    preset,
)
