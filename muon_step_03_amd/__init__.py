"""Muon optimizer step (with the AdamW step of the hybrid optimizer and the
layer operators that make their gradients) for MI355X (gfx950): HIP kernels
behind a C ABI.

The HIP library (libmuon.so, built in-tree by ``muon_step_03_amd.build``) is
loaded on first use; without it every entry point raises.
"""
from .api import (  # noqa: F401
    AUX_BETAS, AUX_EPS, AUX_LR, AUX_WEIGHT_DECAY, AdamWStep, HybridMuonAdamW, MuonError,
    MuonStep, NS_COEFFICIENTS, adamw_step, adamw_step_grouped, adamw_tensor, muon_step,
    muon_step_batched, muon_step_grouped, muon_step_grouped_noalloc, pointer_table,
    stacked_chunks, stacked_group, chunk_size, table_group, workspace_bytes,
    workspace_bytes_grouped,
)
from .layer_ops import (  # noqa: F401
    ActCheckpoint, LayerNormOut, checkpoint_restore, checkpoint_save, layernorm_backward,
    layernorm_forward, layernorm_workspace_bytes, weight_grad, weight_grad_workspace_bytes,
)
from .layers import layer_norm, linear  # noqa: F401
