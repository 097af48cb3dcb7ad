"""gated_delta_rule_loop_amd - the gated delta rule recurrence on MI355X (gfx950).

The computation lives in libgdr.so (hand-written HIP kernels behind the C ABI
of include/gdr.h).  This package is its thin binding: the functions below
marshal torch device tensors into the C ABI and nothing else.  Build the
library with `python -m gated_delta_rule_loop_amd.build`.
"""
from ._binding import (  # noqa: F401
    GdrError,
    gdr_block_norm,
    gdr_block_norm_bwd,
    gdr_block_norm_workspace,
    gdr_causal_conv1d,
    gdr_causal_conv1d_bwd,
    gdr_causal_conv1d_fold,
    gdr_causal_conv1d_workspace,
    gdr_check_indices,
    gdr_fused_recurrent_update,
    gdr_fwd_output_shape,
    gdr_last_error_message,
    gdr_linear_attention_bwd,
    gdr_linear_attention_fwd,
    gdr_linear_attention_step,
    gdr_linear_attention_workspace,
    gdr_recurrence_fwd,
    gdr_recurrence_verify_ring,
    gdr_set_debug_checks,
    gdr_ring_record_elements,
    gdr_selective_scan_bwd,
    gdr_selective_scan_fold,
    gdr_selective_scan_fwd,
    gdr_selective_scan_step,
    gdr_selective_scan_workspace,
    gdr_snapshot_rollback,
    gdr_state_fold,
    gdr_verify_drafts,
    gdr_verify_drafts_workspace,
    gdr_version,
    lib,
)
