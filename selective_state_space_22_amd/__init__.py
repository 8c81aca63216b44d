"""MI355X (gfx950) selective scan (S6): HIP kernels behind a C ABI.

    from selective_state_space_22_amd import mamba_scan_fwd, mamba_scan_bwd, mamba_state_update

The functions are thin ctypes wrappers of libmamba_mi355x.so (see
include/mamba_mi355x.h, include/mamba_mi355x_lm.h for what a model of tokens
needs around the scan, and include/mamba_mi355x_layer.h for what a layer does); build the library with
``python -m selective_state_space_22_amd.build``.
"""
from .binding import (MAMBA_IO_BF16, MAMBA_IO_F32, MambaError, load_library, mamba_block_fwd,
                      mamba_get_option, mamba_set_option, mamba_stream_status,
                      mamba_block_fwd_workspace_size, mamba_scan_bwd,
                      mamba_scan_bwd_workspace_size, mamba_scan_fwd, mamba_scan_fwd_complex,
                      mamba_scan_fwd_complex_workspace_size, mamba_scan_fwd_noalloc, mamba_scan_fwd_workspace_size,
                      mamba_selection_fwd, mamba_selection_fwd_workspace_size, mamba_ssm_fwd,
                      mamba_ssm_fwd_workspace_size, mamba_state_update, mamba_state_update_complex, mamba_version,
                      status_string)
from .layer import (mamba_conv_bwd, mamba_conv_bwd_workspace_size, mamba_conv_fwd, mamba_conv_ssm_update,
                    mamba_conv_ssm_update_workspace_size, mamba_conv_update, mamba_draft_verify,
                    mamba_draft_verify_workspace_size, mamba_residual_norm_bwd,
                    mamba_residual_norm_bwd_workspace_size, mamba_residual_norm_fwd)
from .lm import (MAMBA_GATED_STATE_CHUNK, mamba_embed_bwd, mamba_embed_bwd_workspace_size, mamba_embed_fwd,
                 mamba_gated_scan_bwd, mamba_gated_scan_bwd_workspace_size, mamba_gated_scan_fwd,
                 mamba_gated_scan_fwd_workspace_size, mamba_gated_state_update, mamba_sample)

__all__ = ["mamba_block_fwd", "mamba_block_fwd_workspace_size", "mamba_scan_fwd", "mamba_scan_fwd_complex", "mamba_scan_fwd_complex_workspace_size", "mamba_scan_bwd",
           "mamba_state_update", "mamba_state_update_complex", "mamba_scan_fwd_workspace_size",
           "mamba_scan_bwd_workspace_size", "mamba_selection_fwd", "mamba_selection_fwd_workspace_size",
           "mamba_ssm_fwd", "mamba_ssm_fwd_workspace_size", "mamba_version", "status_string", "load_library", "MambaError",
           "MAMBA_IO_F32", "MAMBA_IO_BF16", "mamba_set_option", "mamba_get_option", "mamba_stream_status",
           "mamba_scan_fwd_noalloc", "MAMBA_GATED_STATE_CHUNK", "mamba_embed_bwd", "mamba_embed_bwd_workspace_size",
           "mamba_embed_fwd", "mamba_gated_scan_bwd", "mamba_gated_scan_bwd_workspace_size", "mamba_gated_scan_fwd",
           "mamba_gated_scan_fwd_workspace_size", "mamba_gated_state_update", "mamba_sample",
           "mamba_conv_bwd", "mamba_conv_bwd_workspace_size", "mamba_conv_fwd", "mamba_conv_ssm_update",
           "mamba_conv_ssm_update_workspace_size", "mamba_conv_update", "mamba_draft_verify",
           "mamba_draft_verify_workspace_size", "mamba_residual_norm_bwd", "mamba_residual_norm_bwd_workspace_size",
           "mamba_residual_norm_fwd"]
