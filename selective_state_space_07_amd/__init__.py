"""MI355X (gfx950) selective-scan mixer core behind the C ABI of libmamba_scan.

`fwd` (full-sequence prefill, optionally over packed documents), `bwd` (the
prefill's gradients), `step` (one-token decode), `ssd_fwd` / `ssd_bwd` /
`ssd_step` (the Mamba-2 SSD scan) and `lin_attn_fwd` / `lin_attn_bwd` / `lin_attn_step` (linear
attention with a decay for each head) and `group_norm_fwd` / `group_norm_bwd`
(the gated group norm behind a scan), `conv_fwd` / `conv_bwd` / `conv_step` (the
short causal convolution in front of one), `add_rms_norm_fwd` /
`add_rms_norm_fp8` / `add_rms_norm_bwd` (the norm between two blocks, with the
residual's addition) take torch tensors on the GPU and call the library's HIP kernels; PyTorch only provides device
memory and the stream. The raw C entry points are re-exported under their C
names. There is no fallback: without the library or a gfx950 device every
call raises MambaScanError.
"""
from ._binding import (EXPORTS, MAMBA_BF16, MAMBA_F32, MambaScanError, library_path, load,
                       mamba_scan_abi_version, mamba_scan_bwd, mamba_scan_bwd_ckpt,
                       mamba_scan_bwd_ckpt_workspace_bytes, mamba_scan_bwd_workspace_bytes, mamba_scan_ckpt_bytes,
                       mamba_scan_fwd_ckpt,
                       mamba_scan_call_count, mamba_scan_fwd, mamba_scan_fwd_seq, mamba_scan_fwd_workspace_bytes,
                       mamba2_ssd_fwd, mamba2_ssd_fwd_seq, mamba2_ssd_bwd, mamba2_ssd_bwd_workspace_bytes, mamba2_ssd_fwd_workspace_bytes, mamba2_ssd_step, mamba_scan_last_error, mamba_scan_status_str,
                       mamba_scan_step, mamba_scan_testing_fwd, mamba_scan_testing_fwd_workspace_bytes,
                       mamba_scan_fwd_noalloc, NOALLOC_SCRATCH_BYTES, mamba_scan_fwd_xc,
                       mamba_scan_step_xc, mamba_scan_step_xc_dtproj, mamba_scan_fwd_xc_dtproj)
from .api import Params, bwd, ckpt_like, fwd, step, workspace_bytes
from .conv import conv_bwd, conv_fwd, conv_step, conv_workspace_bytes
from .gnorm import group_norm_bwd, group_norm_fwd, group_norm_workspace_bytes
from .linattn import lin_attn_bwd, lin_attn_fwd, lin_attn_step, lin_attn_workspace_bytes
from .rmsnorm import add_rms_norm_bwd, add_rms_norm_fp8, add_rms_norm_fwd, add_rms_norm_workspace_bytes
from .ssd import ssd_bwd, ssd_bwd_workspace_bytes, ssd_fwd, ssd_step, ssd_workspace_bytes

__all__ = ["fwd", "bwd", "step", "lin_attn_fwd", "lin_attn_bwd", "lin_attn_step", "lin_attn_workspace_bytes",
           "group_norm_fwd", "group_norm_bwd", "group_norm_workspace_bytes", "conv_fwd", "conv_bwd", "conv_step", "conv_workspace_bytes",
           "add_rms_norm_fwd", "add_rms_norm_fp8", "add_rms_norm_bwd", "add_rms_norm_workspace_bytes", "ckpt_like", "mamba_scan_bwd_ckpt", "mamba_scan_bwd_ckpt_workspace_bytes",
           "mamba_scan_ckpt_bytes", "mamba_scan_fwd_ckpt", "ssd_fwd", "ssd_bwd", "ssd_step", "ssd_workspace_bytes", "ssd_bwd_workspace_bytes", "mamba2_ssd_bwd", "mamba2_ssd_bwd_workspace_bytes", "Params", "workspace_bytes", "MambaScanError", "MAMBA_F32", "MAMBA_BF16", "EXPORTS",
           "load", "library_path", "mamba_scan_abi_version", "mamba_scan_bwd", "mamba_scan_bwd_workspace_bytes",
           "mamba_scan_call_count", "mamba_scan_fwd",
           "mamba_scan_fwd_seq", "mamba_scan_fwd_workspace_bytes", "mamba2_ssd_fwd", "mamba2_ssd_fwd_seq", "mamba2_ssd_fwd_workspace_bytes", "mamba2_ssd_step", "mamba_scan_last_error", "mamba_scan_status_str", "mamba_scan_step",
           "mamba_scan_testing_fwd", "mamba_scan_testing_fwd_workspace_bytes", "mamba_scan_fwd_noalloc",
           "NOALLOC_SCRATCH_BYTES", "mamba_scan_fwd_xc",
           "mamba_scan_step_xc", "mamba_scan_step_xc_dtproj", "mamba_scan_fwd_xc_dtproj"]
