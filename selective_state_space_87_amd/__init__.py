"""MI355X-native selective state-space scan.

The compute path is the HIP library ``libssm_scan.so`` (C ABI, declared in
``include/ssm_scan.h``). The Python functions here only marshal torch device
tensors into that ABI; the library is loaded on first use and a missing or
unloadable library raises at once.
"""

from .binding import (  # noqa: F401
    ssm_abi_version,
    ssm_causal_conv1d_fwd,
    ssm_causal_conv1d_update,
    ssm_gated_delta_bwd,
    ssm_gated_delta_bwd_workspace_bytes,
    ssm_gated_delta_fwd,
    ssm_gated_delta_update,
    ssm_gated_delta_workspace_bytes,
    ssm_rms_norm_bwd,
    ssm_rms_norm_bwd_workspace_bytes,
    ssm_rms_norm_fwd,
    ssm_scan_bwd_workspace_bytes,
    ssm_scan_chunks,
    ssm_scan_workspace_bytes,
    ssm_selective_scan_bwd,
    ssm_selective_scan_fwd,
    ssm_selective_state_update,
    ssm_ssd_fwd,
    SSMError,
)
