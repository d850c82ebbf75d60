"""GB300-native (sm_103a) Mamba-2 SSD chunked scan: forward, backward,
decode step and the block's conv1d and grouped norm; the block's other
operators, the gated delta rule and the optimizer's step.

The computation lives in ``libssd_gb300.so`` (CUDA kernels behind the C ABI
of include/ssd_scan.h and the headers beside it); this package only marshals
torch tensors into it.
"""
from .scan import (abi_version, bwd_workspace_bytes, causal_conv1d,  # noqa: F401
                   group_rmsnorm_, host_workspace_bytes, scan_status, ssd_chunk_fused,
                   ssd_chunk_scan, ssd_chunk_state, ssd_decode_step, ssd_dt_cumsum,
                   ssd_scan, ssd_scan_bwd, ssd_scan_fwd, ssd_scan_fwd_host, ssd_state_passing,
                   workspace_bytes)
from .block import (add_rmsnorm, add_rmsnorm_bwd, add_rmsnorm_fwd,  # noqa: F401
                    block_abi_version, causal_conv1d_bwd, causal_conv1d_step, clip_grads,
                    gated_rmsnorm, gated_rmsnorm_bwd, gated_rmsnorm_fwd, grad_norm, linear,
                    linear_bwd, linear_fwd)
from .delta import (delta_abi_version, delta_decode_step, delta_scan,  # noqa: F401
                    delta_scan_bwd, delta_scan_fwd)
from .optim import adamw_moments, adamw_state, adamw_step, optim_abi_version  # noqa: F401
