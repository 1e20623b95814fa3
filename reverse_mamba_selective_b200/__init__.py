"""B200-native right-to-left selective-scan sidecar (R2LM) and partial-bidirectional scan.

The compute lives in libr2l.so (CUDA, sm_100a; C ABI in include/r2l.h) and, for the
linear-attention mixer, in libr2l_mixer.so (include/r2l_mixer.h).  This package only
builds them (``_build``) and marshals arguments to them (``r2l``, ``mixer``).
"""

from .mixer import (  # noqa: F401
    LinattnArgs, MixerError, QkNormRopeArgs, load_mixer, r2l_linattn, r2l_linattn_bwd, r2l_linattn_step,
    r2l_mixer_abi_version, r2l_mixer_device_status, r2l_qk_norm_rope, r2l_qk_norm_rope_bwd,
)
from .r2l import (  # noqa: F401
    R2L_BF16, R2L_ERR_CUDA, R2L_ERR_INVALID_ARG, R2L_ERR_TIMEOUT, R2L_ERR_UNSUPPORTED, R2L_F32, R2L_OK,
    R2LError, ScanArgs, SidecarWeights, bidir_scan, fwd_scan_from_state, load, make_scan_args, make_sidecar_weights,
    r2l_abi_version, r2l_decode_step, r2l_device_status, r2l_dt_proj, r2l_in_proj, r2l_residual_apply, r2l_scan_block,
    r2l_scan_block_bwd,
    r2l_sidecar_forward, r2l_wait_selftest, r2l_x_proj, r2l_x_proj_noalloc, sidecar_workspace_size, status_string,
)
