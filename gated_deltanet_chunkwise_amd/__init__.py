"""MI355X (gfx950) Gated DeltaNet chunkwise forward and backward passes, and the layer
operators around them: short causal convolution, selective state space scan, linear
attention with a decay per head, the norms around a block and 8-bit activation checkpoints.

Thin Python binding of libgdn.so (C ABI in include/gdn.h).  It only marshals
arguments: every step of every pass runs in the library's HIP kernels.
PyTorch is used for device memory and streams.  Importing the package does not
load the library; the first call does, and raises if it was not built
(``python -m gated_deltanet_chunkwise_amd.build``).
"""
from ._binding import (  # noqa: F401
    BWD_NUM_STAGES,
    BWD_STAGES,
    GDN_BF16,
    GDN_F16,
    GDN_F32,
    GDN_SCRATCH_BYTES,
    GDN_SEG_AUTO,
    GdnBackward,
    GdnError,
    GdnForward,
    NUM_STAGES,
    Params,
    STAGES,
    STAGE_ALL,
    STAGE_BITS,
    WorkspaceLayout,
    bwd,
    check,
    decode,
    decode_launcher,
    fuses_output,
    fwd,
    fwd_noalloc,
    gated_delta_rule,
    kda_gate,
    kda_gate_launcher,
    lib_path,
    load_library,
    make_params,
    seg_chunks,
    status_string,
    workspace_layout,
    workspace_size,
)
from ._layers import (  # noqa: F401
    Packed8,
    causal_conv,
    conv_bwd,
    conv_decode,
    conv_decode_launcher,
    conv_fwd,
    pack8,
    scan_bwd,
    scan_decode,
    scan_decode_launcher,
    scan_fwd,
    selective_scan,
    unpack8,
)
from ._linattn import (  # noqa: F401
    linear_attention,
    linear_attn_bwd,
    linear_attn_decode,
    linear_attn_decode_launcher,
    linear_attn_fwd,
)
from ._norms import (  # noqa: F401
    gated_norm,
    gated_norm_bwd,
    gated_norm_fwd,
    residual_norm,
    residual_norm_bwd,
    residual_norm_fwd,
)

__all__ = [
    "gated_norm", "gated_norm_bwd", "gated_norm_fwd", "residual_norm", "residual_norm_bwd", "residual_norm_fwd",
    "linear_attention", "linear_attn_bwd", "linear_attn_decode", "linear_attn_decode_launcher", "linear_attn_fwd",
    "Packed8", "causal_conv", "conv_bwd", "conv_decode", "conv_decode_launcher", "conv_fwd", "pack8", "scan_bwd",
    "scan_decode", "scan_decode_launcher", "scan_fwd", "selective_scan", "unpack8",
    "BWD_NUM_STAGES", "BWD_STAGES", "GdnBackward", "bwd",
    "GDN_BF16", "GDN_F16", "GDN_F32", "GDN_SCRATCH_BYTES", "GDN_SEG_AUTO", "GdnError", "GdnForward", "NUM_STAGES", "Params", "STAGES", "STAGE_ALL", "STAGE_BITS", "WorkspaceLayout",
    "check", "decode", "decode_launcher", "fuses_output", "fwd", "fwd_noalloc", "gated_delta_rule", "kda_gate", "kda_gate_launcher", "lib_path", "load_library", "make_params", "seg_chunks", "status_string",
    "workspace_layout", "workspace_size",
]
