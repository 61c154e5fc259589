"""GB300 (sm_103a) chunked gated-delta-rule forward with dynamic FP8 E4M3 state/W QDQ, linear
attention with a decay for each head, and the norms around both.

The computation lives in the CUDA library ``libgdnqat.so`` (C ABI: include/gdnqat.h);
this package is its ctypes binding plus the seeded synthetic-input generators.
"""
from .gdnqat import (  # noqa: F401
    EXPORTED,
    GDN_FLAG_KDA,
    GDN_FLAG_STATE_INT8,
    GDN_FLAG_STATE_QDQ,
    GDN_FLAG_W_QDQ,
    ChunkArgs,
    GdnError,
    chunk_bwd_workspace_bytes,
    chunk_workspace_bytes,
    fp8_tile_qdq,
    gdn_check_device_status,
    gdn_chunk_bwd,
    gdn_chunk_fwd,
    gdn_decode_step,
    gdn_prefill_decode_fwd,
    int8_block_qdq,
    kda_chunk_bwd,
    kda_chunk_fwd,
    kda_prefill_decode_fwd,
    lib_path,
    load,
    prefill_decode_workspace_bytes,
    status_string,
    workspace_bytes,
)
from .layer import (  # noqa: F401
    gated_norm_bwd,
    gated_norm_fwd,
    la_chunk_bwd,
    la_chunk_fwd,
    la_chunk_workspace_bytes,
    la_decode_step,
    residual_norm_bwd,
    residual_norm_fwd,
)
