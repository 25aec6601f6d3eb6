"""GB300-native KDA (Kimi Delta Attention) mixer step: decode, draft verify + commit, prefill.

The compute lives in libkda.so (hand-written sm_103a CUDA behind the C ABI in include/kda.h);
``verify_kda_decode_gb300.kda`` is its ctypes binding, ``verify_kda_decode_gb300.paged`` that of the
paged key-value cache and its attention, ``verify_kda_decode_gb300.rope`` that of the rotary positions.  Importing the package loads the library
(building it in-tree with nvcc first if it is missing) and fails if that is not possible.
"""
from .kda import (  # noqa: F401
    EXPORTS, KdaError, KdaLayer, KdaPool, kda_commit, kda_decode, kda_decode_resume, kda_get_error,
    kda_prefill, kda_prefill_varlen, kda_prefill_varlen_workspace_size,
    kda_prefill_noalloc, kda_prefill_noalloc_max_bytes, kda_prefill_workspace_size, kda_verify,
    kda_verify_resume,
    library, prepare_decode, prepare_verify, PreparedCall,
)
from .paged import (  # noqa: F401
    KdaKvCache, kda_attn_decode, kda_attn_prefill, kda_attn_workspace_size, kda_kv_append, kda_kv_compact,
    kda_kv_extend, kda_kv_fork, kda_kv_get_error, kda_kv_truncate, kda_kv_workspace_size,
)
from .rope import KdaRope, kda_kv_append_rope, kda_rope  # noqa: F401
