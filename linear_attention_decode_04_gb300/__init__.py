"""GB300-native fused KDA (Kimi Delta Attention) single-token decode step and
chunked varlen prefill, and the operators of a serving step around them
(block tables, q/k norm with rotation and 8-bit cache write, attention over
that cache, verification of drafted tokens; residual addition with norm and
8-bit output, matrix products with fused epilogues, log probabilities).

The compute lives in one hand-written CUDA library (``csrc/``) behind a C ABI
(``include/kda_decode.h``); ``kda_decode`` here only marshals torch tensors
into that call.  The library is loaded on first use; a missing library, or
one built for another ABI version, raises instead of falling back to anything
else (``build.build()`` recompiles any source newer than its object).
"""
from .binding import (  # noqa: F401
    KDA_EARLY_PREFETCH,
    KDA_FUSED_GATE,
    KDA_CONV_STATE_SD,
    KDA_OUT_NORM,
    KDA_UPDATE_CONV_STATE,
    KdaDecodeCall,
    MAX_TOKENS_PER_SEQ,
    KdaPrefillCall,
    KdaError,
    kda_chunk_metadata,
    kda_decode,
    kda_prefill,
    kda_status_string,
    library_path,
    load_library,
    longest_first_order,
)
from .step_ops import (  # noqa: F401
    KDA_ROPE_INTERLEAVED,
    KdaBlockTablesCall,
    KdaCacheAttentionCall,
    KdaQkRopeCall,
    KdaVerifyDraftCall,
    cache_attention_workspace,
    kda_block_tables,
    kda_cache_attention,
    kda_qk_rope,
    kda_verify_draft,
    rope_frequencies,
)
from .layer_ops import (  # noqa: F401
    KdaAddNormCall,
    KdaLinearCall,
    KdaLogprobsCall,
    kda_add_norm,
    kda_linear,
    kda_logprobs,
)
