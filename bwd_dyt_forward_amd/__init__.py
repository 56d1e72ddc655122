"""Fused Dynamic Tanh (DyT) layer for AMD Instinct MI355X (gfx950).

y = gamma * tanh(alpha * x) + beta over an M x N row-major activation and its
backward (dx, dgamma, dbeta, dalpha), also with the residual add fused in
front (h = x + r, y = DyT(h)), computed by hand-written HIP kernels
behind a C ABI (``include/dyt.h``, library ``libdyt.so`` in this package).
The Python functions below carry the ABI's names and only marshal tensors.

Around it stand the operators a transformer block needs next to its
normalisation: layer norm (plain and residual) and attention with grouped key
heads, masks and a learned relative position bias, forward and backward
(``include/dyt_block.h``, library ``libdyt_block.so``); and what a decoder needs
around such blocks: root-mean-square norm (also with an 8-bit output),
embedding, log probabilities of tokens, AdamW (``include/dyt_lm.h``, library
``libdyt_lm.so``).
"""
from ._lib import (  # noqa: F401
    DYT_BF16,
    DYT_F16,
    DYT_F32,
    DYT_OK,
    LIB_FILE,
    DytError,
    dyt_abi_version,
    dyt_backward,
    dyt_backward_finish,
    dyt_backward_noalloc,
    dyt_backward_partials,
    dyt_backward_residual,
    dyt_backward_residual_partials,
    dyt_backward_workspace_size,
    dyt_forward,
    dyt_forward_residual,
    dyt_get_forward_plan,
    dyt_get_forward_residual_plan,
    dyt_get_plan,
    dyt_set_xcd_flip_override,
    dyt_status_string,
    dyt_xcd_hint,
    lib,
)

from .module import DyT, DyTFunction, DyTResidual, DyTResidualFunction, dyt, dyt_residual  # noqa: E402,F401

_BLOCK_ALL = [
    "BLOCK_LIB_FILE", "block_lib", "dyt_ln_forward", "dyt_ln_forward_residual", "dyt_ln_backward",
    "dyt_ln_backward_residual", "dyt_ln_backward_workspace_size", "dyt_attn_forward", "dyt_attn_backward",
    "dyt_attn_bucket_borders", "LayerNorm", "LayerNormFunction", "layer_norm", "LayerNormResidual",
    "LayerNormResidualFunction", "layer_norm_residual", "Attention", "AttentionFunction", "attention", "KVCache",
]

_LM_ALL = [
    "LM_LIB_FILE", "lm_lib", "DYT_LOGPROB_MAX_TOP", "DYT_ADAMW_BLOCK", "dyt_rms_forward", "dyt_rms_forward_residual",
    "dyt_rms_forward_q8", "dyt_rms_forward_residual_q8", "dyt_rms_backward", "dyt_rms_backward_residual",
    "dyt_rms_backward_workspace_size", "dyt_embed_forward", "dyt_embed_backward", "dyt_embed_backward_workspace_size",
    "dyt_logprob_forward", "dyt_logprob_backward", "dyt_logprob_forward_workspace_size", "dyt_adamw_step",
    "dyt_adamw_values", "RMSNorm", "RMSNormFunction", "rms_norm", "RMSNormResidual", "RMSNormResidualFunction",
    "rms_norm_residual", "Embedding", "EmbeddingFunction", "embedding", "LogProbFunction", "token_log_probs", "AdamW",
]

# DyT needs its own library only: where the block operators' is missing or from
# other sources, their names say so when they are used.
try:
    from ._block import (  # noqa: E402,F401
        BLOCK_LIB_FILE,
        block_lib,
        dyt_attn_backward,
        dyt_attn_bucket_borders,
        dyt_attn_forward,
        dyt_ln_backward,
        dyt_ln_backward_residual,
        dyt_ln_backward_workspace_size,
        dyt_ln_forward,
        dyt_ln_forward_residual,
    )
    from .block import (  # noqa: E402,F401
        Attention,
        AttentionFunction,
        KVCache,
        LayerNorm,
        LayerNormFunction,
        LayerNormResidual,
        LayerNormResidualFunction,
        attention,
        layer_norm,
        layer_norm_residual,
    )
except ImportError as _e:
    _block_missing = str(_e)
else:
    _block_missing = None

# Likewise the operators around a decoder's blocks (their binding shares the
# block operators' checks).
try:
    from ._lm import (  # noqa: E402,F401
        DYT_ADAMW_BLOCK,
        DYT_LOGPROB_MAX_TOP,
        LM_LIB_FILE,
        dyt_adamw_step,
        dyt_adamw_values,
        dyt_embed_backward,
        dyt_embed_backward_workspace_size,
        dyt_embed_forward,
        dyt_logprob_backward,
        dyt_logprob_forward,
        dyt_logprob_forward_workspace_size,
        dyt_rms_backward,
        dyt_rms_backward_residual,
        dyt_rms_backward_workspace_size,
        dyt_rms_forward,
        dyt_rms_forward_q8,
        dyt_rms_forward_residual,
        dyt_rms_forward_residual_q8,
        lm_lib,
    )
    from .lm import (  # noqa: E402,F401
        AdamW,
        Embedding,
        EmbeddingFunction,
        LogProbFunction,
        RMSNorm,
        RMSNormFunction,
        RMSNormResidual,
        RMSNormResidualFunction,
        embedding,
        rms_norm,
        rms_norm_residual,
        token_log_probs,
    )
except ImportError as _e:
    _lm_missing = str(_e)
else:
    _lm_missing = None

if _block_missing or _lm_missing:
    def __getattr__(name):
        if _block_missing and name in _BLOCK_ALL:
            raise ImportError(_block_missing)
        if _lm_missing and name in _LM_ALL:
            raise ImportError(_lm_missing)
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")

__all__ = [
    "DyT", "DyTFunction", "dyt", "DyTResidual", "DyTResidualFunction", "dyt_residual",
    "DYT_F32", "DYT_BF16", "DYT_F16", "DYT_OK", "DytError", "LIB_FILE", "lib",
    "dyt_forward", "dyt_backward", "dyt_backward_partials", "dyt_backward_finish",
    "dyt_backward_workspace_size", "dyt_backward_noalloc", "dyt_forward_residual", "dyt_backward_residual",
    "dyt_backward_residual_partials",
    "dyt_status_string", "dyt_abi_version", "dyt_get_plan", "dyt_get_forward_plan",
    "dyt_get_forward_residual_plan", "dyt_xcd_hint", "dyt_set_xcd_flip_override",
    *([] if _block_missing else _BLOCK_ALL),
    *([] if _lm_missing else _LM_ALL),
]
