"""Kimi Delta Attention (KDA) on MI355X (gfx950): chunkwise prefill and
recurrent decode, and the gradients of the recurrence, as hand-written HIP
kernels behind a C ABI (include/kda.h).

The Python layer only marshals arguments: torch tensors supply device memory
and the current HIP stream; every step of the operator runs in libkda.so.
"""
__all__ = ["chunk_fwd", "recurrent_fwd", "recurrent_step", "recurrent_bwd", "KdaError", "chunk_fwd_workspace_bytes",
           "recurrent_bwd_workspace_bytes", "dplr_recurrent_fwd", "chunk_fwd_noalloc",
           "dplr_chunk_fwd", "chunk_bwd", "chunk_bwd_workspace_bytes"]
# the operators of a layer around the recurrence
_LAYER = ["selective_scan_fwd", "selective_scan_step", "selective_scan_bwd", "short_conv_fwd", "short_conv_step",
          "short_conv_bwd", "layer_norm_fwd", "layer_norm_bwd", "selective_scan_fwd_workspace_bytes",
          "selective_scan_bwd_workspace_bytes", "short_conv_bwd_workspace_bytes", "layer_norm_bwd_workspace_bytes"]
# latent attention between the recurrence's layers
_LATENT = ["rotary_frequencies", "rotary_fwd", "rotary_bwd", "latent_cache_append", "latent_attention_step",
           "latent_attention_fwd", "latent_attention_bwd", "latent_attention_step_workspace_bytes",
           "latent_attention_bwd_workspace_bytes"]
__all__ += _LAYER + _LATENT


def __getattr__(name):
    if name not in __all__:
        raise AttributeError(name)
    if name in _LAYER:
        from . import layer_ops as module
    elif name in _LATENT:
        from . import latent_ops as module
    else:
        from . import ops as module
    value = globals()[name] = getattr(module, name)  # found here from now on
    return value
