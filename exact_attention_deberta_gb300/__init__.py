"""Exact DeBERTa-v2/v3 disentangled attention for NVIDIA GB300, with the steps around
it: token embeddings, projections, the cross attention that reads the states, and a
decoder's own attention (rotary positions, causal attention, a cache in 8 bits).

The computation lives in ``libdfattn.so`` (hand-written sm_103a CUDA behind the
C ABI of ``include/df_attn.h``); ``binding`` is its ctypes marshalling layer and
``synth`` draws seeded synthetic inputs.  Build the library with
``exact_attention_deberta_gb300.build.build()``.
"""

__all__ = ["binding", "build", "synth"]


def __getattr__(name):
    if name in ("df_attn_fwd", "df_attn_plan", "df_rel_index_table", "df_attn_workspace_size",
                "df_attn_supported", "df_attn_get_device_status", "df_cross_attn_fwd", "df_cross_attn_bwd",
                "df_embedding", "df_embedding_bwd", "df_self_attn_fwd", "df_self_attn_bwd", "df_rotary",
                "df_rotary_table", "df_cache_new", "df_cache_append", "df_cache_read", "df_cache_attn"):
        from . import binding
        return getattr(binding, name)
    raise AttributeError(name)
