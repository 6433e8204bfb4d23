"""The part of the binding that a decoder's own attention needs: causal attention with a
window and sinks.  Argument marshalling only, as ``binding``, whose helpers it uses and
through which every call here is reached as well (``binding.df_self_attn_fwd``)."""

from __future__ import annotations

import ctypes

from . import binding as b

__all__ = ["df_self_attn_fwd", "df_self_attn_bwd"]

b._lib.df_self_attn_fwd.argtypes = [b._vp] * 6 + [b._i] * 8 + [ctypes.c_float] + [b._i] * 3 + [b._vp] * 5
b._lib.df_self_attn_fwd.restype = b._i
b._lib.df_self_attn_bwd.argtypes = [b._vp] * 10 + [b._i] * 8 + [ctypes.c_float] + [b._i] * 3 + [b._vp] * 5 + [b._sz, b._vp]
b._lib.df_self_attn_bwd.restype = b._i


def _reach(window, sinks):
    window, sinks = int(window or 0), int(sinks)
    b._int_sizes(window=window, sinks=sinks)
    return window, sinks


def df_self_attn_fwd(q, k, v, key_mask=None, cu_seqlens_q=None, cu_seqlens_k=None, *, max_seqlen_q=None,
                     max_seqlen_k=None, window=0, sinks=0, scale=None, out=None, with_stats=False, status=None,
                     stream=None):
    """Causal attention: the queries are the last tokens of their sequence (all of them, or
    the next part of a prompt) and see the keys up to their own position; with ``window``
    the last ``window`` of those and the sequence's first ``sinks``.  Layouts, arguments and
    results as ``df_cross_attn_fwd``."""
    if stream is not None:
        with b._current(stream, q):
            return df_self_attn_fwd(q, k, v, key_mask, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=max_seqlen_q,
                                    max_seqlen_k=max_seqlen_k, window=window, sinks=sinks, scale=scale, out=out,
                                    with_stats=with_stats, status=status)
    return b._attn_fwd(b._lib.df_self_attn_fwd, "df_self_attn_fwd", _reach(window, sinks), q, k, v, key_mask, cu_seqlens_q,
                     cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, out, with_stats, status)


def df_self_attn_bwd(q, k, v, out, stats, dout, key_mask=None, cu_seqlens_q=None, cu_seqlens_k=None, *,
                     max_seqlen_q=None, max_seqlen_k=None, window=0, sinks=0, scale=None, grads=None, workspace=None,
                     status=None, stream=None):
    """Gradients (dq, dk, dv), in the inputs' dtype, of ``df_self_attn_fwd`` with the same
    arguments; ``out`` and ``stats`` as its call with ``with_stats`` gave them.  The
    workspace is ``df_cross_attn_bwd_workspace_size``."""
    if stream is not None:
        with b._current(stream, q):
            return df_self_attn_bwd(q, k, v, out, stats, dout, key_mask, cu_seqlens_q, cu_seqlens_k,
                                    max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k, window=window, sinks=sinks,
                                    scale=scale, grads=grads, workspace=workspace, status=status)
    return b._attn_bwd(b._lib.df_self_attn_bwd, "df_self_attn_bwd", _reach(window, sinks), q, k, v, out, stats, dout,
                     key_mask, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, scale, grads, workspace, status)
