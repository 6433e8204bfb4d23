"""The part of the binding that a decoder's own attention needs: causal attention with a
window and sinks, rotary positions.  Argument marshalling only, as ``binding``, whose helpers it uses and
through which every call here is reached as well (``binding.df_self_attn_fwd``)."""

from __future__ import annotations

import ctypes

import torch

from . import binding as b

__all__ = ["df_self_attn_fwd", "df_self_attn_bwd", "df_rotary", "df_rotary_table"]

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


_ll = ctypes.c_longlong
b._lib.df_rotary.argtypes = ([b._i, b._PP, ctypes.POINTER(b._i), ctypes.POINTER(_ll), b._PP, ctypes.POINTER(_ll), b._vp] +
                             [b._i] * 6 + [b._vp, ctypes.c_float, b._i, b._vp])
b._lib.df_rotary.restype = b._i
b._lib.df_rotary_table.argtypes = [b._i] + [ctypes.c_double] * 5 + [b._vp]
b._lib.df_rotary_table.restype = b._i


def df_rotary_table(rot, base=10000.0, factor=1.0, original_len=0.0, low=1.0, high=32.0, device="cuda"):
    """Frequencies of ``df_rotary`` for ``rot`` columns (int64 [rot / 2] on ``device``, made
    once): base^(-2i / rot), for long contexts divided by ``factor``, all of them
    (``original_len`` 0) or, by parts, those that turn less than ``high`` times within
    ``original_len`` positions."""
    table = torch.empty(max(int(rot) // 2, 1), dtype=torch.int64)
    b._check(b._lib.df_rotary_table(int(rot), float(base), float(factor), float(original_len), float(low), float(high),
                                    table.data_ptr()), "df_rotary_table")
    return table.to(device)


def _token_stride(name, x, lead):
    """Elements between tokens of [..., heads, d]: the leading dimensions as one."""
    st, n = x.stride(), 1
    if st[-1] != 1 and x.shape[-1] > 1 or st[-2] != x.shape[-1] and x.shape[-2] > 1:
        raise ValueError(f"{name}: heads and columns must be next to one another")
    step = x.shape[-2] * x.shape[-1]
    for i in range(lead - 1, -1, -1):
        if x.shape[i] > 1:
            if n == 1:
                step = st[i]
            elif st[i] != n * step:
                raise ValueError(f"{name}: tokens must be a constant distance apart")
            n *= x.shape[i]
    return step


def df_rotary(x, positions, table, *, interleaved=False, inverse=False, amplitude=1.0, out=None, stream=None):
    """Rotary positions of ``x`` [..., heads, d], or of several such tensors (queries and keys)
    that share ``positions`` [...] (int32 or int64), by ``table`` (``df_rotary_table``): the
    first 2 * len(table) columns of each head, as pairs half of those apart or, with
    ``interleaved``, next to each other.  ``inverse`` is the gradient.  ``out`` may be ``x``
    itself.  Tokens may be parts of wider rows."""
    xs = (x,) if isinstance(x, torch.Tensor) else tuple(x)
    if stream is not None:
        with b._current(stream, xs[0] if xs else None):
            return df_rotary(x, positions, table, interleaved=interleaved, inverse=inverse, amplitude=amplitude, out=out)
    n = len(xs)
    if not 1 <= n <= 2:
        raise ValueError("x must be one tensor or two")
    dt, lead, d = xs[0].dtype, xs[0].shape[:-2], xs[0].shape[-1]
    if dt not in b._DTYPE or any(t.dtype != dt or t.dim() < 3 or t.shape[:-2] != lead or t.shape[-1] != d for t in xs):
        raise ValueError("x must be bf16, fp16 or fp32 tensors [..., heads, d] that share all but heads")
    if positions.dtype not in (torch.int32, torch.int64) or positions.shape != lead:
        raise ValueError("positions must be int32 or int64, of x's shape without heads and columns")
    if table.dtype != torch.int64 or table.dim() != 1:
        raise ValueError("table must be what df_rotary_table gives")
    if out is None:
        outs = tuple(torch.empty(t.shape, dtype=dt, device=t.device) for t in xs)
    else:
        outs = (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if len(outs) != n or any(o.dtype != dt or o.shape != t.shape for o, t in zip(outs, xs)):
            raise ValueError("out must match x in number, shape and dtype")
    idx = b._on_device((positions, table), "positions table")
    if any(t.get_device() != idx for t in xs + outs):
        raise ValueError("x and out must be CUDA tensors on the device of positions")
    T, k = positions.numel(), len(lead)
    b._int_sizes(tokens=T, columns=d)
    strides = [(_ll * n)(*[_token_stride(name, t, k) for t in ts]) for name, ts in (("x", xs), ("out", outs))]
    b._check(b._call_on(idx, b._lib.df_rotary, n, b._ptr_array(xs), (b._i * n)(*[t.shape[-2] for t in xs]), strides[0],
                        b._ptr_array(outs), strides[1], positions.data_ptr(), 1 if positions.dtype == torch.int64 else 0,
                        T, d, 2 * table.numel(), 1 if interleaved else 0, 1 if inverse else 0, table.data_ptr(),
                        float(amplitude), b._DTYPE[dt]), "df_rotary")
    return outs[0] if isinstance(x, torch.Tensor) else list(outs)
