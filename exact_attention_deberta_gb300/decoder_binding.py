"""The part of the binding that a decoder's own attention needs: causal attention with a
window and sinks, rotary positions, the 8-bit paged cache.  Argument marshalling only, as ``binding``, whose helpers it uses and
through which every call here is reached as well (``binding.df_self_attn_fwd``)."""

from __future__ import annotations

import ctypes

import torch

from . import binding as b

__all__ = ["df_self_attn_fwd", "df_self_attn_bwd", "df_rotary", "df_rotary_table", "df_cache_new",
           "df_cache_append", "df_cache_read", "df_cache_attn"]

b._lib.df_self_attn_fwd.argtypes = [b._vp] * 6 + [b._i] * 8 + [ctypes.c_float] + [b._i] * 3 + [b._vp] * 5
b._lib.df_self_attn_fwd.restype = b._i
b._lib.df_self_attn_bwd.argtypes = [b._vp] * 10 + [b._i] * 8 + [ctypes.c_float] + [b._i] * 3 + [b._vp] * 5 + [b._sz, b._vp]
b._lib.df_self_attn_bwd.restype = b._i


_INT = 2 ** 31  # sizes go to the library as C ints


def _reach(window, sinks):
    window, sinks = int(window or 0), int(sinks)
    if not (0 <= window < _INT and 0 <= sinks < _INT):
        raise ValueError(f"window = {window} or sinks = {sinks} is out of range")
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
b._lib.df_rotary.argtypes = ([b._vp, b._i, _ll, b._vp, _ll] * 2 + [b._vp] + [b._i] * 6 +
                             [b._vp, ctypes.c_float, b._i, b._vp])
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
    if x.is_contiguous():
        return x.shape[-2] * x.shape[-1]
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
    first, dt = xs[0], xs[0].dtype
    lead, d = first.shape[:-2], first.shape[-1]
    if dt not in b._DTYPE or len(lead) < 1 or (n == 2 and (xs[1].dtype != dt or xs[1].shape[:-2] != lead or
                                                           xs[1].shape[-1] != d)):
        raise ValueError("x must be bf16, fp16 or fp32 tensors [..., heads, d] that share all but heads")
    if positions.dtype not in (torch.int32, torch.int64) or positions.shape != lead:
        raise ValueError("positions must be int32 or int64, of x's shape without heads and columns")
    if table.dtype != torch.int64 or table.dim() != 1:
        raise ValueError("table must be what df_rotary_table gives")
    if out is None:
        outs = tuple([torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=dt, device=t.device)
                      for t in xs])
    else:
        outs = (out,) if isinstance(out, torch.Tensor) else tuple(out)
        if len(outs) != n or any(o.dtype != dt or o.shape != t.shape for o, t in zip(outs, xs)):
            raise ValueError("out must match x in number, shape and dtype")
    idx = b._on_device((positions, table), "positions table")
    for t in xs + outs:
        if t.get_device() != idx:
            raise ValueError("x and out must be CUDA tensors on the device of positions")
    T, k = positions.numel(), len(lead)
    if T >= _INT or d >= _INT:
        raise ValueError("x is too large")
    rows = []
    for t, o in zip(xs, outs):
        rows += (t.data_ptr(), t.shape[-2], _token_stride("x", t, k), o.data_ptr(), _token_stride("out", o, k))
    if n == 1:
        rows += (None, 0, 0, None, 0)
    b._check(b._call_on(idx, b._lib.df_rotary, *rows, positions.data_ptr(), 1 if positions.dtype == torch.int64 else 0,
                        T, d, 2 * table.numel(), 1 if interleaved else 0, 1 if inverse else 0, table.data_ptr(),
                        float(amplitude), b._DTYPE[dt]), "df_rotary")
    return outs[0] if isinstance(x, torch.Tensor) else list(outs)


b._lib.df_cache_bytes.argtypes = [b._i] * 4
b._lib.df_cache_bytes.restype = b._sz
b._lib.df_cache_append.argtypes = [b._vp] * 3 + [b._i] * 6 + [b._vp, b._i, b._i, b._vp, b._i, b._vp, b._vp, b._vp]
b._lib.df_cache_append.restype = b._i
b._lib.df_cache_read.argtypes = [b._vp, b._i, b._i, b._vp, b._i, b._vp, b._vp] + [b._i] * 6 + [b._vp] * 4
b._lib.df_cache_read.restype = b._i
b._lib.df_cache_attn.argtypes = ([b._vp, b._vp] + [b._i] * 6 + [ctypes.c_float] + [b._i] * 4 + [b._vp, b._i, b._i, b._vp,
                                 b._i, b._vp, b._i] + [b._vp] * 4)
b._lib.df_cache_attn.restype = b._i

BLOCK = 16  # tokens that share a scale


def df_cache_new(n_pages, heads, page, d, device="cuda"):
    """Memory of a cache of ``n_pages`` pages of ``page`` tokens: uint8
    [n_pages, heads, page / 16, 32 d + 16], not initialised."""
    n_pages, heads, page, d = int(n_pages), int(heads), int(page), int(d)
    b._int_sizes(n_pages=n_pages, heads=heads, page=page, d=d)
    if b._lib.df_cache_bytes(n_pages, heads, page, d) == 0:
        raise ValueError("pages must be multiples of 16 tokens, the head size a multiple of 32 up to 128")
    return torch.empty((n_pages, heads, page // BLOCK, 32 * d + 16), dtype=torch.uint8, device=device)


def _on_device(tensors, names):
    """``binding._on_device`` for tensors that are mostly as they should be (a small call is
    bound by the host)."""
    idx = tensors[0].get_device()
    if idx >= 0:
        for t in tensors:
            if t is not None and not (t.get_device() == idx and t.is_contiguous()):
                break
        else:
            return idx
    return b._on_device(tensors, names)


def _cache_shape(cache, page_table, lengths):
    """(sequences, heads, head size, pages, tokens of a page, pages of a sequence)."""
    shape, pages = cache.shape, page_table.shape
    if cache.dtype != torch.uint8 or len(shape) != 4 or shape[3] < 48 or shape[3] % 32 != 16:
        raise ValueError("cache must be uint8 [n_pages, heads, page / 16, 32 d + 16]")
    if page_table.dtype != torch.int32 or len(pages) != 2:
        raise ValueError("page_table must be int32 [B, max_pages]")
    if lengths.dtype != torch.int32 or lengths.shape != pages[:1]:
        raise ValueError("lengths must be int32 [B]")
    n_pages, heads, per, record = shape
    if n_pages >= _INT or per >= _INT // BLOCK or pages[0] >= _INT or pages[1] >= _INT:
        raise ValueError("the cache or its page table is too large")
    return pages[0], heads, record // 32, n_pages, per * BLOCK, pages[1]


def _cache_rows(name, x, cu, B):
    """(length, rows) of [B, n, ..] or, with offsets, [total, ..]."""
    shape = x.shape
    if len(shape) != (4 if cu is None else 3):
        raise ValueError(f"{name} must be [B, n, heads, d], or [total, heads, d] with cu_seqlens")
    if cu is None:
        if shape[0] != B:
            raise ValueError(f"{name} and lengths disagree on the number of sequences")
        n, total = shape[1], shape[0] * shape[1]
    else:
        if cu.dtype != torch.int32 or cu.dim() != 1 or cu.shape[0] != B + 1:
            raise ValueError("cu_seqlens must be an int32 vector [B + 1]")
        n, total = 0, shape[0]
    if total >= _INT:
        raise ValueError(f"{name} has too many rows")
    return n, total


def df_cache_append(k, v, cache, page_table, lengths, cu_seqlens=None, *, status=None, stream=None):
    """Appends tokens to ``cache`` (``df_cache_new``): k, v [B, n, heads, d], or packed
    [total, heads, d] with cu_seqlens, become the tokens from ``lengths`` [B] on of their
    sequences, whose pages are ``page_table`` [B, max_pages] (int32).  ``lengths`` itself is
    the caller's to add to.  Returns ``cache``."""
    if stream is not None:
        with b._current(stream, k):
            return df_cache_append(k, v, cache, page_table, lengths, cu_seqlens, status=status)
    idx = _on_device((k, v, cache, page_table, lengths, cu_seqlens, status),
                       "k v cache page_table lengths cu_seqlens status")
    B, heads, d, n_pages, page, max_pages = _cache_shape(cache, page_table, lengths)
    if k.dtype not in b._DTYPE or v.dtype != k.dtype or v.shape != k.shape or tuple(k.shape[-2:]) != (heads, d):
        raise ValueError("k and v must be bf16 or fp16, with the cache's heads and head size")
    n, total = _cache_rows("k", k, cu_seqlens, B)
    if status is not None:
        b._status_word(status)
    b._check(b._call_on(idx, b._lib.df_cache_append, k.data_ptr(), v.data_ptr(), b._addr(cu_seqlens), B, heads, n, total, d,
                        b._DTYPE[k.dtype], cache.data_ptr(), n_pages, page, page_table.data_ptr(), max_pages,
                        lengths.data_ptr(), b._addr(status)), "df_cache_append")
    return cache


def df_cache_read(cache, page_table, lengths, cu_seqlens=None, *, rows=None, dtype=torch.bfloat16, out=None, status=None,
                  stream=None):
    """The tokens that sequences hold, as (k, v) in ``dtype``: [B, rows, heads, d], or
    [rows, heads, d] packed by cu_seqlens.  Rows beyond a sequence's length are zeros."""
    if stream is not None:
        with b._current(stream, cache):
            return df_cache_read(cache, page_table, lengths, cu_seqlens, rows=rows, dtype=dtype, out=out, status=status)
    B, heads, d, n_pages, page, max_pages = _cache_shape(cache, page_table, lengths)
    if out is None:
        if rows is None:
            raise ValueError("rows (of each sequence, or of all of them with cu_seqlens) or out must be given")
        shape = (int(rows), heads, d) if cu_seqlens is not None else (B, int(rows), heads, d)
        if not 0 <= shape[-3] < _INT:
            raise ValueError("rows is out of range")
        k = torch.empty(shape, dtype=dtype, device=cache.device)
        out = k, torch.empty_like(k)
    k, v = out
    if k.dtype not in b._DTYPE or v.dtype != k.dtype or v.shape != k.shape or tuple(k.shape[-2:]) != (heads, d):
        raise ValueError("out must be two tensors of bf16, fp16 or fp32, with the cache's heads and head size")
    idx = _on_device((cache, page_table, lengths, cu_seqlens, k, v, status),
                       "cache page_table lengths cu_seqlens out out status")
    n, total = _cache_rows("out", k, cu_seqlens, B)
    if status is not None:
        b._status_word(status)
    b._check(b._call_on(idx, b._lib.df_cache_read, cache.data_ptr(), n_pages, page, page_table.data_ptr(), max_pages,
                        lengths.data_ptr(), b._addr(cu_seqlens), B, heads, n, total, d, b._DTYPE[k.dtype], k.data_ptr(),
                        v.data_ptr(), b._addr(status)), "df_cache_read")
    return k, v


def df_cache_attn(q, cache, page_table, lengths, cu_seqlens_q=None, *, max_seqlen_q=None, max_length=None, causal=True,
                  window=0, sinks=0, scale=None, out=None, lse=None, status=None, stream=None):
    """Attention of a few queries for each sequence, [B, Lq, H, d] or packed [T, H, d] with
    cu_seqlens_q, to the tokens in ``cache``.  ``causal``: the queries are the last of the
    ``lengths`` tokens (append them first) and see those up to their own position, with
    ``window`` and ``sinks`` as ``df_self_attn_fwd``; otherwise every token.  ``max_length``
    bounds ``lengths`` (default: what the page table has room for).  ``lse`` may be a float32
    tensor [..., H] that receives the rows' log-sum-exp."""
    if stream is not None:
        with b._current(stream, q):
            return df_cache_attn(q, cache, page_table, lengths, cu_seqlens_q, max_seqlen_q=max_seqlen_q,
                                 max_length=max_length, causal=causal, window=window, sinks=sinks, scale=scale, out=out,
                                 lse=lse, status=status)
    idx = _on_device((q, cache, page_table, lengths, cu_seqlens_q, out, lse, status),
                       "q cache page_table lengths cu_seqlens_q out lse status")
    B, heads, d, n_pages, page, max_pages = _cache_shape(cache, page_table, lengths)
    if q.dtype not in b._DTYPE or q.shape[-1] != d:
        raise ValueError("q must be bf16 or fp16, with the cache's head size")
    Lq, total = _cache_rows("q", q, cu_seqlens_q, B)
    if cu_seqlens_q is not None:
        if max_seqlen_q is None:
            raise ValueError("packed q needs max_seqlen_q (an upper bound of every length)")
        Lq = int(max_seqlen_q)
    window, sinks = _reach(window, sinks)
    max_length = min(max_pages * page, _INT - 1) if max_length is None else int(max_length)
    if not (0 <= Lq < _INT and 0 <= max_length < _INT):
        raise ValueError("max_seqlen_q or max_length is out of range")
    if out is None:
        out = torch.empty_like(q)
    elif out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("out must match q in shape and dtype")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:-1]):
        raise ValueError("lse must be float32, [..., H]")
    if status is not None:
        b._status_word(status)
    b._check(b._call_on(idx, b._lib.df_cache_attn, q.data_ptr(), b._addr(cu_seqlens_q), B, q.shape[-2], heads, Lq, total, d,
                        d ** -0.5 if scale is None else float(scale), 1 if causal else 0, window, sinks, b._DTYPE[q.dtype],
                        cache.data_ptr(), n_pages, page, page_table.data_ptr(), max_pages, lengths.data_ptr(), max_length,
                        out.data_ptr(), b._addr(lse), b._addr(status)), "df_cache_attn")
    return out
