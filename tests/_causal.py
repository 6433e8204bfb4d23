"""Calls of the causal-attention tests; inputs and bounds are those of the cross attention."""

from _cross import np64


def want(oracle, x, scale, window=0, sinks=0, with_grad=False):
    lists = {n: None if x[n] is None else x[n].cpu().numpy() for n in ("key_mask", "cu_q", "cu_k")}
    return oracle.causal_batch(np64(x["q"]), np64(x["k"]), np64(x["v"]), scale, window, sinks, lists["key_mask"],
                               lists["cu_q"], lists["cu_k"], np64(x["dout"]) if with_grad else None)


def where(x, dev):
    return dict(key_mask=dev["key_mask"], cu_seqlens_q=dev["cu_q"], cu_seqlens_k=dev["cu_k"], max_seqlen_q=x["Lq"],
                max_seqlen_k=x["Lk"])


def call(binding, x, dev, **more):
    return binding.df_self_attn_fwd(dev["q"], dev["k"], dev["v"], **where(x, dev), **more)


def call_bwd(binding, x, dev, out, stats, **more):
    return binding.df_self_attn_bwd(dev["q"], dev["k"], dev["v"], out, stats, dev["dout"], **where(x, dev), **more)
