"""A DeBERTa-v3 encoder on the packed layout, composed from the library's
calls (every step runs in libdfattn.so; this module only orders the calls and
holds the weights).

The pages' benchmark workload is the 12-layer DeBERTa-v3-base encoder
(DisentangledFlash README, "Benchmarks").  A layer: the fused QKV projection
(df_linear, three outputs in the attention's [T, H, d] layout); PK and PQ from
the layer's key and query projections of the layer-normalised relative
embeddings (shared attention keys); disentangled attention (df_attn_fwd,
packed); the output projection and a residual LayerNorm; the feed-forward
block (projection with GELU, projection) and a residual LayerNorm.
``Encoder.embed`` gives the rows that enter the first layer (token embedding and
LayerNorm), and ``CrossAttention`` is the layer of a decoder or a reader that
attends to the encoder's states.
Weights are synthetic (no checkpoint is available): N(0, 0.02) matrices,
N(0, 0.02) biases, LayerNorm gain 1 and shift 0.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import List

import torch

from . import binding


@dataclass
class EncoderConfig:
    hidden: int = 768
    heads: int = 12
    layers: int = 12
    ffn: int = 3072
    buckets: int = 256
    max_rel: int = 512
    eps: float = 1e-7
    vocab: int = 0  # rows of the token embeddings; 0: the caller brings hidden rows

    @property
    def span(self):
        return binding.default_span(self.buckets, self.max_rel)


def synthetic_weights(cfg: EncoderConfig, dtype=torch.bfloat16, device="cuda", seed=0):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, std=0.02):
        return (torch.randn(*shape, generator=g) * std).to(dtype).to(device)

    def ones(n):
        return torch.ones(n, dtype=dtype, device=device)

    def zeros(n):
        return torch.zeros(n, dtype=dtype, device=device)

    h, f = cfg.hidden, cfg.ffn
    layers = [dict(w_qkv=rnd(3 * h, h), b_qkv=rnd(3 * h), w_o=rnd(h, h), b_o=rnd(h), ln1_g=ones(h), ln1_b=zeros(h),
                   w_1=rnd(f, h), b_1=rnd(f), w_2=rnd(h, f), b_2=rnd(h), ln2_g=ones(h), ln2_b=zeros(h))
              for _ in range(cfg.layers)]
    shared = dict(rel_embeddings=rnd(2 * cfg.span, h), rel_g=ones(h), rel_b=zeros(h))
    if cfg.vocab:
        shared.update(word_embeddings=rnd(cfg.vocab, h), emb_g=ones(h), emb_b=zeros(h))
    return layers, shared


def synthetic_cross_weights(cfg: EncoderConfig, dtype=torch.bfloat16, device="cuda", seed=0):
    """Weights of one CrossAttention layer of the encoder's width."""
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape):
        return (torch.randn(*shape, generator=g) * 0.02).to(dtype).to(device)

    h = cfg.hidden
    w = {n: rnd(h, h) for n in ("w_q", "w_k", "w_v", "w_o")}
    w.update({n: rnd(h) for n in ("b_q", "b_k", "b_v", "b_o")})
    w.update(ln_g=torch.ones(h, dtype=dtype, device=device), ln_b=torch.zeros(h, dtype=dtype, device=device))
    return w


class Encoder:
    """encoder(hidden [T, hidden], cu_seqlens [S + 1], max_seqlen) -> [T, hidden]."""

    def __init__(self, cfg: EncoderConfig, layers: List[dict], shared: dict):
        self.cfg, self.layers, self.shared = cfg, layers, shared

    def embed(self, input_ids, stream=None, status=None):
        """Rows [T, hidden] of packed token ids [T]: their embeddings, normalised.  An id
        outside the vocabulary counts as a row of zeros; ``status`` (a device int32, as for
        ``binding.df_embedding``) reports it."""
        sh = self.shared
        rows = binding.df_embedding(input_ids, sh["word_embeddings"], status=status, stream=stream)
        return binding.df_layernorm(rows, sh["emb_g"], sh["emb_b"], eps=self.cfg.eps, stream=stream)

    def __call__(self, hidden, cu_seqlens, max_seqlen, stream=None, trace=None):
        """``trace``: an optional list; each layer appends a dict of the tensors
        its attention call took and gave (q, k, v, pk, pq, ctx), which the layer
        computes anyway (nothing extra runs)."""
        if stream is not None:
            with binding._current(stream, hidden):
                return self(hidden, cu_seqlens, max_seqlen, trace=trace)
        cfg = self.cfg
        hid, H = cfg.hidden, cfg.heads
        T = hidden.shape[0]
        sh = self.shared
        rel = binding.df_layernorm(sh["rel_embeddings"], sh["rel_g"], sh["rel_b"], eps=cfg.eps)
        ws = None
        h = hidden
        for p in self.layers:
            w, b = p["w_qkv"], p["b_qkv"]
            q, k, v = binding.qkv_projection(h, w, b, H)
            pk, pq = binding.rel_projection(rel, w[hid:2 * hid], b[hid:2 * hid], w[:hid], b[:hid], H)
            if ws is None:
                size = binding.df_attn_workspace_size(cu_seqlens.numel() - 1, H, max_seqlen, hid // H,
                                                      cfg.buckets, cfg.max_rel, cfg.span)
                ws = torch.empty(max(size, 256), dtype=torch.uint8, device=hidden.device)
            ctx = binding.df_attn_fwd(q, k, v, pk, pq, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen,
                                      buckets=cfg.buckets, max_rel=cfg.max_rel, span=cfg.span, workspace=ws)
            if trace is not None:
                trace.append(dict(q=q, k=k, v=v, pk=pk, pq=pq, ctx=ctx))
            (a,) = binding.df_linear(ctx.view(T, hid), [p["w_o"]], [p["b_o"]])
            h1 = binding.df_layernorm(a, p["ln1_g"], p["ln1_b"], residual=h, eps=cfg.eps)
            (f,) = binding.df_linear(h1, [p["w_1"]], [p["b_1"]], activation=binding.LINEAR_GELU)
            (f2,) = binding.df_linear(f, [p["w_2"]], [p["b_2"]])
            h = binding.df_layernorm(f2, p["ln2_g"], p["ln2_b"], residual=h1, eps=cfg.eps)
        return h


class CrossAttention:
    """A layer that attends to an encoder's packed states: projections, cross
    attention, output projection, residual LayerNorm.

    ``project`` gives the states' keys and values once; a program that generates
    keeps them and calls ``attend`` with one row per sequence.  ``status`` (a device
    int32, zeroed by the caller) receives what the calls report: offsets that are not
    in order, whose sequences' rows then hold anything, and waits that ran out."""

    def __init__(self, cfg: EncoderConfig, weights: dict):
        self.cfg, self.w = cfg, weights

    def project(self, states, stream=None, status=None):
        """states [T, hidden] -> k, v, each [T, heads, hidden / heads]."""
        w, H = self.w, self.cfg.heads
        outs = binding.df_linear(states, [w["w_k"], w["w_v"]], [w["b_k"], w["b_v"]], status=status, stream=stream)
        return [o.view(states.shape[0], H, self.cfg.hidden // H) for o in outs]

    def attend(self, x, k, v, cu_seqlens_q, max_seqlen_q, cu_seqlens_k, max_seqlen_k, stream=None, status=None):
        """x [Tq, hidden], packed by cu_seqlens_q, against the keys and values of the same
        sequences, packed by cu_seqlens_k -> [Tq, hidden]."""
        w, cfg = self.w, self.cfg
        T, hid = x.shape
        (q,) = binding.df_linear(x, [w["w_q"]], [w["b_q"]], status=status, stream=stream)
        ctx = binding.df_cross_attn_fwd(q.view(T, cfg.heads, hid // cfg.heads), k, v, cu_seqlens_q=cu_seqlens_q,
                                        max_seqlen_q=max_seqlen_q, cu_seqlens_k=cu_seqlens_k,
                                        max_seqlen_k=max_seqlen_k, status=status, stream=stream)
        (o,) = binding.df_linear(ctx.view(T, hid), [w["w_o"]], [w["b_o"]], status=status, stream=stream)
        return binding.df_layernorm(o, w["ln_g"], w["ln_b"], residual=x, eps=cfg.eps, stream=stream)
