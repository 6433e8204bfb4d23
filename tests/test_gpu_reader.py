"""The embedding and the cross attention together, as a program that reads an
encoder's states uses them: tokens -> encoder -> states -> cross attention of
target tokens, one target token at a time, and a training step down to the
gradient of the embedding table.  Against the float64 oracles."""

import numpy as np
import pytest
import torch

import oracle
from _cross import np64

pytestmark = pytest.mark.gpu


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()


def test_tokens_to_states_to_reader(lib):
    from exact_attention_deberta_gb300.encoder import (CrossAttention, Encoder, EncoderConfig,
                                                       synthetic_cross_weights, synthetic_weights)
    cfg = EncoderConfig(hidden=256, heads=4, layers=1, ffn=512, vocab=500)
    layers, shared = synthetic_weights(cfg, seed=2)
    w = synthetic_cross_weights(cfg, seed=3)
    enc, cross = Encoder(cfg, layers, shared), CrossAttention(cfg, w)
    n_src, n_tgt = [150, 1, 77], [9, 30, 4]
    rng = np.random.default_rng(4)
    src, tgt = (rng.integers(0, cfg.vocab, sum(n)) for n in (n_src, n_tgt))
    cu_k, cu_q = _cu(n_src), _cu(n_tgt)
    x = enc.embed(torch.from_numpy(src).cuda())
    states = enc(x, cu_k, max(n_src))
    k, v = cross.project(states)
    y = enc.embed(torch.from_numpy(tgt).cuda())
    out = cross.attend(y, k, v, cu_q, max(n_tgt), cu_k, max(n_src))

    # the embedded rows: a LayerNorm of the table's rows, in bf16
    sh = {n: np64(t) for n, t in shared.items()}
    rows = oracle.layer_norm(oracle.embed(src, sh["word_embeddings"], 1.0), sh["emb_g"], sh["emb_b"], cfg.eps)
    half = torch.finfo(torch.bfloat16).eps / 2
    assert (np.abs(np64(x) - rows) <= half * np.abs(rows) * 1.01 + 1e-5 * (1 + np.abs(rows))).all()
    # the reader on its own (rounded) inputs
    ww = {n: np64(t) for n, t in w.items()}
    q = np64(lib.df_linear(y, [w["w_q"]], [w["b_q"]])[0]).reshape(-1, 4, 64)
    ctx = oracle.cross_batch(q, np64(k), np64(v), 0.125, cu_q=cu_q.cpu().numpy(), cu_k=cu_k.cpu().numpy())["out"]
    o = ctx.reshape(-1, 256) @ ww["w_o"].T + ww["b_o"]
    want = oracle.layer_norm(np64(y) + o, ww["ln_g"], ww["ln_b"], cfg.eps)
    # the attention's output and the projection's are rounded to bf16 before a
    # LayerNorm of rows whose standard deviation is about 1, then the result is
    attn = half * (1.01 * np.abs(ctx).max() * np.abs(ww["w_o"]).sum(axis=1).max() * 2 + np.abs(o).max())
    assert np.abs(np64(out) - want).max() <= 1.1 * attn * (2 + np.abs(want).max()) + half * np.abs(want).max()

    # one target token per sequence, with the keys and values kept: the same rows
    at = [int(c) for c in cu_q.cpu()[:3]]
    one = cross.attend(y[at].contiguous(), k, v, _cu([1, 1, 1]), 1, cu_k, max(n_src))
    # another tiling of the keys adds in another order: within the bound above
    assert np.abs(np64(one) - want[at]).max() <= 1.1 * attn * (2 + np.abs(want).max()) + half * np.abs(want).max()


def test_training_step_down_to_the_table(lib):
    # queries are scaled embeddings; the gradient of sum(out * dout) by the table
    V, H, Hk, d, scale = 40, 4, 2, 64, 0.5
    n_src, n_tgt = [90, 200], [33, 60]
    rng = np.random.default_rng(1)
    g = torch.Generator().manual_seed(2)
    normal = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    table, k, v, dout = normal(V, H * d), normal(290, Hk, d), normal(290, Hk, d), normal(93, H, d)
    ids = rng.integers(0, V, 93)
    dev = torch.from_numpy(ids).cuda()
    cu_q, cu_k = _cu(n_tgt), _cu(n_src)
    kw = dict(cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, max_seqlen_q=60, max_seqlen_k=200)
    q = lib.df_embedding(dev, table, scale=scale).view(93, H, d)
    out, stats = lib.df_cross_attn_fwd(q, k, v, with_stats=True, **kw)
    dq, dk, dv = lib.df_cross_attn_bwd(q, k, v, out, stats, dout, **kw)
    grad = lib.df_embedding_bwd(dev, dq.view(93, H * d), V, scale=scale, padding_idx=3)

    w = oracle.cross_batch(np64(q), np64(k), np64(v), d ** -0.5, cu_q=cu_q.cpu().numpy(), cu_k=cu_k.cpu().numpy(),
                           dout=np64(dout))
    want, _, _ = oracle.embed_grad(ids, w["dq"].reshape(93, H * d), V, scale, padding_idx=3)
    # the table's gradient carries dq's roundings (three halves of bf16, _cross.py), the
    # sums over equal tokens add none of that size
    norm = lambda z: float(np.sqrt((z ** 2).sum()))  # noqa: E731
    assert norm(np64(grad) - want) <= 3 * 2.0 ** -8 * norm(want)
    assert (np64(grad)[3] == 0).all()


@pytest.mark.parametrize("handle", [False, True])
def test_stream_given_as_an_argument(lib, handle):
    # results and workspaces then belong to that stream: freed ones are not handed out
    # to the current stream while it still runs
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, v, dout = n(4, 300, 4, 64), n(4, 500, 4, 64), n(4, 500, 4, 64), n(4, 300, 4, 64)
    table, ids, drows = n(3000, 256), torch.randint(0, 3000, (9000,), generator=g).cuda(), n(9000, 256)
    def run(**on):
        o, stats = lib.df_cross_attn_fwd(q, k, v, with_stats=True, **on)
        return (o, stats.lse, *lib.df_cross_attn_bwd(q, k, v, o, stats, dout, **on),
                lib.df_embedding(ids, table, **on), lib.df_embedding_bwd(ids, drows, 3000, **on))
    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = run(stream=side.cuda_stream if handle else side)
        junk = [torch.full((4, 300, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 4
