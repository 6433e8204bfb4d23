"""The CrossAttention layer against the float64 oracle, element by element at the roundings'
worst and sequence by sequence at their root mean square, with weights that make the
attention matter: the latter bound is far below what leaving the attention out,
attending across sequences, attending evenly or to another head's keys changes."""

import numpy as np
import pytest
import torch

import oracle
from _cross import U32, np64, out_bound

pytestmark = pytest.mark.gpu


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads", [4, 2])
def test_attend_within_roundings(lib, dtype, heads):
    from exact_attention_deberta_gb300.encoder import CrossAttention, EncoderConfig
    hid, d = 256, 256 // heads
    cfg = EncoderConfig(hidden=hid, heads=heads)
    g = torch.Generator().manual_seed(heads)
    rnd = lambda std, *s: (torch.randn(*s, generator=g) * std).to(dtype).cuda()  # noqa: E731
    w = {n: rnd(s, hid, hid) for n, s in (("w_q", 0.1), ("w_k", 0.1), ("w_v", 0.06), ("w_o", 0.06))}
    w.update({n: rnd(0.1, hid) for n in ("b_q", "b_k", "b_v", "b_o", "ln_b")}, ln_g=1 + rnd(0.1, hid))
    n_src, n_tgt = [150, 6, 77], [9, 30, 4]
    cu_k, cu_q = _cu(n_src), _cu(n_tgt)
    states, x = rnd(1.0, sum(n_src), hid), rnd(1.0, sum(n_tgt), hid)
    cross = CrossAttention(cfg, w)
    k, v = cross.project(states)
    out = cross.attend(x, k, v, cu_q, max(n_tgt), cu_k, max(n_src))
    at = [int(c) for c in cu_q.cpu()[:3]]  # the first token of each sequence, by itself
    one = cross.attend(x[at].contiguous(), k, v, _cu([1, 1, 1]), 1, cu_k, max(n_src))

    ww, half = {n: np64(t) for n, t in w.items()}, torch.finfo(dtype).eps / 2
    q = np64(lib.df_linear(x, [w["w_q"]], [w["b_q"]])[0]).reshape(-1, heads, d)
    kk, vv, xx, cq, ck = np64(k), np64(v), np64(x), cu_q.cpu().numpy(), cu_k.cpu().numpy()

    def layer(ctx):  # what follows the attention, and what a row's normalisation divides by
        o = ctx.reshape(-1, hid) @ ww["w_o"].T + ww["b_o"]
        y = xx + o
        return o, y, oracle.layer_norm(y, ww["ln_g"], ww["ln_b"], cfg.eps)

    r = oracle.cross_batch(q, kk, vv, d ** -0.5, cu_q=cq, cu_k=ck)
    o, y, want = layer(r["out"])
    sigma = np.sqrt(y.var(axis=1, keepdims=True) + cfg.eps)
    n = (y - y.mean(axis=1, keepdims=True)) / sigma
    mean = lambda z: z.mean(axis=1, keepdims=True)  # noqa: E731
    # The attention's output: its weights' rounding and its own (_cross.py).  The projection's:
    # 256 additions in fp32 and the result's rounding.  Through (y - mean) / sigma to first
    # order, 5 % for what is left, 1e-5 for its fp32, and the result's rounding.
    ctx = sum(out_bound(r, dtype, d)).reshape(-1, hid)
    fp32 = (hid + 2) * U32 * (np.abs(r["out"]).reshape(-1, hid) @ np.abs(ww["w_o"]).T + np.abs(ww["b_o"]))
    last = 1e-5 * (1 + np.abs(want))
    e = ctx @ np.abs(ww["w_o"]).T + fp32
    e = e + half * (np.abs(o) + e)
    e = 1.05 * (e + mean(e) + np.abs(n) * mean(np.abs(n) * e)) / sigma * np.abs(ww["ln_g"]) + last
    worst = e + half * (np.abs(want) + e)
    # the same with independent signs: squares add up
    e2 = (ctx ** 2) @ (ww["w_o"] ** 2).T + fp32 ** 2 + (half * o) ** 2
    e2 = 1.05 ** 2 * (e2 + (1 + n ** 2) * mean(e2) / hid * 2) / sigma ** 2 * ww["ln_g"] ** 2 + last ** 2
    rms = np.sqrt(e2 + (half * want) ** 2)
    norm = lambda z, s: float(np.sqrt((z[cq[s]:cq[s + 1]] ** 2).sum()))  # noqa: E731
    # what mistakes would change is far outside of it, in every sequence
    other_cu = dict(cu_q=np.array([0, len(q)]), cu_k=np.array([0, len(kk)]))
    mistakes = [0 * r["out"]] + [oracle.cross_batch(a, b, vv, d ** -0.5, **c)["out"] for a, b, c in (
        (q, kk, other_cu), (0 * q, kk, dict(cu_q=cq, cu_k=ck)), (q, kk[:, ::-1], dict(cu_q=cq, cu_k=ck)))]
    for s in range(3):
        for m in mistakes:
            assert norm(layer(m)[2] - want, s) > 25 * norm(rms, s)
    err = np.abs(np64(out) - want)
    assert (err <= worst).all()
    assert all(norm(err, s) <= norm(rms, s) for s in range(3))
    assert (np.abs(np64(one) - want[at]) <= worst[at]).all()
