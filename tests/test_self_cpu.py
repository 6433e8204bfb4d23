"""Causal attention without a GPU: the oracle against torch's own attention in float64 and
against difference quotients, and the host refusals of the entry points."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from _causal import want
from _cross import inputs, np64


@pytest.fixture(scope="module")
def binding():
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding as b
    return b


@pytest.mark.parametrize("n,m,window,sinks", [(1, 1, 0, 0), (5, 5, 2, 1), (3, 9, 4, 2), (9, 4, 2, 0), (4, 8, 100, 3)])
def test_visible_by_the_rule(n, m, window, sinks):
    got = oracle.visible(n, m, window, sinks)
    for i in range(n):
        p = i + m - n
        for j in range(m):
            assert got[i, j] == (j <= p and (window == 0 or p - j < window or j < sinks))


@pytest.mark.parametrize("G,window,sinks", [(1, 0, 0), (3, 4, 2)])
def test_oracle_matches_autograd(G, window, sinks):
    x = inputs(3, 2 * G, 2, 16, 7, 11, torch.float64, "padded", "masked", seed=1, nk=[11, 9, 8])
    x["key_mask"][:, 0] = 1
    q, k, v = (x[n].clone().requires_grad_(True) for n in ("q", "k", "v"))
    kk, vv = (t.repeat_interleave(G, dim=2).transpose(1, 2) for t in (k, v))
    seen = torch.from_numpy(oracle.visible(7, 11, window, sinks))[None, None] & (x["key_mask"] != 0)[:, None, None, :]
    assert bool(seen.any(dim=-1).all()) or window  # (rows without a key: torch gives NaN)
    out = torch.nn.functional.scaled_dot_product_attention(q.transpose(1, 2), kk, vv, attn_mask=seen,
                                                           scale=0.3).transpose(1, 2)
    out.backward(x["dout"])
    w = want(oracle, x, 0.3, window, sinks, with_grad=True)
    for name, t in (("out", out.detach()), ("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
        assert np.allclose(w[name], t.numpy(), atol=1e-11), name


def test_oracle_gradients_are_difference_quotients():
    x = inputs(2, 4, 2, 8, 4, 6, torch.float64, "packed", "packed", seed=2, nq=[2, 4], nk=[5, 3])
    w = want(oracle, x, 0.4, 2, 1, with_grad=True)
    g = np64(x["dout"])
    assert (w["out"][2] == 0).all() and np.isinf(w["lse"][2]).all()  # the last sequence's first row sees no key
    for name in ("q", "k", "v"):
        flat = x[name].view(-1)
        for i in range(0, flat.numel(), 7):
            keep, got = float(flat[i]), []
            for s in (1e-4, -1e-4):
                flat[i] = keep + s
                got.append((want(oracle, x, 0.4, 2, 1)["out"] * g).sum())
            flat[i] = keep
            assert abs((got[0] - got[1]) / 2e-4 - w["d" + name].reshape(-1)[i]) < 1e-6


def _call(b, grad, **over):
    a = dict(q=0x10000, k=0x20000, v=0x30000, mask=None, cu_q=None, cu_k=None, B=2, H=4, Hk=2, Lq=3, Lk=9, Tq=6, Tk=18,
             d=64, scale=0.125, window=0, sinks=0, dtype=0, out=0x40000, lo=None, lse=0x50000, dout=0x60000, dq=0x70000,
             dk=0x80000, dv=0x90000, ws=0xa0000, bytes=1 << 20)
    a.update(over)
    p = lambda n: None if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    mid = [p("mask"), p("cu_q"), p("cu_k")] + [a[n] for n in ("B", "H", "Hk", "Lq", "Lk", "Tq", "Tk", "d", "scale", "window",
                                                              "sinks", "dtype")]
    if not grad:
        return b.raw_library.df_self_attn_fwd(p("q"), p("k"), p("v"), *mid, p("out"), p("lo"), p("lse"), None, None)
    return b.raw_library.df_self_attn_bwd(p("q"), p("k"), p("v"), p("out"), p("lo"), p("lse"), p("dout"), *mid, p("dq"),
                                          p("dk"), p("dv"), None, p("ws"), a["bytes"], None)


REFUSED = [(dict(window=-1), 1), (dict(sinks=-1), 1), (dict(q=None), 1), (dict(H=3), 1), (dict(Tq=7), 1),
           (dict(scale=float("nan")), 1), (dict(mask=0xb0000, cu_k=0xc0000), 1), (dict(dtype=2), 2), (dict(d=60), 2),
           (dict(d=136), 2), (dict(H=258, Hk=2), 2), (dict(v=0x30008), 3)]


@pytest.mark.parametrize("over,status", REFUSED)
def test_entry_points_refuse_on_the_host(binding, over, status):
    assert _call(binding, False, **over) == status, over
    assert _call(binding, True, **over) == status, over


def test_results_that_overlap_are_refused(binding):
    b = binding
    assert _call(b, False, out=0x10000) == b.DF_ERR_INVALID_ARG
    assert _call(b, False, lo=0x40000) == b.DF_ERR_INVALID_ARG
    assert _call(b, True, dk=0x20010) == b.DF_ERR_INVALID_ARG
    assert _call(b, True, bytes=64) == b.DF_ERR_WORKSPACE


def test_binding_refuses(binding):
    b = binding
    z = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        b.df_self_attn_fwd(z, z, z)
    for kw in (dict(window=-1), dict(sinks=2 ** 31)):
        with pytest.raises(ValueError, match="out of range"):
            b.df_self_attn_fwd(z, z, z, **kw)
