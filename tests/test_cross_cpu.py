"""Cross attention without a GPU: the oracle against torch's own attention in
float64 and its gradients, against differences of its own forward, and the host
refusals of the entry points."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from _cross import inputs, np64, want


@pytest.fixture(scope="module")
def binding():
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding as b
    return b


@pytest.mark.parametrize("G", [1, 3])
def test_oracle_matches_autograd(G):
    x = inputs(3, 2 * G, 2, 16, 7, 11, torch.float64, "padded", "masked", seed=1, nk=[11, 4, 6])
    q, k, v = (x[n].clone().requires_grad_(True) for n in ("q", "k", "v"))
    kk, vv = (t.repeat_interleave(G, dim=2).transpose(1, 2) for t in (k, v))
    mask = (x["key_mask"] != 0)[:, None, None, :]
    out = torch.nn.functional.scaled_dot_product_attention(q.transpose(1, 2), kk, vv, attn_mask=mask,
                                                           scale=0.3).transpose(1, 2)
    out.backward(x["dout"])
    w = want(oracle, x, 0.3, with_grad=True)
    for name, t in (("out", out.detach()), ("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
        assert np.allclose(w[name], t.numpy(), atol=1e-11), name


def test_oracle_gradients_are_difference_quotients():
    x = inputs(2, 4, 2, 8, 3, 5, torch.float64, "packed", "packed", seed=2, nq=[2, 3], nk=[5, 3])
    w = want(oracle, x, 0.4, with_grad=True)
    g = np64(x["dout"])
    for name in ("q", "k", "v"):
        flat = x[name].view(-1)
        for i in range(0, flat.numel(), 7):
            keep, got = float(flat[i]), []
            for s in (1e-4, -1e-4):
                flat[i] = keep + s
                got.append((want(oracle, x, 0.4)["out"] * g).sum())
            flat[i] = keep
            assert abs((got[0] - got[1]) / 2e-4 - w["d" + name].reshape(-1)[i]) < 1e-6


def test_oracle_rows_without_keys():
    x = inputs(3, 2, 1, 8, 4, 6, torch.float64, "packed", "masked", seed=3, nq=[4, 0, 3], nk=[6, 6, 0])
    w = want(oracle, x, 1.0, with_grad=True)
    assert (w["out"][4:] == 0).all() and np.isinf(w["lse"][4:]).all() and (w["dq"][4:] == 0).all()
    assert (w["dk"][1:] == 0).all() and (w["dv"][1:] == 0).all()


def _fwd(b, **over):
    a = dict(q=0x10000, k=0x20000, v=0x30000, mask=None, cu_q=None, cu_k=None, B=2, H=4, Hk=2, Lq=3, Lk=9, Tq=6, Tk=18,
             d=64, scale=0.125, dtype=0, out=0x40000, lo=None, lse=None)
    a.update(over)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return b.raw_library.df_cross_attn_fwd(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["mask"]), vp(a["cu_q"]), vp(a["cu_k"]), a["B"], a["H"], a["Hk"],
        a["Lq"], a["Lk"], a["Tq"], a["Tk"], a["d"], a["scale"], a["dtype"], vp(a["out"]), vp(a["lo"]), vp(a["lse"]),
        None, None)


def _bwd(b, **over):
    a = dict(q=0x10000, k=0x20000, v=0x30000, mask=None, cu_q=None, cu_k=None, B=2, H=4, Hk=2, Lq=3, Lk=9, Tq=6, Tk=18,
             d=64, scale=0.125, dtype=0, out=0x40000, lo=None, lse=0x50000, dout=0x60000, dq=0x70000, dk=0x80000,
             dv=0x90000, ws=0xa0000, bytes=1 << 20)
    a.update(over)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return b.raw_library.df_cross_attn_bwd(
        vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["out"]), vp(a["lo"]), vp(a["lse"]), vp(a["dout"]), vp(a["mask"]),
        vp(a["cu_q"]), vp(a["cu_k"]), a["B"], a["H"], a["Hk"], a["Lq"], a["Lk"], a["Tq"], a["Tk"], a["d"], a["scale"],
        a["dtype"], vp(a["dq"]), vp(a["dk"]), vp(a["dv"]), None, vp(a["ws"]), a["bytes"], None)


REFUSED = [  # arguments, status
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(B=-1), 1), (dict(H=0), 1), (dict(Hk=0), 1),
    (dict(H=3), 1), (dict(Lq=-1), 1), (dict(Lk=-1), 1), (dict(Tq=7), 1), (dict(Tk=17), 1), (dict(d=0), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(dtype=3), 1), (dict(mask=0x50000, cu_k=0x60000), 1), (dict(dtype=2), 2), (dict(d=60), 2), (dict(d=136), 2),
    (dict(H=258, Hk=2), 2), (dict(q=0x10008), 3), (dict(k=0x20004), 3), (dict(v=0x30008), 3), (dict(cu_q=0x60002), 3)]


@pytest.mark.parametrize("over,status", REFUSED)
def test_entry_points_refuse_on_the_host(binding, over, status):
    assert _fwd(binding, **over) == status, over
    assert _bwd(binding, **over) == status, over


def test_forward_refuses_its_own_arguments(binding):
    b = binding
    assert _fwd(b, out=None) == b.DF_ERR_INVALID_ARG
    assert _fwd(b, out=0x40008) == b.DF_ERR_ALIGNMENT
    assert _fwd(b, lo=0x50008) == b.DF_ERR_ALIGNMENT
    assert _fwd(b, lse=0x50002) == b.DF_ERR_ALIGNMENT
    assert _fwd(b, Lq=0, Tq=0, q=None, out=None) == b.DF_OK  # nothing to do
    with pytest.raises(ValueError, match="CUDA tensor"):
        z = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
        b.df_cross_attn_fwd(z, z, z)


def test_backward_refuses_its_own_arguments(binding):
    b = binding
    for name in ("out", "lse", "dout", "dq", "dk", "dv"):
        assert _bwd(b, **{name: None}) == b.DF_ERR_INVALID_ARG, name
    for name in ("out", "lo", "dout", "dq", "dk", "dv"):
        assert _bwd(b, **{name: 0xb0008}) == b.DF_ERR_ALIGNMENT, name
    assert _bwd(b, lse=0x50002) == b.DF_ERR_ALIGNMENT
    assert _bwd(b, ws=0xa0080) == b.DF_ERR_ALIGNMENT
    need = b.df_cross_attn_bwd_workspace_size(6, 4)
    assert need >= 6 * 4 * 8
    assert _bwd(b, bytes=need - 1) == b.DF_ERR_WORKSPACE
    assert _bwd(b, ws=None) == b.DF_ERR_WORKSPACE
    assert b.df_cross_attn_bwd_workspace_size(-1, 4) == 0
    assert _bwd(b, Lq=0, Lk=0, Tq=0, Tk=0) == b.DF_OK  # nothing to do
