"""The embedding operators without a GPU: the oracle against torch's own
embedding and its gradient in float64, and the refusals of the C entry points
and of the binding (every call here returns before its first CUDA call)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def binding():
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding as b
    return b


@pytest.mark.parametrize("pad", [None, 0, 4])
def test_oracle_matches_autograd(pad):
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, 7, (3, 11), generator=g)
    table = torch.randn(7, 8, generator=g, dtype=torch.float64, requires_grad=True)
    dout = torch.randn(3, 11, 8, generator=g, dtype=torch.float64)
    out = torch.nn.functional.embedding(ids, table, padding_idx=pad) * 2.5
    out.backward(dout)
    assert np.allclose(oracle.embed(ids.numpy(), table.detach().numpy(), 2.5), out.detach().numpy(), atol=1e-12)
    grad, mass, count = oracle.embed_grad(ids.numpy(), dout.numpy(), 7, 2.5, pad)
    assert np.allclose(grad, table.grad.numpy(), atol=1e-12)
    assert (mass >= np.abs(grad) - 1e-12).all()
    assert count.sum() == (ids.numel() if pad is None else int((ids != pad).sum()))


def test_oracle_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(2)
    ids, table, dout = rng.integers(0, 5, 9), rng.standard_normal((5, 8)), rng.standard_normal((9, 8))
    grad, _, _ = oracle.embed_grad(ids, dout, 5, 0.75)
    for v in range(5):
        for c in range(8):
            e = np.zeros_like(table)
            e[v, c] = 1e-3
            up, down = (np.sum(oracle.embed(ids, table + s * e, 0.75) * dout) for s in (1, -1))
            assert abs((up - down) / 2e-3 - grad[v, c]) < 1e-9


def _lookup(b, **over):
    a = dict(ids=0x1000, ids64=0, T=4, table=0x2000, V=10, N=64, out=0x3000, dtype=0)
    a.update(over)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return b.raw_library.df_embedding(vp(a["ids"]), a["ids64"], a["T"], vp(a["table"]), a["V"], a["N"], 1.0,
                                      vp(a["out"]), a["dtype"], None, None)


def _grad(b, **over):
    a = dict(ids=0x1000, ids64=0, T=4, dout=0x2000, V=10, N=64, pad=-1, acc=0, grad=0x3000, dtype=0, ws=0x10000,
             bytes=1 << 30)
    a.update(over)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return b.raw_library.df_embedding_bwd(vp(a["ids"]), a["ids64"], a["T"], vp(a["dout"]), a["V"], a["N"], 1.0,
                                          a["pad"], a["acc"], vp(a["grad"]), a["dtype"], None, vp(a["ws"]),
                                          a["bytes"], None)


def test_entry_points_refuse_on_the_host(binding):
    b = binding
    for call in (_lookup, _grad):
        for bad in (dict(T=-1), dict(T=(1 << 30) + 1), dict(V=0), dict(N=0), dict(dtype=3), dict(ids=None)):
            assert call(b, **bad) == b.DF_ERR_INVALID_ARG, (call.__name__, bad)
        assert call(b, N=60) == b.DF_ERR_UNSUPPORTED
        assert call(b, N=65544) == b.DF_ERR_UNSUPPORTED
        assert call(b, ids=0x1002) == b.DF_ERR_ALIGNMENT
        assert call(b, ids=0x1004, ids64=1) == b.DF_ERR_ALIGNMENT
    assert _lookup(b, table=None) == b.DF_ERR_INVALID_ARG
    assert _lookup(b, table=0x2008) == b.DF_ERR_ALIGNMENT
    assert _lookup(b, out=0x3004) == b.DF_ERR_ALIGNMENT
    assert _lookup(b, T=0, ids=None) == b.DF_OK
    assert _grad(b, dout=None) == b.DF_ERR_INVALID_ARG
    assert _grad(b, grad=None) == b.DF_ERR_INVALID_ARG
    assert _grad(b, pad=10) == b.DF_ERR_INVALID_ARG
    assert _grad(b, pad=-2) == b.DF_ERR_INVALID_ARG
    assert _grad(b, dout=0x2008) == b.DF_ERR_ALIGNMENT
    assert _grad(b, grad=0x3008) == b.DF_ERR_ALIGNMENT
    assert _grad(b, ws=0x10010) == b.DF_ERR_ALIGNMENT
    assert _grad(b, ws=None) == b.DF_ERR_WORKSPACE
    need = b.df_embedding_bwd_workspace_size(4, 64, 10)
    assert need >= 256 and _grad(b, bytes=need - 1) == b.DF_ERR_WORKSPACE
    assert b.df_embedding_bwd_workspace_size(4, 60, 10) == 0
    assert b.df_embedding_bwd_workspace_size(0, 64, 10) >= 256


def test_binding_refuses(binding):
    ids = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros(10, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.df_embedding(ids, table)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.df_embedding_bwd(ids, torch.zeros(4, 64), 10)
    with pytest.raises(ValueError, match="matrix"):
        binding.df_embedding(ids, torch.zeros(10, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="dout"):
        binding.df_embedding_bwd(ids, torch.zeros(5, 64), 10)
