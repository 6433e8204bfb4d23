"""Packed rows whose offsets do not begin at 0, in the attention calls of a decoder: the results are
those of the rows alone, and the rows in front of the first sequence are left as they were."""

import pytest
import torch

from _cache import fill, offsets, tokens

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def behind(x, first, value):
    """x [rows, ..] behind `first` rows of `value`, on the GPU."""
    return torch.cat([torch.full((first, *x.shape[1:]), value, dtype=x.dtype, device="cuda"), x.cuda()])


@pytest.mark.parametrize("first_q,first_k", [(1, 1), (200, 200), (0, 131), (37, 0)])
@pytest.mark.parametrize("lens,H,Hk,d,dtype", [([300, 0, 129], 4, 2, 64, BF), ([90] * 40, 8, 4, 128, HF),
                                               ([130, 256], 3, 3, 96, BF), ([200] * 30, 6, 6, 64, HF)])
def test_causal_attention(lib, lens, H, Hk, d, dtype, first_q, first_k):
    g = torch.Generator().manual_seed(d + first_k)
    q, k, v, do = (torch.randn(sum(lens), h, d, generator=g).to(dtype) for h in (H, Hk, Hk, H))
    cu = offsets(lens).cuda()
    kw = dict(max_seqlen_q=max(lens), max_seqlen_k=max(lens), window=70, sinks=3)
    q0, k0, v0, do0 = (x.cuda() for x in (q, k, v, do))
    want, stats = lib.df_self_attn_fwd(q0, k0, v0, cu_seqlens_q=cu, cu_seqlens_k=cu, with_stats=True, **kw)
    grads = lib.df_self_attn_bwd(q0, k0, v0, want, stats, do0, cu_seqlens_q=cu, cu_seqlens_k=cu, **kw)
    nan, status = float("nan"), torch.zeros(1, dtype=torch.int32, device="cuda")
    q1, do1, k1, v1 = behind(q, first_q, nan), behind(do, first_q, nan), behind(k, first_k, nan), behind(v, first_k, nan)
    kw.update(cu_seqlens_q=cu + first_q, cu_seqlens_k=cu + first_k, status=status)
    out = torch.full_like(q1, 7.0)
    _, stats1 = lib.df_self_attn_fwd(q1, k1, v1, out=out, with_stats=True, **kw)
    assert torch.equal(out[first_q:], want) and bool((out[:first_q] == 7).all())
    assert torch.equal(stats1.lse[first_q:], stats.lse) and torch.equal(stats1.out_lo[first_q:], stats.out_lo)
    got = tuple(torch.full_like(x, 7.0) for x in (q1, k1, v1))
    lib.df_self_attn_bwd(q1, k1, v1, out, stats1, do1, grads=got, **kw)
    for x, ref, first in zip(got, grads, (first_q, first_k, first_k)):
        assert torch.equal(x[first:], ref) and bool((x[:first] == 7).all())
    assert int(status.item()) == lib.DF_OK


@pytest.mark.parametrize("first", [1, 16, 1000])
@pytest.mark.parametrize("H,Hk,d,n", [(4, 2, 64, [2, 0, 3]), (16, 2, 128, [4, 1, 4])])
def test_attention_to_the_cache(lib, first, H, Hk, d, n):
    calls = tokens([[50, 3, 130]], Hk, d, BF, seed=first)
    cache, table, held = fill(lib, calls, Hk, d, 16)
    q = torch.randn(sum(n), H, d, generator=torch.Generator().manual_seed(first)).to(BF)
    cu, kw = offsets(n).cuda(), dict(max_seqlen_q=max(n), window=40, sinks=2)
    want = lib.df_cache_attn(q.cuda(), cache, table, held, cu, **kw)
    q1, status = behind(q, first, float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q1, 7.0)
    lib.df_cache_attn(q1, cache, table, held, cu + first, out=out, status=status, **kw)
    assert torch.equal(out[first:], want) and bool((out[:first] == 7).all())
    assert int(status.item()) == lib.DF_OK
