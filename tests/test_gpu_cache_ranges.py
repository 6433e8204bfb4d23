"""Queries and values at the ends of their types' ranges, attended to and read back."""

import numpy as np
import pytest
import torch

from _cache import fill, oracles, tokens
from _cross import check_forward, np64
from test_gpu_cache import want_attn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def attend(lib, calls, q, heads, d, **kw):
    """(out, lse, oracle) of padded queries q [B, Lq, H, d] after the calls."""
    cache, table, held = fill(lib, calls, heads, d, 32)
    lse = torch.zeros(q.shape[:-1], device="cuda")
    out = lib.df_cache_attn(q.cuda(), cache, table, held, lse=lse, **kw)
    lens = [int(n) for n in held.tolist()]
    w = want_attn(np64(q).reshape(-1, *q.shape[2:]), lens, [q.shape[1]] * len(lens), oracles(calls, heads, d), True,
                  kw.get("window", 0), 0, d ** -0.5)
    return out.view(-1, *q.shape[2:]), lse.view(-1, q.shape[2]), w


@pytest.mark.parametrize("B,H,Hk,d,Lq,longest,window", [(2, 4, 2, 64, 1, 200, 0), (1, 32, 8, 128, 1, 3000, 0),
                                                        (2, 16, 2, 96, 3, 150, 40)])
def test_values_far_beyond_fp16(lib, B, H, Hk, d, Lq, longest, window):
    """Sums of some 200 values around 1e34 and the 150 nearest: representable, as are their
    partial sums with weights of 1 at most."""
    lens = [longest, 77][:B]
    calls = [(n, k, (v.float() * 1e34).to(BF)) for n, k, v in tokens([lens], Hk, d, BF, seed=d)]
    q = torch.randn(B, Lq, H, d, generator=torch.Generator().manual_seed(d)).to(BF)
    out, lse, w = attend(lib, calls, q, Hk, d, window=window)
    check_forward(out, w, BF, d, lse)


def test_one_value_at_the_top_and_equal_ones(lib):
    d = 64
    one = torch.exp2(torch.arange(d) % 14 + 113.0).view(1, 1, d).to(BF)
    many = torch.full((4096, 1, d), 2.0 ** 113).to(BF)
    for v in (one, -one, many):
        calls = [([v.shape[0]], torch.zeros_like(v), v)]
        out, lse, w = attend(lib, calls, torch.ones(1, 1, 2, d, dtype=BF), 1, d)
        check_forward(out, w, BF, d, lse)
