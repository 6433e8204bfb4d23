"""Weights far below the largest one: fp16 has to hold them on their way into the product
with v.  A few keys with values of 0 take nearly all of a row's weight (as the first
tokens of a text often do), and what comes out is the sum over all the others."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("orders", [14.0, 20.5, 25.5])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 12800])
def test_weights_far_below_the_largest_count(lib, rows, dtype, d, orders):
    # one query tile (a cluster divides the keys), and more than half the SMs have
    n = 8192
    q = torch.zeros(1, rows, 1, d, dtype=dtype)
    k, v = torch.zeros(1, n, 1, d, dtype=dtype), torch.full((1, n, 1, d), 16.0, dtype=dtype)
    q[..., 0] = 4.0
    k[0, ::512, 0, 0] = orders * np.log(2) / 4  # for every CTA and group of warps that takes part
    k[0, 128::512, 0, 0] = orders * np.log(2) / 4
    v[0, ::512], v[0, 128::512] = 0.0, 0.0
    out, stats = lib.df_cross_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=1.0, with_stats=True)
    s = 4.0 * k[0, :, 0, 0].double()
    w = torch.exp(s - s.max())
    want = float((w * v[0, :, 0, 0].double()).sum() / w.sum())
    lse = float(s.max() + w.sum().log())
    # Half a step for the weights (fp16: of 2^-32 of the largest weight, below 2^-21 of it) and
    # for the result; n additions in fp32; the score's rounding, |s| 2^-24, and exp2's 2^-22.
    half = torch.finfo(dtype).eps / 2
    weight = max(half, 2.0 ** (orders - 32) if dtype == torch.float16 else 0.0)
    fp32 = n * 2.0 ** -24 + 18 * 2.0 ** -23 + 2.0 ** -21
    low = 2.0 ** -25 if dtype == torch.float16 else 0.0
    err = lambda x: float((x.double() - want).abs().max())  # noqa: E731
    assert err(out) <= (half + weight + fp32) * want * 1.01 + low
    assert err(out.double() + stats.out_lo.double()) <= (weight + fp32) * want * 1.01 + 2 * low
    assert float((stats.lse.double() - lse).abs().max()) <= fp32 + 2.0 ** -20
