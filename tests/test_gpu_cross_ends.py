"""The end of an item, where every softmax thread reads the sums of both of the
CTA's teams: many items of few key tiles, one after another on each SM, so that a
team's sums stand beside the other's of this item and of the one before."""

import pytest
import torch

import oracle
from _cross import call, check_forward, inputs, to_dev, want

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("d,dtype", [(64, BF), (64, HF), (128, BF), (128, HF), (32, BF), (96, HF)])
@pytest.mark.parametrize("nk", [(1, 129, 128, 257), (0, 140, 500, 12, 300)])
def test_items_of_few_tiles(lib, d, dtype, nk):
    B, H = 400, 2
    x = inputs(B, H, H, d, 5, max(nk), dtype, "packed", "packed", seed=d + len(nk), nq=[1 + b % 5 for b in range(B)],
               nk=[nk[b % len(nk)] for b in range(B)])
    # values of very different size from one item to the next: what is left of another
    # item's sums would be far outside the bounds
    at = [int(c) for c in x["cu_k"]]
    for b in range(B):
        x["v"][at[b]:at[b + 1]] *= 2.0 ** (b % 7 - 3)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first, stats = call(lib, x, dev, with_stats=True, status=status)
    check_forward(first, want(oracle, x, d ** -0.5), dtype, d, stats.lse, stats.out_lo)
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(50):
        other += (call(lib, x, dev, status=status) != first).sum()
    assert int(other.item()) == 0 and int(status.item()) == lib.DF_OK
