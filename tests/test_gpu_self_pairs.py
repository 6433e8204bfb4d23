"""Causal attention where there is more work than a round of the SMs: items of two query tiles
that follow one another, against the float64 oracle; what one of the tiles
sees and the other does not, tiles without a partner, keys that are not numbers."""

import numpy as np
import pytest
import torch

import oracle
from _causal import call, call_bwd, want
from _cross import check_backward, check_forward, inputs, to_dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

CASES = [  # B, H, Hk, d, Lq, Lk, dtype, q, k, window, sinks
    (60, 6, 6, 64, 256, 256, BF, "padded", "full", 0, 0),       # two whole tiles
    (50, 6, 6, 64, 300, 300, HF, "padded", "full", 0, 0),       # a tile without a partner, and a part
    (40, 10, 10, 64, 130, 130, BF, "padded", "full", 1, 0),
    (30, 8, 8, 64, 520, 520, BF, "padded", "full", 64, 3),      # a window within a tile
    (30, 8, 8, 32, 520, 520, HF, "padded", "full", 128, 130),   # sinks of two tiles
    (24, 8, 8, 64, 700, 700, BF, "padded", "full", 257, 1),
    (40, 6, 2, 64, 200, 200, BF, "padded", "masked", 70, 2),    # 42 tokens a tile
    (30, 10, 2, 40, 150, 260, HF, "padded", "masked", 0, 0),    # the last part of longer keys
    (40, 12, 4, 64, 170, 90, BF, "padded", "full", 33, 1),      # rows before the first key
    (70, 8, 8, 64, 330, 330, BF, "packed", "packed", 0, 0),
    (70, 8, 4, 56, 330, 400, HF, "packed", "packed", 100, 5),
    (60, 8, 8, 64, 260, 300, HF, "packed", "masked", 77, 2),
    (2, 130, 2, 64, 90, 90, BF, "padded", "full", 40, 3),       # one token a tile, 65 heads
    (4, 128, 1, 64, 60, 60, HF, "packed", "packed", 0, 0),
    (50, 6, 6, 128, 256, 256, BF, "padded", "full", 0, 0),
    (40, 6, 6, 128, 300, 300, HF, "padded", "full", 0, 0),
    (24, 8, 8, 96, 520, 520, BF, "padded", "full", 64, 3),
    (24, 8, 8, 128, 520, 520, HF, "padded", "full", 128, 130),
    (20, 8, 8, 128, 700, 700, BF, "padded", "full", 257, 1),
    (30, 6, 2, 72, 200, 200, BF, "padded", "masked", 70, 2),
    (40, 12, 4, 128, 170, 90, HF, "padded", "full", 33, 1),
    (60, 8, 8, 128, 330, 330, BF, "packed", "packed", 0, 0),
    (60, 8, 4, 120, 330, 400, HF, "packed", "packed", 100, 5),
    (50, 8, 8, 128, 260, 300, BF, "packed", "masked", 77, 2),
    (2, 130, 2, 128, 90, 90, HF, "padded", "full", 40, 3),
    (90, 8, 8, 128, 140, 140, BF, "packed", "packed", 1, 0),    # items of a tile or two
]


@pytest.mark.parametrize("B,H,Hk,d,Lq,Lk,dtype,q,k,window,sinks", CASES)
def test_matches_oracle(lib, B, H, Hk, d, Lq, Lk, dtype, q, k, window, sinks):
    x = inputs(B, H, Hk, d, Lq, Lk, dtype, q, k, seed=B + H + Lq + Lk + window)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks, status=status)
    out = torch.full_like(dev["q"], float("nan"))
    got, stats = call(lib, x, dev, out=out, with_stats=True, **kw)
    w = want(oracle, x, d ** -0.5, window, sinks, with_grad=True)
    check_forward(got, w, dtype, d, stats.lse, stats.out_lo)
    assert torch.equal(call(lib, x, dev, **kw), got)
    grads = [torch.full_like(dev[n], float("nan")) for n in ("q", "k", "v")]
    call_bwd(lib, x, dev, got, stats, grads=grads, **kw)
    check_backward(grads, w, dtype, d)
    assert int(status.item()) == lib.DF_OK


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_a_cta(lib, d):
    """Every CTA takes many items of unequal length, one after another."""
    n = [int(i) for i in np.random.default_rng(0).integers(0, 700, 220)]
    x = inputs(220, 12, 12, d, 700, 700, BF, "packed", "packed", seed=3, nq=n, nk=n)
    dev = to_dev(x)
    got, stats = call(lib, x, dev, with_stats=True, window=150, sinks=2)
    at = np.concatenate([[0], np.cumsum(n)])
    for b in (0, 57, 110, 219):
        rows = slice(int(at[b]), int(at[b + 1]))
        part = {name: x[name][rows] for name in ("q", "k", "v", "dout")}
        cu = torch.tensor([0, n[b]], dtype=torch.int32)
        w = want(oracle, dict(part, key_mask=None, cu_q=cu, cu_k=cu), d ** -0.5, 150, 2)
        check_forward(got[rows], w, BF, d, stats.lse[rows], stats.out_lo[rows])
    for _ in range(3):
        assert torch.equal(call(lib, x, dev, window=150, sinks=2), got)


@pytest.mark.parametrize("d", [64, 128])
def test_keys_that_are_not_numbers(lib, d):
    """Masked ones stay out; one that counts makes its rows, and no other sequence's, NaN."""
    B, L = 60, 256
    n = [int(i) for i in np.random.default_rng(1).integers(3, L + 1, B)]
    n[0] = 200
    x = inputs(B, 6, 6, d, L, L, BF, "padded", "masked", seed=4, nk=n)
    x["key_mask"][0, :200] = 1
    dev = to_dev(x)
    clean = call(lib, x, dev, window=100, sinks=2)
    off = dev["key_mask"] == 0
    for junk in (float("nan"), float("inf"), -float("inf")):
        for name in ("k", "v"):
            dev[name][off] = junk
        assert torch.equal(call(lib, x, dev, window=100, sinks=2), clean)
    dev["k"][0, 140, 3] = float("nan")  # seen by rows 140 .. 239
    got = call(lib, x, dev, window=100, sinks=2)
    assert torch.equal(got[1:], clean[1:])
    assert bool(torch.isnan(got[0, 140:240, 3]).all())
    keep = torch.ones(L, dtype=torch.bool)
    keep[140:240] = False
    assert torch.equal(got[0, keep.cuda()], clean[0, keep.cuda()])
    others = [h for h in range(6) if h != 3]
    assert torch.equal(got[0][:, others], clean[0][:, others])
    # without a mask, in both tiles of an item
    x = inputs(B, 6, 6, d, L, L, HF, "padded", "full", seed=5)
    dev = to_dev(x)
    clean = call(lib, x, dev, window=100, sinks=2)
    for at in (1, 60, 127, 128, 200):
        bad = {**dev, "k": dev["k"].clone()}
        bad["k"][2, at, 1] = float("nan")
        got = call(lib, x, bad, window=100, sinks=2)
        seen = torch.zeros(L, dtype=torch.bool)
        seen[at:(L if at < 2 else min(at + 100, L))] = True
        assert bool(torch.isnan(got[2, seen.cuda(), 1]).all())
        got[2, seen.cuda(), 1] = clean[2, seen.cuda(), 1]
        assert torch.equal(got, clean), at
