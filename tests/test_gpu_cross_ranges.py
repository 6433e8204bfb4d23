"""Cross-attention gradients of inputs that span a wide range: fp16 holds dS scaled by
powers of two, which have to suit every row and sequence, not the largest of the
batch (tests/_cross.py counts the roundings)."""

import pytest
import torch

import oracle
from _cross import call, call_bwd, check_backward, inputs, to_dev, want

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _step(lib, x):
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    return call_bwd(lib, x, dev, out, stats)


@pytest.mark.parametrize("d,G", [(64, 1), (128, 3), (32, 2)])
@pytest.mark.parametrize("dtype", [HF, BF])
def test_sequences_whose_gradients_differ_by_far(lib, d, G, dtype):
    x = inputs(3, 2 * G, 2, d, 40, 1500, dtype, "packed", "packed", seed=d, nq=[40, 33, 7], nk=[700, 1500, 1])
    for rows, e in ((slice(0, 40), 10), (slice(40, 73), -10), (slice(73, 80), 0)):
        x["dout"][rows] *= 2.0 ** e
    check_backward(_step(lib, x), want(oracle, x, d ** -0.5, with_grad=True), dtype, d)


@pytest.mark.parametrize("d,G", [(64, 1), (128, 3)])
@pytest.mark.parametrize("dtype", [HF, BF])
def test_rows_and_heads_whose_gradients_differ_by_far(lib, d, G, dtype):
    # within one sequence: the small rows' dq is as right as the large ones'
    x = inputs(2, 2 * G, 2, d, 150, 2000, dtype, "padded", "masked", seed=d, nk=[2000, 900])
    x["dout"][:, 0::3] *= 2.0 ** 9
    x["dout"][:, 1::3] *= 2.0 ** -11
    x["dout"][:, :, G:] *= 2.0 ** -3
    w = want(oracle, x, d ** -0.5, with_grad=True)
    got = _step(lib, x)
    check_backward(got, w, dtype, d)
    for part in (slice(0, None, 3), slice(1, None, 3), slice(2, None, 3)):  # each size by itself
        err = (got[0].double().cpu() - torch.from_numpy(w["dq"]))[:, part].norm()
        tiny = 2.0 ** -25 if dtype == HF else 0.0  # results below fp16's normal range
        n = w["dq"][:, part].size
        assert float(err) <= 3 * torch.finfo(dtype).eps / 2 * float(torch.from_numpy(w["dq"])[:, part].norm()) \
            + tiny * n ** 0.5


@pytest.mark.parametrize("size", [1e3, 3e4])
@pytest.mark.parametrize("d,k", [(64, "masked"), (128, "packed")])
def test_values_of_any_size(lib, size, d, k):
    # all of a sequence's, and a single one among ordinary ones
    x = inputs(3, 4, 2, d, 60, 300, HF, "padded", k, seed=7, nk=[300, 200, 150])
    v = x["v"].view(-1, 2, d)
    v[:250] = (v[:250].float() * (size / 4)).clamp(-size, size).to(HF)
    v[550] = size
    x["dout"] = (x["dout"].float() * 2.0 ** -10).to(HF)
    check_backward(_step(lib, x), want(oracle, x, d ** -0.5, with_grad=True), HF, d)


@pytest.mark.parametrize("d", [64, 128])
def test_keys_and_rows_that_do_not_count_set_no_scale(lib, d):
    x = inputs(3, 4, 2, d, 90, 300, HF, "padded", "masked", seed=d, nk=[300, 0, 131])
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    clean = call_bwd(lib, x, dev, out, stats)
    off = dev["key_mask"] == 0
    for junk in (float("nan"), float("inf"), 65504.0):
        for n in ("k", "v"):
            dev[n] = dev[n].clone()
            dev[n][off] = junk
        assert all(torch.equal(a, b) for a, b in zip(call_bwd(lib, x, dev, out, stats), clean))
    # packed: rows of another sequence, and behind the last one
    x = inputs(2, 4, 2, d, 90, 300, HF, "packed", "packed", seed=d, nq=[90, 50], nk=[153, 200])
    for n in ("q", "k", "v", "dout"):
        x[n] = torch.cat([x[n], torch.zeros((70,) + tuple(x[n].shape[1:]), dtype=HF)])
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    clean = call_bwd(lib, x, dev, out, stats)
    dev["v"][153:] = 65504.0
    dev["dout"][90:] = 65504.0
    dirty = call_bwd(lib, x, dev, out, stats)
    assert torch.equal(dirty[0][:90], clean[0][:90])
    assert all(torch.equal(a[:153], b[:153]) for a, b in zip(dirty[1:], clean[1:]))


def test_many_sequences_and_long_ones(lib):
    # the maxima are formed by several blocks per sequence, or one block per sequence
    for B, L, H in ((3000, 6, 2), (1, 40000, 1)):
        x = inputs(B, H, H, 16, 4, L, HF, "packed", "packed", seed=B, nq=[1 + b % 4 for b in range(B)],
                   nk=[L - b % min(L, 5) for b in range(B)])
        at = [int(c) for c in x["cu_q"]]
        for b in range(B):
            x["dout"][at[b]:at[b + 1]] *= 2.0 ** (8 - 8 * (b % 3))
        if B == 1:
            x["v"][-3] = 2000.0
        check_backward(_step(lib, x), want(oracle, x, 0.25, with_grad=True), HF, 16)


@pytest.mark.parametrize("size", [1e3, 3e4])
@pytest.mark.parametrize("d", [64, 128])
def test_large_values_of_a_few_keys(lib, size, d):
    # weights near 1/2, so that dS is about |dout| |v| / 4
    x = inputs(4, 4, 2, d, 60, 5, HF, "padded", "packed", seed=9, nk=[1, 2, 3, 5])
    x["v"] = (x["v"].float() * (size / 4)).clamp(-size, size).to(HF)
    x["dout"] = (x["dout"].float() * 2.0 ** -10).to(HF)
    check_backward(_step(lib, x), want(oracle, x, d ** -0.5, with_grad=True), HF, d)
