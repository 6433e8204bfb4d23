"""GPU parity of the cross-attention gradients against the float64 oracle on the
same rounded inputs, within bounds counted in roundings (tests/_cross.py)."""

import numpy as np
import pytest
import torch

import oracle
from _cross import call, call_bwd, check_backward, inputs, np64, to_dev, want

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

CASES = [  # B, H, Hk, d, Lq, Lk, dtype, q, k
    (1, 1, 1, 64, 1, 1, BF, "padded", "full"),
    (2, 2, 2, 64, 5, 2, HF, "padded", "full"),
    (2, 2, 2, 64, 64, 128, BF, "padded", "full"),
    (2, 3, 3, 64, 128, 129, HF, "padded", "full"),
    (3, 4, 4, 64, 130, 300, BF, "padded", "masked"),
    (5, 4, 2, 64, 257, 513, BF, "packed", "packed"),
    (2, 2, 1, 128, 100, 700, BF, "padded", "full"),
    (4, 6, 2, 128, 70, 390, HF, "packed", "masked"),
    (3, 8, 1, 128, 300, 260, BF, "padded", "packed"),
    (40, 2, 2, 64, 9, 200, BF, "packed", "packed"),
    (2, 2, 2, 32, 65, 333, BF, "padded", "masked"),
    (2, 3, 1, 96, 177, 150, HF, "packed", "packed"),
    (2, 2, 2, 8, 33, 140, BF, "padded", "full"),
    (1, 128, 1, 64, 3, 200, BF, "padded", "full"),
    (2, 65, 1, 72, 3, 150, HF, "packed", "full"),
    (70, 4, 4, 64, 1, 260, BF, "padded", "packed"),
    (9, 12, 12, 64, 300, 200, BF, "padded", "masked"),
    (60, 4, 2, 128, 150, 140, BF, "packed", "packed"),
]


def _step(lib, x, dev, scale=None, **more):
    out, stats = call(lib, x, dev, scale=scale, with_stats=True)
    return call_bwd(lib, x, dev, out, stats, scale=scale, **more)


@pytest.mark.parametrize("B,H,Hk,d,Lq,Lk,dtype,q,k", CASES)
def test_backward_matches_oracle(lib, B, H, Hk, d, Lq, Lk, dtype, q, k):
    x = inputs(B, H, Hk, d, Lq, Lk, dtype, q, k, seed=B + H + Lq + Lk)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((lib.df_cross_attn_bwd_workspace_size(x["q"].numel() // (H * d), H),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    nan = tuple(torch.full_like(dev[n], float("nan")) for n in ("q", "k", "v"))
    got = _step(lib, x, dev, grads=nan, workspace=ws, status=status)
    check_backward(got, want(oracle, x, d ** -0.5, with_grad=True), dtype, d)
    assert int(status.item()) == lib.DF_OK
    for a, b in zip(got, _step(lib, x, dev)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sigma,scale,size", [(4.0, None, 1.0), (1.0, 1e-3, 1.0), (1.0, None, 2.0 ** -14),
                                              (1.0, None, 1024.0)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_large_scores_and_small_gradients(lib, sigma, scale, size, dtype):
    # fp16 gradients of 2^-14 times unit inputs come back as fp16 subnormals: the
    # result's own rounding bounds them, not that of dS on the way
    x = inputs(2, 4, 2, 64, 90, 400, dtype, "padded", "masked", seed=5, sigma=sigma)
    x["dout"] = (x["dout"].float() * size / sigma).to(dtype)
    got = _step(lib, x, to_dev(x), scale=scale)
    s = 64 ** -0.5 if scale is None else float(np.float32(scale))
    check_backward(got, want(oracle, x, s, with_grad=True), dtype, 64)


def test_gradient_is_the_difference_quotient(lib):
    # along a random direction of each input, against the float64 forward's central
    # difference (step 1e-4: its own error is below 1e-6 of these sums)
    x = inputs(2, 4, 2, 64, 20, 150, HF, "padded", "full", seed=8)
    got = _step(lib, x, to_dev(x))
    g = np64(x["dout"])
    for name, grad in zip(("q", "k", "v"), got):
        direction = np.random.default_rng(1).standard_normal(x[name].shape)
        ends = []
        for sign in (1, -1):
            moved = {**x, name: x[name].double() + sign * 1e-4 * torch.from_numpy(direction)}
            ends.append((want(oracle, moved, 0.125)["out"] * g).sum())
        quotient, grad = (ends[0] - ends[1]) / 2e-4, np64(grad)
        # three independent roundings of the gradient (check_backward), projected
        norm = lambda z: float(np.sqrt((z ** 2).sum()))  # noqa: E731
        bound = 3 * torch.finfo(HF).eps / 2 * norm(grad) * norm(direction)
        assert abs(float((grad * direction).sum()) - quotient) <= bound, name


@pytest.mark.parametrize("d,G", [(64, 1), (128, 3)])
def test_masked_and_foreign_rows_may_hold_anything(lib, d, G):
    x = inputs(3, 2 * G, 2, d, 90, 300, BF, "padded", "masked", seed=d, nk=[300, 0, 131])
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    clean = call_bwd(lib, x, dev, out, stats)
    off = dev["key_mask"] == 0
    for junk in (float("nan"), float("inf"), torch.finfo(BF).min):
        for n in ("k", "v"):
            dev[n] = dev[n].clone()
            dev[n][off] = junk
        for a, b in zip(call_bwd(lib, x, dev, out, stats), clean):
            assert torch.equal(a, b)
    assert all(int((t[off] != 0).sum()) == 0 for t in clean[1:]) and int((clean[0][1] != 0).sum()) == 0
    x = inputs(3, 2 * G, 2, d, 90, 300, BF, "packed", "packed", seed=d, nq=[90, 50, 70], nk=[153, 5, 300])
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    clean = call_bwd(lib, x, dev, out, stats)
    for n, rows in (("q", slice(90, 140)), ("dout", slice(90, 140)), ("k", slice(153, 158)), ("v", slice(153, 158))):
        dev[n] = dev[n].clone()
        dev[n][rows] = float("nan")
    dirty = call_bwd(lib, x, dev, out, stats)
    for a, b, rows in zip(dirty, clean, ((90, 140), (153, 158), (153, 158))):
        assert torch.equal(a[:rows[0]], b[:rows[0]]) and torch.equal(a[rows[1]:], b[rows[1]:])


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_behind_the_last_sequence_and_empty_sequences(lib, dtype):
    x = inputs(5, 4, 2, 64, 200, 200, dtype, "packed", "packed", seed=3, nq=[0, 150, 0, 200, 7], nk=[9, 0, 30, 200, 1])
    w = want(oracle, x, 0.125, with_grad=True)
    Tq, Tk = 357, 240
    for n in ("q", "k", "v", "dout"):
        x[n] = torch.cat([x[n], torch.full((300,) + tuple(x[n].shape[1:]), float("nan"), dtype=dtype)])
    x["dout"][Tq + 20:] = 60000.0
    dq, dk, dv = _step(lib, x, to_dev(x))
    for t, T in ((dq, Tq), (dk, Tk), (dv, Tk)):
        assert int((t[T:] != 0).sum()) == 0
    check_backward((dq[:Tq], dk[:Tk], dv[:Tk]), w, dtype, 64)


@pytest.mark.parametrize("d", [64, 128])
def test_key_tiles_without_a_valid_key(lib, d):
    # masks with holes that span whole tiles of 128 keys, at either end and inside
    x = inputs(3, 4, 2, d, 140, 700, BF, "padded", "masked", seed=d + 1, nk=[700, 300, 700])
    x["key_mask"][0, 120:400] = 0
    x["key_mask"][2, :600] = 0
    got = _step(lib, x, to_dev(x))
    check_backward(got, want(oracle, x, d ** -0.5, with_grad=True), BF, d)


def test_large_gradient_of_a_row_without_keys(lib):
    # it does not set the scale that the other rows' small gradients are held at: dS of
    # 2^-12 dout next to 2^15 would be below fp16's subnormals
    x = inputs(2, 2, 2, 64, 70, 200, HF, "padded", "masked", seed=3, nk=[200, 0])
    x["dout"][0] = (x["dout"][0].float() * 2.0 ** -12).to(HF)
    x["dout"][1] = 2.0 ** 15
    w = want(oracle, x, 0.125, with_grad=True)
    check_backward(_step(lib, x, to_dev(x)), w, HF, 64)


def test_two_calls_at_once(lib):
    xs = [inputs(12, 4, 2, 128, 150, 300, HF, "packed", "packed", seed=s) for s in (1, 2)]
    devs = [to_dev(x) for x in xs]
    fwd = [call(lib, x, dev, with_stats=True) for x, dev in zip(xs, devs)]
    alone = [call_bwd(lib, x, dev, *f) for x, dev, f in zip(xs, devs, fwd)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call_bwd(lib, xs[i], devs[i], *fwd[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for grads in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(grads, alone[i]))


def test_no_keys_no_queries(lib):
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    for Lq, Lk, B in ((3, 0, 2), (0, 9, 2), (0, 0, 2), (3, 9, 0)):
        q, k = z(B, Lq, 4, 64), z(B, Lk, 4, 64)
        out, stats = lib.df_cross_attn_fwd(q, k, k, with_stats=True)
        nan = tuple(torch.full_like(t, float("nan")) for t in (q, k, k))
        got = lib.df_cross_attn_bwd(q, k, k, out, stats, q, grads=nan)
        assert all(int((t != 0).sum()) == 0 for t in got)


def test_other_stream_and_captured_replay(lib):
    x = inputs(3, 4, 2, 64, 50, 400, HF, "padded", "masked", seed=4)
    dev = to_dev(x)
    side = torch.cuda.Stream()
    out, stats = call(lib, x, dev, with_stats=True)
    grads = tuple(torch.empty_like(dev[n]) for n in ("q", "k", "v"))
    ws = torch.empty(lib.df_cross_attn_bwd_workspace_size(150, 4), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o2, s2 = call(lib, x, dev, with_stats=True)
        call_bwd(lib, x, dev, o2, s2, grads=grads, workspace=ws)
    y = inputs(3, 4, 2, 64, 50, 400, HF, "padded", "masked", seed=6)
    y["dout"] *= 0.01
    for n in ("q", "k", "v", "key_mask", "dout"):
        dev[n].copy_(y[n])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_backward(grads, want(oracle, y, 0.125, with_grad=True), HF, 64)
    with torch.cuda.stream(side):
        again = _step(lib, x, dev)
    side.synchronize()
    for a, b in zip(again, grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128])
def test_wait_budget_runs_out_and_recovers(lib, d):
    x = inputs(2, 2, 2, d, 700, 900, BF, seed=9)
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.df_attn_set_wait_budget(1)
    try:
        call_bwd(lib, x, dev, out, stats, status=status)
        torch.cuda.synchronize()
    finally:
        lib.df_attn_set_wait_budget(0)
    assert int(status.item()) == lib.DF_ERR_DEVICE_TIMEOUT
    check_backward(call_bwd(lib, x, dev, out, stats), want(oracle, x, d ** -0.5, with_grad=True), BF, d)


def test_refusals(lib):
    x = inputs(2, 4, 2, 64, 3, 9, BF, seed=1)
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    with pytest.raises(ValueError, match="dout"):
        lib.df_cross_attn_bwd(dev["q"], dev["k"], dev["v"], out, stats, dev["dout"].half())
    with pytest.raises(ValueError, match="lse"):
        lib.df_cross_attn_bwd(dev["q"], dev["k"], dev["v"], out, lib.CrossStats(stats.lse[:1], stats.out_lo), dev["dout"])
    with pytest.raises(lib.DFError):
        call_bwd(lib, x, dev, out, stats, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lib.DFError):
        call_bwd(lib, x, dev, out, stats, scale=-1.0)
    # without out_lo the call still runs
    got = lib.df_cross_attn_bwd(dev["q"], dev["k"], dev["v"], out, lib.CrossStats(stats.lse, None), dev["dout"])
    assert all(bool(torch.isfinite(t).all()) for t in got)
