"""GPU parity of causal attention with a window and sinks, forward and backward, against the
float64 oracle on the same rounded inputs, within bounds counted in roundings."""

import numpy as np
import pytest
import torch

import oracle
from _causal import call, call_bwd, want
from _cross import check_backward, check_forward, inputs, np64, to_dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

CASES = [  # B, H, Hk, d, Lq, Lk, dtype, q, k, window, sinks
    (1, 1, 1, 64, 1, 1, BF, "padded", "full", 0, 0),
    (2, 2, 2, 64, 130, 130, HF, "padded", "full", 0, 0),
    (2, 2, 1, 128, 257, 257, BF, "padded", "full", 0, 0),
    (2, 2, 2, 64, 700, 700, BF, "padded", "full", 1, 0),
    (1, 2, 2, 64, 900, 900, HF, "padded", "full", 130, 3),
    (2, 3, 1, 128, 600, 600, BF, "padded", "masked", 100, 1),
    (1, 4, 2, 96, 513, 513, HF, "padded", "masked", 128, 200),
    (1, 2, 2, 32, 400, 1000, BF, "padded", "full", 129, 127),
    (2, 6, 2, 128, 70, 640, HF, "padded", "masked", 200, 128),
    (3, 4, 4, 64, 1, 900, BF, "padded", "full", 300, 4),
    (2, 2, 2, 64, 300, 100, BF, "padded", "full", 0, 0),      # rows before the first key
    (2, 2, 1, 128, 300, 100, HF, "padded", "full", 20, 2),
    (5, 4, 2, 64, 400, 513, BF, "packed", "packed", 0, 0),    # any two lengths
    (5, 4, 1, 128, 300, 400, HF, "packed", "packed", 64, 5),
    (4, 2, 2, 64, 260, 300, HF, "packed", "masked", 77, 2),
    (3, 5, 1, 72, 200, 300, BF, "packed", "full", 90, 0),
    (1, 128, 1, 64, 40, 200, BF, "padded", "full", 50, 9),    # one token a tile
    (2, 65, 1, 64, 9, 300, HF, "padded", "full", 33, 0),
    (1, 1, 1, 64, 1500, 1500, BF, "padded", "full", 2 ** 31 - 1, 7),
    (40, 2, 2, 64, 60, 60, BF, "packed", "packed", 16, 1),
    (2, 2, 2, 64, 300, 2500, BF, "padded", "full", 0, 0),     # clusters share a tile
    (1, 2, 1, 128, 60, 3000, HF, "padded", "full", 1100, 300),
]


@pytest.mark.parametrize("B,H,Hk,d,Lq,Lk,dtype,q,k,window,sinks", CASES)
def test_matches_oracle(lib, B, H, Hk, d, Lq, Lk, dtype, q, k, window, sinks):
    x = inputs(B, H, Hk, d, Lq, Lk, dtype, q, k, seed=B + H + Lq + Lk + window % 1000)
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
    again = call_bwd(lib, x, dev, got, stats, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    assert int(status.item()) == lib.DF_OK


@pytest.mark.parametrize("dtype,d", [(BF, 64), (HF, 128)])
def test_a_window_over_everything_is_no_window(lib, dtype, d):
    x = inputs(2, 4, 2, d, 333, 333, dtype, "padded", "full", seed=3)
    dev = to_dev(x)
    a, sa = call(lib, x, dev, with_stats=True)
    b, sb = call(lib, x, dev, with_stats=True, window=333, sinks=9)
    assert torch.equal(a, b) and torch.equal(sa.lse, sb.lse)
    for s, t in zip(call_bwd(lib, x, dev, a, sa), call_bwd(lib, x, dev, b, sb, window=333, sinks=9)):
        assert torch.equal(s, t)


def test_chunks_of_a_prompt_give_the_whole(lib):
    x = inputs(2, 4, 2, 64, 500, 500, BF, "padded", "full", seed=8)
    dev = to_dev(x)
    whole = call(lib, x, dev, window=140, sinks=3)
    w = want(oracle, x, 64 ** -0.5, 140, 3)
    parts, at = [], 0
    for n in (1, 127, 130, 242):
        c = {**x, "Lq": n, "Lk": at + n}
        cd = {**dev, "q": dev["q"][:, at:at + n].contiguous(), "k": dev["k"][:, :at + n].contiguous(),
              "v": dev["v"][:, :at + n].contiguous()}
        parts.append(call(lib, c, cd, window=140, sinks=3))
        at += n
    check_forward(torch.cat(parts, dim=1), w, BF, 64)
    check_forward(whole, w, BF, 64)


def test_gradients_are_difference_quotients(lib):
    """Directional differences of the kernel's own forward, in fp16 with out + out_lo (both
    carry the result to 2^-22 of it)."""
    x = inputs(1, 2, 1, 64, 200, 200, HF, "padded", "full", seed=4)
    dev = to_dev(x)
    kw = dict(window=60, sinks=2)
    out, stats = call(lib, x, dev, with_stats=True, **kw)
    grads = call_bwd(lib, x, dev, out, stats, **kw)
    w = want(oracle, x, 64 ** -0.5, 60, 2, with_grad=True)
    g = torch.Generator().manual_seed(1)
    for n, grad in zip(("q", "k", "v"), grads):
        step = torch.randn(x[n].shape, generator=g)
        ends = [(x[n].float() + s * 0.25 * step).to(HF) for s in (1, -1)]
        diff, total = [], 0.0
        for e in ends:
            o, s = call(lib, x, {**dev, n: e.cuda()}, with_stats=True, **kw)
            diff.append(((np64(o) + np64(s.out_lo)) * np64(x["dout"])).sum())
        move = np64(ends[0]) - np64(ends[1])
        # the oracle's own difference over the same step stands for the curvature
        ref = [(want(oracle, {**x, n: e}, 64 ** -0.5, 60, 2)["out"] * np64(x["dout"])).sum() for e in ends]
        total = (np64(grad) * move).sum()
        curve = abs((ref[0] - ref[1]) - (w["d" + n] * move).sum())
        # each of the forward's weights, and the gradient's three roundings, are off by half a
        # step, of either sign: their sum over the entries by its root mean square, six times
        half = 2.0 ** -11
        noise = 6 * half * (np.sqrt((w["out_mass"] ** 2 * np64(x["dout"]) ** 2).sum()) * 2 +
                            3 * np.sqrt((w["d" + n + "_mass"] ** 2 * move ** 2).sum()))
        assert abs((diff[0] - diff[1]) - total) <= curve + noise, (n, diff[0] - diff[1], total, curve, noise)


@pytest.mark.parametrize("d", [64, 128])
def test_later_sequences_and_masked_keys_may_hold_anything(lib, d):
    x = inputs(3, 4, 2, d, 200, 200, BF, "packed", "packed", seed=d, nq=[150, 7, 190], nk=[150, 30, 190])
    dev = to_dev(x)
    kw = dict(window=60, sinks=2)
    clean, stats = call(lib, x, dev, with_stats=True, **kw)
    grads = call_bwd(lib, x, dev, clean, stats, **kw)
    rows = slice(int(x["cu_k"][1]), int(x["cu_k"][2]))
    for junk in (float("nan"), float("inf")):
        bad = {**dev, "k": dev["k"].clone(), "v": dev["v"].clone(), "dout": dev["dout"].clone()}
        bad["k"][rows] = junk
        bad["v"][rows] = junk
        got = call(lib, x, bad, **kw)
        assert torch.equal(got[:150], clean[:150]) and torch.equal(got[157:], clean[157:])
        for name, s, t in zip("qkv", call_bwd(lib, x, bad, clean, stats, **kw), grads):
            n = 157 if name == "q" else 180
            assert torch.equal(s[:150], t[:150]) and torch.equal(s[n:], t[n:]), name
    x = inputs(2, 4, 2, d, 300, 300, HF, "padded", "masked", seed=d, nk=[300, 120])
    dev = to_dev(x)
    clean = call(lib, x, dev, **kw)
    off = dev["key_mask"] == 0
    for n in ("k", "v"):
        dev[n][off] = float("nan")
    assert torch.equal(call(lib, x, dev, **kw), clean)
    assert int((clean[1, 122 + 60:] != 0).any(dim=-1).sum()) > 0  # sinks are seen at any distance


def test_packed_rows_behind_the_last_sequence_are_zeros(lib):
    x = inputs(2, 2, 2, 64, 90, 120, BF, "packed", "packed", seed=5, nq=[60, 50], nk=[120, 50])
    dev = to_dev(x)
    pad = lambda t: torch.cat((t, torch.full_like(t[:9], float("nan"))))  # noqa: E731
    big = {**dev, **{n: pad(dev[n]) for n in ("q", "k", "v", "dout")}}
    out, stats = call(lib, x, big, with_stats=True, window=30)
    assert int((out[110:] != 0).sum()) == 0 and bool((stats.lse[110:] == -np.inf).all())
    small, ss = call(lib, x, dev, with_stats=True, window=30)
    assert torch.equal(out[:110], small)
    for s, t, n in zip(call_bwd(lib, x, big, out, stats, window=30), call_bwd(lib, x, dev, small, ss, window=30),
                       (110, 170, 170)):
        assert torch.equal(s[:n], t) and int((s[n:] != 0).sum()) == 0


def test_bad_offsets_are_reported(lib):
    x = inputs(2, 2, 2, 64, 90, 120, BF, "packed", "packed", seed=5, nq=[60, 50], nk=[120, 50])
    dev = to_dev(x)
    dev["cu_k"] = torch.tensor([0, 120, 171], dtype=torch.int32, device="cuda")  # behind the rows
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = call(lib, x, dev, window=30, status=status)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG
    assert int((out[60:] != 0).sum()) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_captured_and_replayed_with_new_inputs(lib, dtype):
    x = inputs(2, 4, 2, 64, 260, 260, dtype, "padded", "full", seed=11)
    y = inputs(2, 4, 2, 64, 260, 260, dtype, "padded", "full", seed=12)
    dev, other = to_dev(x), to_dev(y)
    kw = dict(window=100, sinks=1)
    ws = torch.empty(lib.df_cross_attn_bwd_workspace_size(520, 4), dtype=torch.uint8, device="cuda")

    def step():
        out, stats = call(lib, x, dev, with_stats=True, **kw)
        return (out,) + tuple(call_bwd(lib, x, dev, out, stats, workspace=ws, **kw))

    first = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for n in ("q", "k", "v", "dout"):
        dev[n].copy_(other[n])
    graph.replay()
    eager = step()
    assert all(torch.equal(a, b) for a, b in zip(held, eager))
    assert not torch.equal(held[0], first[0])
