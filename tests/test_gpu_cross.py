"""GPU parity of the cross-attention forward against the float64 oracle on the
same rounded inputs, within bounds counted in roundings (tests/_cross.py)."""

import numpy as np
import pytest
import torch

import oracle
from _cross import call, call_bwd, check_forward, inputs, np64, to_dev, want

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

CASES = [  # B, H, Hk, d, Lq, Lk, dtype, q, k
    (1, 1, 1, 64, 1, 1, BF, "padded", "full"),
    (2, 2, 2, 64, 5, 128, HF, "padded", "full"),
    (2, 3, 3, 64, 128, 129, BF, "padded", "full"),
    (3, 4, 4, 64, 130, 300, HF, "padded", "masked"),
    (5, 4, 2, 64, 257, 513, BF, "packed", "packed"),
    (2, 2, 1, 128, 100, 700, BF, "padded", "full"),
    (4, 6, 2, 128, 70, 390, HF, "packed", "masked"),
    (3, 8, 1, 128, 40, 260, BF, "padded", "packed"),
    (40, 2, 2, 64, 9, 200, BF, "packed", "packed"),
    (2, 2, 2, 32, 65, 333, BF, "padded", "masked"),
    (2, 3, 1, 96, 77, 150, HF, "packed", "packed"),
    (2, 2, 2, 8, 33, 140, BF, "padded", "full"),
    (1, 128, 1, 64, 3, 200, BF, "padded", "full"),
    (2, 65, 1, 72, 2, 150, HF, "packed", "full"),
    (3, 24, 8, 64, 1, 1000, BF, "padded", "packed"),
    (1, 1, 1, 128, 1, 3000, HF, "padded", "masked"),
    (70, 4, 4, 64, 1, 260, BF, "padded", "packed"),
    (9, 12, 12, 64, 300, 200, BF, "padded", "masked"),
    # many items of one key tile for each SM, and of an odd number of tiles
    (300, 4, 4, 128, 40, 90, BF, "padded", "full"),
    (300, 4, 4, 64, 40, 90, HF, "padded", "full"),
    (200, 4, 4, 128, 9, 390, HF, "padded", "packed"),
    (200, 4, 2, 64, 9, 390, BF, "packed", "masked"),
]


@pytest.mark.parametrize("B,H,Hk,d,Lq,Lk,dtype,q,k", CASES)
def test_forward_matches_oracle(lib, B, H, Hk, d, Lq, Lk, dtype, q, k):
    x = inputs(B, H, Hk, d, Lq, Lk, dtype, q, k, seed=B + H + Lq + Lk)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(dev["q"], float("nan"))
    got, stats = call(lib, x, dev, out=out, with_stats=True, status=status)
    w = want(oracle, x, d ** -0.5)
    check_forward(got, w, dtype, d, stats.lse, stats.out_lo)
    assert int(status.item()) == lib.DF_OK
    assert torch.equal(call(lib, x, dev), got)  # without statistics, and again: the same bits


@pytest.mark.parametrize("sigma,scale", [(4.0, None), (16.0, None), (1.0, 2.5), (1.0, 1e-3)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_large_and_small_scores(lib, sigma, scale, dtype):
    x = inputs(2, 4, 2, 64, 90, 400, dtype, "padded", "masked", seed=5, sigma=sigma)
    got, stats = call(lib, x, to_dev(x), scale=scale, with_stats=True)
    w = want(oracle, x, 64 ** -0.5 if scale is None else float(np.float32(scale)))
    check_forward(got, w, dtype, 64, stats.lse, stats.out_lo)


@pytest.mark.parametrize("d,Lq,Lk", [(64, 40, 300), (128, 1, 900), (96, 200, 140)])
def test_masked_and_foreign_rows_may_hold_anything(lib, d, Lq, Lk):
    # masked keys, keys behind a packed sequence, and the other sequences' rows
    x = inputs(3, 4, 2, d, Lq, Lk, BF, "padded", "masked", seed=d, nk=[Lk, 0, Lk // 2])
    dev = to_dev(x)
    clean = call(lib, x, dev)
    off = dev["key_mask"] == 0
    for junk in (float("nan"), float("inf"), -float("inf"), torch.finfo(BF).min):
        for n in ("k", "v"):
            dev[n] = dev[n].clone()
            dev[n][off] = junk
        assert torch.equal(call(lib, x, dev), clean)
    assert int((clean[1] != 0).sum()) == 0  # no valid key
    x = inputs(3, 4, 2, d, Lq, Lk, BF, "packed", "packed", seed=d, nq=[Lq, Lq, Lq], nk=[Lk // 2 + 3, 5, Lk])
    dev = to_dev(x)
    clean = call(lib, x, dev)
    a, b = int(x["cu_k"][1]), int(x["cu_k"][2])
    for n in ("k", "v"):
        dev[n] = dev[n].clone()
        dev[n][a:b] = float("nan")
    dev["q"] = dev["q"].clone()
    dev["q"][Lq:2 * Lq] = float("nan")
    dirty = call(lib, x, dev)
    assert torch.equal(dirty[:Lq], clean[:Lq]) and torch.equal(dirty[2 * Lq:], clean[2 * Lq:])


def test_rows_behind_the_last_sequence_and_empty_sequences(lib):
    x = inputs(5, 4, 2, 64, 200, 200, BF, "packed", "packed", seed=3, nq=[0, 150, 0, 200, 7], nk=[9, 0, 30, 200, 1])
    w = want(oracle, x, 0.125)
    for n in ("q", "k", "v"):
        more = torch.full((300,) + tuple(x[n].shape[1:]), float("nan"), dtype=BF)
        x[n] = torch.cat([x[n], more])
    dev = to_dev(x)
    got, stats = call(lib, x, dev, with_stats=True, out=torch.full_like(dev["q"], 7.0))
    T = 357
    assert int((got[T:] != 0).sum()) == 0 and bool((stats.lse[T:] == -float("inf")).all())
    check_forward(got[:T], w, BF, 64, stats.lse[:T], stats.out_lo[:T])
    assert int((got[:150] != 0).sum()) == 0  # queries of a sequence without keys


@pytest.mark.parametrize("B,d,Lq,Lk", [(2, 64, 40, 2000), (40, 64, 40, 300), (2, 128, 40, 2000), (40, 128, 40, 300)])
def test_nan_that_counts_stays_in_its_rows(lib, B, d, Lq, Lk):
    # few query tiles (clusters) and many; a query row of NaN, and one NaN key of one sequence
    x = inputs(B, 4, 4, d, Lq, Lk, BF, seed=11)
    dev = to_dev(x)
    clean = call(lib, x, dev)
    dev["q"][0, 7, 2] = float("nan")
    dev["k"][1, Lk - 1, 1, 0] = float("nan")
    got, stats = call(lib, x, dev, with_stats=True)
    bad = torch.zeros(got.shape[:3], dtype=torch.bool, device="cuda")
    bad[0, 7, 2] = True
    bad[1, :, 1] = True
    assert bool(got[bad].isnan().all()) and bool(stats.lse[bad].isnan().all())
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Lk", [40, 200, 300])
def test_infinite_value_that_counts_is_the_result(lib, d, Lk):
    x = inputs(200, 2, 2, d, 30, Lk, BF, seed=2)
    dev = to_dev(x)
    clean = call(lib, x, dev)
    dev["v"][3, Lk - 1, 1, 5] = float("inf")
    got = call(lib, x, dev)
    assert bool((got[3, :, 1, 5] == float("inf")).all())
    got[3, :, 1, 5] = clean[3, :, 1, 5]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("d", [64, 128])
def test_very_many_short_sequences(lib, d):
    # tiles are found by number: parts of the batch give the same bits
    B, H, Hk = 20000, 4, 2
    x = inputs(B, H, Hk, d, 4, 8, BF, "packed", "packed", seed=d)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, stats = call(lib, x, dev, with_stats=True, status=status)
    grads = call_bwd(lib, x, dev, out, stats, status=status)
    assert int(status.item()) == lib.DF_OK
    for b in (0, 9990, B - 100):
        q, k = (slice(int(x[c][b]), int(x[c][b + 100])) for c in ("cu_q", "cu_k"))
        part = dict(x, Lq=4, Lk=8)
        on = dict(q=dev["q"][q], k=dev["k"][k], v=dev["v"][k], dout=dev["dout"][q], key_mask=None,
                  cu_q=(dev["cu_q"][b:b + 101] - q.start).contiguous(),
                  cu_k=(dev["cu_k"][b:b + 101] - k.start).contiguous())
        o, s = call(lib, part, on, with_stats=True)
        g = call_bwd(lib, part, on, o, s)
        assert torch.equal(o, out[q]) and torch.equal(s.lse, stats.lse[q])
        assert torch.equal(g[0], grads[0][q]) and torch.equal(g[1], grads[1][k]) and torch.equal(g[2], grads[2][k])


def test_two_calls_at_once(lib):
    # on two streams, each with its own tiles to hand out
    xs = [inputs(24, 4, 4, 64, 150, 700, BF, "packed", "packed", seed=s) for s in (1, 2)]
    devs = [to_dev(x) for x in xs]
    alone = [call(lib, x, dev) for x, dev in zip(xs, devs)]
    outs = [[torch.empty_like(dev["q"]) for _ in range(10)] for dev in devs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for i in range(10):
        for x, dev, out, s in zip(xs, devs, outs, streams):
            with torch.cuda.stream(s):
                call(lib, x, dev, out=out[i], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == lib.DF_OK
    assert all(torch.equal(o, a) for out, a in zip(outs, alone) for o in out)


@pytest.mark.parametrize("B,H,Hk,d,Lq,Lk,q,k", [
    (200, 12, 12, 64, 140, 300, "packed", "packed"),   # many items, some of one tile or none
    (60, 12, 4, 128, 90, 500, "packed", "packed"),
    (80, 8, 8, 128, 1, 700, "padded", "packed"),       # single tokens
    (3, 2, 2, 64, 30, 2000, "padded", "masked"),       # clusters
])
def test_repeated_launches_give_equal_bits(lib, B, H, Hk, d, Lq, Lk, q, k):
    # back to back, so that the CTAs of one call end beside those of the next
    x = inputs(B, H, Hk, d, Lq, Lk, BF, q, k, seed=B)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first, stats = call(lib, x, dev, with_stats=True, status=status)
    grads = call_bwd(lib, x, dev, first, stats, status=status)
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(40):
        out, st = call(lib, x, dev, with_stats=True, status=status)
        other += (out != first).sum() + (st.lse != stats.lse).sum()
        for a, b in zip(call_bwd(lib, x, dev, out, st, status=status), grads):
            other += (a != b).sum()
    assert int(other.item()) == 0 and int(status.item()) == lib.DF_OK


def test_no_keys_no_queries_no_sequences(lib):
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    out, stats = lib.df_cross_attn_fwd(z(2, 3, 4, 64), z(2, 0, 4, 64), z(2, 0, 4, 64), with_stats=True)
    assert int((out != 0).sum()) == 0 and bool((stats.lse == -float("inf")).all())
    assert lib.df_cross_attn_fwd(z(2, 0, 4, 64), z(2, 9, 4, 64), z(2, 9, 4, 64)).numel() == 0
    assert lib.df_cross_attn_fwd(z(0, 3, 4, 64), z(0, 9, 4, 64), z(0, 9, 4, 64)).numel() == 0


def test_packed_rows_without_a_sequence(lib):
    z = lambda *s: torch.ones(*s, dtype=BF, device="cuda")  # noqa: E731
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, stats = lib.df_cross_attn_fwd(z(300, 4, 64), z(200, 4, 64), z(200, 4, 64), cu_seqlens_q=cu, cu_seqlens_k=cu,
                                       max_seqlen_q=0, max_seqlen_k=0, with_stats=True)
    assert int((out != 0).sum()) == 0 and bool((stats.lse == -float("inf")).all())
    grads = lib.df_cross_attn_bwd(z(300, 4, 64), z(200, 4, 64), z(200, 4, 64), out, stats, z(300, 4, 64),
                                  cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=0, max_seqlen_k=0)
    assert all(int((g != 0).sum()) == 0 for g in grads)


@pytest.mark.parametrize("side", ["q", "k"])
def test_offsets_beyond_32_bits(lib, side):
    # two sequences, the second one's rows behind 2^32 values of the first one's
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    H, d, far = 16, 128, (1 << 32) // (16 * 128) + 77
    x = inputs(1, H, H, d, 60, 300, BF, seed=4)
    dev = to_dev(x)
    want_out, stats = call(lib, x, dev, with_stats=True)
    want = call_bwd(lib, x, dev, want_out, stats)
    rows = {n: t[0] for n, t in dev.items() if n in ("q", "k", "v", "dout")}
    cu = {}
    for s, names, L in (("q", ("q", "dout"), 60), ("k", ("k", "v"), 300)):
        front = far if s == side else 0
        cu[s] = torch.tensor([0, front, front + L], dtype=torch.int32, device="cuda")
        for n in names:
            big = torch.zeros(front + L, H, d, dtype=BF, device="cuda")
            big[front:] = rows[n]
            rows[n] = big
    kw = dict(cu_seqlens_q=cu["q"], cu_seqlens_k=cu["k"], max_seqlen_q=60, max_seqlen_k=300)
    out, st = lib.df_cross_attn_fwd(rows["q"], rows["k"], rows["v"], with_stats=True, **kw)
    assert torch.equal(out[-60:], want_out[0]) and torch.equal(st.lse[-60:], stats.lse[0])
    got = lib.df_cross_attn_bwd(rows["q"], rows["k"], rows["v"], out, st, rows["dout"], **kw)
    for g, w in zip(got, want):
        assert torch.equal(g[-w.shape[1]:], w[0])


def test_bad_offsets_are_reported(lib):
    x = inputs(3, 2, 2, 64, 40, 100, BF, "packed", "packed", seed=1, nq=[40, 40, 40], nk=[100, 90, 80])
    dev = to_dev(x)
    w = want(oracle, x, 0.125)
    for name, bad in (("cu_k", [0, 100, 90, 270]), ("cu_k", [0, 100, 190, 1 << 29]), ("cu_q", [0, 40, 80, 500])):
        d2 = dict(dev)
        d2[name] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = call(lib, x, d2, status=status)
        assert int(status.item()) == lib.DF_ERR_INVALID_ARG
        first = {n: v[:40] for n, v in w.items()}
        check_forward(got[:40], first, BF, 64)  # the sequence before it is not touched


def test_longer_than_the_stated_bound(lib):
    # max_seqlen sizes the launch only
    x = inputs(2, 4, 4, 64, 300, 500, BF, "packed", "packed", seed=2, nq=[300, 20], nk=[500, 400])
    x["Lq"] = x["Lk"] = 1
    check_forward(call(lib, x, to_dev(x)), want(oracle, x, 0.125), BF, 64)


def test_other_stream_and_captured_replay(lib):
    x = inputs(3, 4, 2, 64, 50, 400, BF, "padded", "masked", seed=4)
    dev = to_dev(x)
    side = torch.cuda.Stream()
    out = torch.empty_like(dev["q"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(lib, x, dev, out=out)
    y = inputs(3, 4, 2, 64, 50, 400, BF, "padded", "masked", seed=6)
    for n in ("q", "k", "v", "key_mask"):
        dev[n].copy_(y[n])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_forward(out, want(oracle, y, 0.125), BF, 64)
    with torch.cuda.stream(side):
        again = call(lib, x, dev)
    side.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("d,Lq,Lk", [(64, 700, 900), (128, 700, 900), (64, 1, 2000)])
def test_wait_budget_runs_out_and_recovers(lib, d, Lq, Lk):
    x = inputs(2, 2, 2, d, Lq, Lk, BF, seed=9)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.df_attn_set_wait_budget(1)
    try:
        call(lib, x, dev, status=status)
        torch.cuda.synchronize()
    finally:
        lib.df_attn_set_wait_budget(0)
    assert int(status.item()) == lib.DF_ERR_DEVICE_TIMEOUT
    check_forward(call(lib, x, dev), want(oracle, x, d ** -0.5), BF, d)


def test_refusals(lib):
    z = lambda *s, t=BF: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    q, k = z(2, 3, 4, 64), z(2, 9, 2, 64)
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(lib.DFError):
            lib.df_cross_attn_fwd(q, k, k, **bad)
    with pytest.raises(lib.DFError):
        lib.df_cross_attn_fwd(z(2, 3, 3, 64), k, k)  # 3 query heads, 2 key heads
    with pytest.raises(lib.DFError):
        lib.df_cross_attn_fwd(z(2, 3, 4, 136), z(2, 9, 2, 136), z(2, 9, 2, 136))
    with pytest.raises(lib.DFError):
        lib.df_cross_attn_fwd(z(2, 3, 4, 64, t=torch.float32), k.float(), k.float())
    with pytest.raises(ValueError):
        lib.df_cross_attn_fwd(q, k, k.half())
    with pytest.raises(ValueError):
        lib.df_cross_attn_fwd(q, k.transpose(1, 2), k.transpose(1, 2))
    with pytest.raises(ValueError):
        lib.df_cross_attn_fwd(q, k, k, key_mask=torch.ones(2, 8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        lib.df_cross_attn_fwd(q, z(3, 9, 2, 64), z(3, 9, 2, 64))
    cu = torch.tensor([0, 9, 18], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="max_seqlen_k"):
        lib.df_cross_attn_fwd(q, z(18, 2, 64), z(18, 2, 64), cu_seqlens_k=cu)
    odd = torch.zeros(2 * 3 * 4 * 64 + 4, dtype=BF, device="cuda")[4:].view(2, 3, 4, 64)
    with pytest.raises(lib.DFError):
        lib.df_cross_attn_fwd(odd, k, k)
