"""The decoder's attention at its limits: waits that run out, calls beside one another on two
streams, more sequences than a CTA has threads, bounds that rows break, rows beyond 32 bits."""

import numpy as np
import pytest
import torch

import oracle
from _cache import fill, offsets, oracles, tokens
from _causal import call, call_bwd, want
from _cross import check_backward, check_forward, inputs, np64, to_dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def attended(q, lens, nq, both, window, sinks, scale):
    """The oracle's results for packed rows q of sequences that hold `lens` tokens."""
    at, rows = np.concatenate([[0], np.cumsum(nq)]), []
    for b, n in enumerate(lens):
        k, v = (o.values()[:n] for o in both[b])
        rows.append(oracle.causal_rows(np64(q[at[b]:at[b + 1]]), k, v, np.ones(n, bool), scale, window, sinks))
    return {name: np.concatenate([r[name] for r in rows]) for name in rows[0]}


@pytest.mark.parametrize("H,Hk,d,Lq", [(24, 24, 64, 1), (32, 8, 128, 8), (16, 8, 96, 12)])
def test_waits_of_the_cache_run_out_and_recover(lib, H, Hk, d, Lq):
    """(Enough work that copies queue for the memory; alone, they land before they are waited for.)"""
    B, n, page = 48, 8192, 64
    cache = lib.df_cache_new(B * n // page, Hk, page, d)
    table = torch.randperm(B * n // page, generator=torch.Generator().manual_seed(d)).to(torch.int32).view(B, -1).cuda()
    held = torch.full((B,), n, dtype=torch.int32, device="cuda")
    k = torch.randn(B, n, Hk, d, generator=torch.Generator(device="cuda").manual_seed(d), dtype=BF, device="cuda")
    lib.df_cache_append(k, k, cache, table, torch.zeros_like(held))
    q = torch.randn(B, Lq, H, d, generator=torch.Generator().manual_seed(d)).to(BF).cuda()
    want = lib.df_cache_attn(q, cache, table, held)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.df_attn_set_wait_budget(1)
    try:
        lib.df_cache_attn(q, cache, table, held, status=status)
        st = int(status.item())
    finally:
        lib.df_attn_set_wait_budget(0)
    assert st == lib.DF_ERR_DEVICE_TIMEOUT, lib.status_string(st)
    status.zero_()
    assert torch.equal(lib.df_cache_attn(q, cache, table, held, status=status), want)
    assert int(status.item()) == lib.DF_OK


@pytest.mark.parametrize("B,H,Hk,L", [(2, 4, 2, 700), (30, 8, 8, 300)])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF)])
def test_waits_of_causal_attention_run_out_and_recover(lib, d, dtype, B, H, Hk, L):
    """(Items of one query tile, and of two.)"""
    x = inputs(B, H, Hk, d, L, L, dtype, "padded", "full", seed=d)
    dev = to_dev(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(window=300, sinks=2)
    out, stats = call(lib, x, dev, with_stats=True, **kw)
    grads = call_bwd(lib, x, dev, out, stats, **kw)
    for run in (lambda: call(lib, x, dev, status=status, **kw), lambda: call_bwd(lib, x, dev, out, stats, status=status, **kw)):
        status.zero_()
        lib.df_attn_set_wait_budget(1)
        try:
            run()
            st = int(status.item())
        finally:
            lib.df_attn_set_wait_budget(0)
        assert st == lib.DF_ERR_DEVICE_TIMEOUT, lib.status_string(st)
    assert torch.equal(call(lib, x, dev, **kw), out)
    assert all(torch.equal(a, b) for a, b in zip(call_bwd(lib, x, dev, out, stats, **kw), grads))


def test_two_calls_at_once(lib):
    """Training steps with a workspace each, and attention to one cache, on two streams."""
    work = []
    for i, (d, dtype) in enumerate([(64, BF), (128, HF)]):
        x = inputs(3, 8, 4, d, 900, 900, dtype, "padded", "full", seed=i)
        calls = tokens([[2000, 700]], 2, d, dtype, seed=i)
        cache, table, held = fill(lib, calls, 2, d, 32)
        q = torch.randn(2, 4, 8, d, generator=torch.Generator().manual_seed(i)).to(dtype).cuda()
        ws = torch.empty(lib.df_cross_attn_bwd_workspace_size(2700, 8), dtype=torch.uint8, device="cuda")
        work.append((x, to_dev(x), ws, q, cache, table, held))

    def run(job, stream=None):
        x, dev, ws, q, cache, table, held = job
        kw = dict(window=200, sinks=3, stream=stream)
        out, stats = call(lib, x, dev, with_stats=True, **kw)
        grads = call_bwd(lib, x, dev, out, stats, workspace=ws, **kw)
        a = lib.df_cache_attn(q, cache, table, held, window=500, sinks=3, stream=stream)
        b = lib.df_cache_attn(q, cache, table, held, causal=False, stream=stream)
        return [out, *grads, a, b]

    want = [run(job) for job in work]
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(job, s) for job, s in zip(work, streams)]
        same = [run((*job[:2], torch.empty_like(job[2]), *job[3:]), s) for job, s in zip(work, reversed(streams))]
        torch.cuda.synchronize()
        for w, g, h in zip(want, got, same):
            assert all(torch.equal(i, j) and torch.equal(i, k) for i, j, k in zip(w, g, h))


@pytest.mark.parametrize("B", [127, 128, 129, 700])
def test_many_short_sequences(lib, B):
    Hk, H, d = 2, 6, 64
    lens = [(7 * b) % 50 for b in range(B)]  # some hold nothing
    calls = tokens([lens], Hk, d, HF, seed=B)
    cache, table, held = fill(lib, calls, Hk, d, 16)
    q = torch.randn(B, H, d, generator=torch.Generator().manual_seed(B)).to(HF)
    lse = torch.zeros(B, 1, H, device="cuda")
    got = lib.df_cache_attn(q[:, None].cuda(), cache, table, held, window=33, lse=lse)
    check_forward(got[:, 0], attended(q, lens, [1] * B, oracles(calls, Hk, d), 33, 0, d ** -0.5), HF, d, lse[:, 0])


@pytest.mark.parametrize("Lq", [3, 20])
def test_rows_beyond_their_bound_are_reported_and_left(lib, Lq):
    """The rows within it are those at the right positions."""
    lens, nq, d = [90, 40, 70], [2, Lq + 5, 3], 64
    calls = tokens([lens], 2, d, BF, seed=Lq)
    cache, table, held = fill(lib, calls, 2, d, 16)
    q = torch.randn(sum(nq), 4, d, generator=torch.Generator().manual_seed(Lq)).to(BF)
    w = attended(q, lens, nq, oracles(calls, 2, d), 30, 2, d ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0).cuda()
    lib.df_cache_attn(q.cuda(), cache, table, held, offsets(nq).cuda(), max_seqlen_q=Lq, window=30, sinks=2, out=out,
                      status=status)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG
    kept = np.r_[0:2 + Lq, 2 + Lq + 5:sum(nq)]
    check_forward(out[torch.from_numpy(kept).cuda()], {n: t[kept] for n, t in w.items()}, BF, d)
    assert int((out[2 + Lq:2 + Lq + 5] != 7.0).sum()) == 0


def test_calls_with_nothing_to_do(lib):
    cache = lib.df_cache_new(2, 2, 16, 64)
    table, held = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    rows = lambda *n: torch.empty(*n, 2, 64, dtype=BF, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for B, n in ((3, 0), (0, 1), (0, 0)):
        lib.df_cache_append(rows(B, n), rows(B, n), cache, table[:B], held[:B], status=status)
        assert lib.df_cache_attn(rows(B, n), cache, table[:B], held[:B], status=status).shape == (B, n, 2, 64)
        assert lib.df_cache_read(cache, table[:B], held[:B], rows=n, status=status)[0].shape == (B, n, 2, 64)
    # no token held, and no page either
    for t in (table, table[:, :0].contiguous()):
        assert int((lib.df_cache_attn(rows(3, 2).zero_(), cache, t, held, status=status) != 0).sum()) == 0
        assert int((lib.df_cache_read(cache, t, held, rows=20, status=status)[0] != 0).sum()) == 0
    assert int((lib.df_cache_read(cache, table[:0], held[:0], offsets([]).cuda(), rows=5, status=status)[1] != 0).sum()) == 0
    assert int(status.item()) == lib.DF_OK


def test_rows_of_attention_beyond_32_bits(lib):
    """2^31 elements of queries, keys and values; the sequences at both ends against the oracle."""
    B, L, H, d = 4096, 130, 64, 64
    assert B * L * H * d > 2 ** 31
    n = [L] * B
    n[1] = 0
    T = sum(n)
    g = torch.Generator(device="cuda").manual_seed(3)
    dev = {name: torch.randn(T, H, d, generator=g, device="cuda", dtype=BF) for name in ("q", "k", "v", "dout")}
    dev.update(key_mask=None, cu_q=offsets(n).cuda(), cu_k=offsets(n).cuda())
    x = dict(Lq=L, Lk=L)
    kw = dict(window=60, sinks=2)
    out, stats = call(lib, x, dev, with_stats=True, **kw)
    grads = call_bwd(lib, x, dev, out, stats, **kw)
    for rows in (slice(0, L), slice(T - L, T)):
        for h in (0, H - 1):
            part = {name: dev[name][rows, h:h + 1].cpu() for name in ("q", "k", "v", "dout")}
            cu = torch.tensor([0, L], dtype=torch.int32)
            w = want(oracle, dict(part, key_mask=None, cu_q=cu, cu_k=cu), d ** -0.5, 60, 2, with_grad=True)
            check_forward(out[rows, h:h + 1], w, BF, d, stats.lse[rows, h:h + 1], stats.out_lo[rows, h:h + 1])
            check_backward([t[rows, h:h + 1] for t in grads], w, BF, d)


def test_rows_of_positions_beyond_32_bits(lib):
    T, heads, d = 700_000, 48, 64
    assert T * heads * d > 2 ** 31
    x = torch.zeros(T, heads, d, dtype=BF, device="cuda")
    some = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    rows = torch.randn(5, heads, d, generator=torch.Generator().manual_seed(1)).to(BF)
    x[some] = rows.cuda()
    positions = torch.arange(T, dtype=torch.int32, device="cuda")
    table = lib.df_rotary_table(d)
    lib.df_rotary(x, positions, table, out=x)
    want = lib.df_rotary(rows.cuda(), positions[some].contiguous(), table)
    assert torch.equal(x[some], want)
    x[some] = 0
    assert int((x != 0).sum()) == 0
