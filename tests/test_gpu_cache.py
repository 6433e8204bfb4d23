"""The 8-bit cache on the GPU: tokens appended in parts against the oracle (equal values, equal
bytes), read back, and attention to it within bounds counted in roundings."""

import numpy as np
import pytest
import torch

import oracle
from _cache import fill, offsets, oracles, tokens
from _cross import check_forward, np64

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

PARTS = [  # heads, d, page, dtype, tokens of each sequence by call
    (2, 64, 16, BF, [[5, 16, 0]]),
    (1, 32, 32, HF, [[1], [1], [14], [1], [40]]),
    (3, 128, 48, BF, [[100, 0, 17, 1], [1, 1, 1, 1], [30, 47, 0, 200]]),
    (2, 96, 64, HF, [[0, 63], [65, 0], [1, 2]]),
    (12, 64, 128, BF, [[700, 3, 128], [1, 1, 1]]),
]


@pytest.mark.parametrize("heads,d,page,dtype,parts", PARTS)
def test_appended_tokens_read_back(lib, heads, d, page, dtype, parts):
    calls = tokens(parts, heads, d, dtype, seed=page + d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache, table, held = fill(lib, calls, heads, d, page, status=status)
    want = oracles(calls, heads, d)
    lens = held.tolist()
    cu = offsets(lens).cuda()
    for t in (F32, BF, HF):
        k, v = lib.df_cache_read(cache, table, held, cu, rows=sum(lens), dtype=t, status=status)
        for i, x in enumerate((k, v)):
            ref = np.concatenate([o[i].values() for o in want])
            assert np.array_equal(np64(x), np64(torch.from_numpy(ref).to(t)))
    # padded, with room behind each sequence
    k, v = lib.df_cache_read(cache, table, held, rows=max(lens) + 7, dtype=F32)
    for b, n in enumerate(lens):
        assert np.array_equal(np64(k[b, :n]), want[b][0].values()) and int((k[b, n:] != 0).sum()) == 0
        assert np.array_equal(np64(v[b, :n]), want[b][1].values()) and int((v[b, n:] != 0).sum()) == 0
    # the records' bytes
    raw, at = cache.cpu().numpy(), table.cpu().numpy()
    for b, n in enumerate(lens):
        for blk in range(-(-n // 16)):
            rows = min(16, n - blk * 16)
            for h in range(heads):
                got = raw[at[b, blk * 16 // page], h, blk % (page // 16)]
                ref = oracle.record(*want[b], blk, h)
                slabs = lambda r: r[:32 * d].reshape(2, d // 32, 16, 32)[:, :, :rows]  # noqa: E731
                assert np.array_equal(slabs(got), slabs(ref)) and np.array_equal(got[32 * d:32 * d + 8], ref[32 * d:])
    assert int(status.item()) == lib.DF_OK


def test_appending_again_changes_nothing_and_touches_nothing_else(lib):
    heads, d, page = 2, 64, 32
    calls = tokens([[20, 40], [7, 30]], heads, d, BF, seed=1)
    cache, table, held = fill(lib, calls, heads, d, page)
    before = cache.clone()
    n, k, v = calls[1]
    old = torch.tensor(calls[0][0], dtype=torch.int32, device="cuda")
    out = lib.df_cache_append(k.cuda(), v.cuda(), cache, table, old, offsets(n).cuda())
    assert out is cache and torch.equal(cache, before)
    raw = cache.cpu().numpy()
    used = {int(x) for x in table.flatten().tolist() if x >= 0}
    assert all((raw[p] == 0xFF).all() for p in set(range(raw.shape[0])) - used)
    # codes behind the last token, and the unused bytes
    rec = raw[int(table[0, 27 // 32]), 0, (27 % 32) // 16]
    assert (rec[:32 * d].reshape(2, 2, 16, 32)[:, :, 27 % 16:] == 0xFF).all() and (rec[32 * d + 8:] == 0xFF).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_extreme_values(lib, dtype):
    heads, d = 1, 32
    top = float(torch.finfo(dtype).max)
    rows = torch.zeros(96, heads, d)
    rows[16:32] = torch.linspace(-1, 1, 32) * 1e-7             # small: fp16 subnormals
    rows[32:48, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), top])
    rows[48:64] = torch.linspace(-1, 1, 32) * top
    rows[64, 0, 0], rows[65:80] = 448.0 * 64, torch.linspace(0.01, 3, 32)  # subnormal codes beside a large one
    rows[80:96] = torch.exp2(torch.arange(16.0) - 8)[:, None, None] * 1.3   # the scale grows token by token
    rows = rows.to(dtype)
    calls = [([80], rows[:80], -rows[:80])] + [([1], rows[80 + i:81 + i], -rows[80 + i:81 + i]) for i in range(16)]
    cache, table, held = fill(lib, calls, heads, d, 16)
    want = oracles(calls, heads, d)[0]
    k, v = lib.df_cache_read(cache, table, held, rows=96, dtype=F32)
    for got, o in ((k, want[0]), (v, want[1])):
        assert np.array_equal(np64(got[0]), o.values().astype(np.float32).astype(np.float64), equal_nan=True)
    k16, _ = lib.df_cache_read(cache, table, held, rows=96, dtype=HF)
    ref = np.clip(np64(k[0]), -65504, 65504).astype(np.float16).astype(np.float64)
    assert np.array_equal(np64(k16[0]), ref, equal_nan=True)


def test_missing_pages_and_bad_lengths_are_reported(lib):
    heads, d, page = 2, 64, 16
    calls = tokens([[40, 40, 40]], heads, d, BF, seed=2)
    cache, table, held = fill(lib, calls, heads, d, page)
    before = cache.clone()
    q = torch.randn(3, 1, 4, d).to(BF).cuda()
    good = lib.df_cache_attn(q, cache, table, held)
    for bad in (-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = lib.df_cache_attn(q, cache, t, held, status=status)
        assert int(status.item()) == lib.DF_ERR_INVALID_ARG
        status.zero_()
        wide = torch.cat([t, torch.full((3, 20000), bad, dtype=torch.int32, device="cuda")], dim=1)
        assert bool(((lib.df_cache_attn(q, cache, wide, held, status=status).float() - out.float()).abs() <= 2.0 ** -6).all())
        assert int(status.item()) == lib.DF_ERR_INVALID_ARG
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2]) and bool(torch.isfinite(out).all())
        # the tokens of the missing page do not count
        want = oracles(calls, heads, d)[1]
        keep = np.r_[0:16, 32:40]
        w = oracle.cross_rows(np64(q[1]), want[0].values()[keep], want[1].values()[keep], np.ones(24, bool), d ** -0.5)
        check_forward(out[1], w, BF, d)
        status.zero_()
        k, v = lib.df_cache_read(cache, t, held, rows=40, dtype=F32, status=status)
        assert int(status.item()) == lib.DF_ERR_INVALID_ARG and int((k[1, 16:32] != 0).sum()) == 0
        status.zero_()
        zero = torch.zeros(3, dtype=torch.int32, device="cuda")
        lib.df_cache_append(calls[0][1].cuda(), calls[0][2].cuda(), cache, t, zero, offsets([40] * 3).cuda(), status=status)
        assert int(status.item()) == lib.DF_ERR_INVALID_ARG and torch.equal(cache, before)
    # a sequence longer than its row of the table
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    long = held.clone()
    long[0] = 2 ** 31 - 1
    out = lib.df_cache_attn(q, cache, table, long, window=8, status=status)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG and int((out[0] != 0).sum()) == 0
    status.zero_()
    long[0] = -5
    out = lib.df_cache_attn(q, cache, table, long, status=status)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG and int((out[0] != 0).sum()) == 0
    status.zero_()
    lib.df_cache_append(calls[0][1].cuda(), calls[0][2].cuda(), cache, table, long, offsets([40, 0, 0]).cuda(), status=status)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG and torch.equal(cache, before)
    # offsets that go back, or behind the rows
    for cu in ([0, 40, 20, 120], [0, 40, 80, 121], [-1, 40, 80, 120]):
        status.zero_()
        lib.df_cache_append(calls[0][1].cuda(), calls[0][2].cuda(), cache, table, zero,
                            torch.tensor(cu, dtype=torch.int32, device="cuda"), status=status)
        assert int(status.item()) == lib.DF_ERR_INVALID_ARG


ATTN = [  # B, H, Hk, d, Lq, page, longest, dtype, causal, window, sinks
    (1, 1, 1, 64, 1, 16, 1, BF, True, 0, 0),
    (3, 4, 4, 64, 1, 64, 300, HF, True, 0, 0),
    (2, 12, 12, 64, 1, 64, 512, BF, True, 0, 0),
    (5, 8, 1, 128, 1, 16, 700, BF, True, 0, 0),
    (3, 9, 1, 32, 1, 48, 200, HF, True, 0, 0),          # 9 rows: both halves of a tile
    (4, 6, 2, 96, 3, 32, 333, BF, True, 40, 0),
    (3, 8, 2, 128, 4, 16, 400, HF, True, 50, 5),
    (2, 16, 2, 64, 4, 128, 260, BF, True, 33, 16),      # 32 rows
    (2, 8, 1, 96, 7, 16, 300, HF, True, 100, 40),       # 56 rows
    (1, 4, 1, 64, 50, 32, 200, BF, True, 20, 1),        # 200 rows: four tiles
    (2, 3, 1, 32, 1, 16, 1000, BF, True, 1, 0),
    (2, 2, 2, 64, 1, 16, 2000, HF, True, 70, 100),
    (3, 4, 2, 128, 5, 64, 150, BF, False, 0, 0),
    (64, 4, 4, 64, 1, 16, 90, BF, False, 0, 0),
    (1, 2, 1, 64, 1, 256, 9000, HF, False, 0, 0),       # clusters of eight
    (1, 32, 1, 128, 3, 64, 5000, BF, True, 0, 0),
]


def sequences(B, longest, Lq, seed):
    n = [int(x) for x in np.random.default_rng(seed).integers(0, longest + 1, B)]
    n[0] = longest
    if B > 2:
        n[1], n[2] = 0, min(Lq, longest)
    return n


def want_attn(x, lens, nq, both, causal, window, sinks, scale):
    rows, at = [], 0
    for b, n in enumerate(nq):
        k, v = both[b][0].values(), both[b][1].values()
        q = x[at:at + n]
        at += n
        rows.append(oracle.causal_rows(q, k, v, np.ones(lens[b], bool), scale, window, sinks) if causal
                    else oracle.cross_rows(q, k, v, np.ones(lens[b], bool), scale))
    return {name: np.concatenate([r[name] for r in rows]) for name in rows[0]}


@pytest.mark.parametrize("B,H,Hk,d,Lq,page,longest,dtype,causal,window,sinks", ATTN)
def test_attention_matches_oracle(lib, B, H, Hk, d, Lq, page, longest, dtype, causal, window, sinks):
    lens = sequences(B, longest, Lq, seed=longest)
    calls = tokens([lens], Hk, d, dtype, seed=d + page)
    cache, table, held = fill(lib, calls, Hk, d, page)
    both = oracles(calls, Hk, d)
    g = torch.Generator().manual_seed(longest + 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(causal=causal, window=window, sinks=sinks, status=status)
    # padded
    q = torch.randn(B, Lq, H, d, generator=g).to(dtype)
    out, lse = torch.full((B, Lq, H, d), float("nan"), dtype=dtype, device="cuda"), torch.zeros(B, Lq, H, device="cuda")
    got = lib.df_cache_attn(q.cuda(), cache, table, held, out=out, lse=lse, **kw)
    assert got is out
    w = want_attn(np64(q).reshape(-1, H, d), lens, [Lq] * B, both, causal, window, sinks, d ** -0.5)
    check_forward(out.view(-1, H, d), w, dtype, d, lse.view(-1, H))
    # another split (which goes by the room in the table)
    wide = torch.cat([table, torch.full((B, 330_000 // page), -1, dtype=torch.int32, device="cuda")], dim=1)
    out, lse = torch.full((B, Lq, H, d), float("nan"), dtype=dtype, device="cuda"), torch.zeros(B, Lq, H, device="cuda")
    got = lib.df_cache_attn(q.cuda(), cache, wide, held, out=out, lse=lse, **kw)
    check_forward(out.view(-1, H, d), w, dtype, d, lse.view(-1, H))
    for t in (table, wide):
        assert torch.equal(lib.df_cache_attn(q.cuda(), cache, t, held, **kw), lib.df_cache_attn(q.cuda(), cache, t, held, **kw))
    # packed, ragged, with rows behind the last sequence; another scale
    nq = [min(Lq, 1 + (3 * b) % (Lq + 1)) for b in range(B)]
    if B > 1:
        nq[-1] = 0
    x = torch.randn(sum(nq) + 3, H, d, generator=g).to(dtype)
    w = want_attn(np64(x), lens, nq, both, causal, window, sinks, float(np.float32(0.31)))
    for t in (table, wide):
        out = torch.full_like(x, 7.0).cuda()
        lib.df_cache_attn(x.cuda(), cache, t, held, offsets(nq).cuda(), max_seqlen_q=Lq, scale=0.31, out=out, **kw)
        check_forward(out[:sum(nq)], w, dtype, d)
        assert int((out[sum(nq):] != 7.0).sum()) == 0
    assert int(status.item()) == lib.DF_OK


@pytest.mark.parametrize("B,H,Hk,d,Lq,page,longest,dtype,causal,window,sinks", [
    (30, 8, 8, 64, 1, 64, 1500, BF, True, 0, 0), (256, 4, 4, 32, 1, 16, 400, HF, True, 0, 0),
    (20, 16, 4, 128, 4, 16, 4000, BF, True, 1000, 20), (12, 16, 8, 96, 9, 32, 4100, HF, False, 0, 0)])
def test_more_work_than_a_round_of_the_gpu(lib, B, H, Hk, d, Lq, page, longest, dtype, causal, window, sinks):
    lens = sequences(B, longest, Lq, seed=B)
    calls = tokens([lens], Hk, d, dtype, seed=B)
    cache, table, held = fill(lib, calls, Hk, d, page)
    q = torch.randn(B, Lq, H, d, generator=torch.Generator().manual_seed(B)).to(dtype)
    got = lib.df_cache_attn(q.cuda(), cache, table, held, causal=causal, window=window, sinks=sinks)
    w = want_attn(np64(q).reshape(-1, H, d), lens, [Lq] * B, oracles(calls, Hk, d), causal, window, sinks, d ** -0.5)
    check_forward(got.view(-1, H, d), w, dtype, d)


def test_split_by_any_bound_of_the_length(lib):
    calls = tokens([[3000]], 2, 64, BF, seed=4)
    cache, table, held = fill(lib, calls, 2, 64, 64)
    both = oracles(calls, 2, 64)
    q = torch.randn(1, 1, 4, 64, generator=torch.Generator().manual_seed(5)).to(BF)
    w = want_attn(np64(q)[0], [3000], [1], both, True, 0, 0, 0.125)
    table = torch.cat([table, torch.full((1, 6000), -1, dtype=torch.int32, device="cuda")], dim=1)
    for bound in (0, 1, 200, 600, 3000, 1 << 20):
        check_forward(lib.df_cache_attn(q.cuda(), cache, table, held, max_length=bound)[0], w, BF, 64)


@pytest.mark.parametrize("sigma", [1e-30, 1e-3, 30.0])
def test_queries_and_values_of_any_size(lib, sigma):
    """bf16 queries and values far outside fp16's range; large scores."""
    calls = tokens([[200, 77]], 2, 64, BF, seed=6, sigma=1.0)
    calls = [(n, k, (v.float() * sigma ** 0.5).to(BF)) for n, k, v in calls]
    cache, table, held = fill(lib, calls, 2, 64, 32)
    both = oracles(calls, 2, 64)
    q = (torch.randn(2, 2, 4, 64, generator=torch.Generator().manual_seed(7)) * sigma).to(BF)
    out, lse = lib.df_cache_attn(q.cuda(), cache, table, held), torch.zeros(2, 2, 4, device="cuda")
    lib.df_cache_attn(q.cuda(), cache, table, held, lse=lse)
    w = want_attn(np64(q).reshape(-1, 4, 64), [200, 77], [2, 2], both, True, 0, 0, 0.125)
    check_forward(out.view(-1, 4, 64), w, BF, 64, lse.view(-1, 4))


def test_pages_behind_the_window_may_be_gone(lib):
    lens, page = [700, 650], 16
    calls = tokens([lens], 2, 64, BF, seed=8)
    cache, table, held = fill(lib, calls, 2, 64, page)
    q = torch.randn(2, 3, 4, 64).to(BF).cuda()
    kw = dict(window=100, sinks=5)
    want = lib.df_cache_attn(q, cache, table, held, **kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        first = (n - 3 - 100 + 1) // page
        table[b, 1:first] = -1
    assert torch.equal(lib.df_cache_attn(q, cache, table, held, status=status, **kw), want)
    assert int(status.item()) == lib.DF_OK


def test_shared_pages_and_not_a_number(lib):
    calls = tokens([[64, 40]], 1, 64, HF, seed=9)
    cache, table, held = fill(lib, calls, 1, 64, 32)
    table[1, 0] = table[0, 0]  # a prefix of two sequences
    q = torch.randn(1, 1, 2, 64).to(HF).cuda().expand(2, 1, 2, 64).contiguous()
    held[0] = held[1]
    one = lib.df_cache_attn(q[:1], cache, table[:1], held[:1])
    assert torch.equal(lib.df_cache_attn(q, cache, table, held)[0], one[0])
    nan = torch.full((1, 1, 64), float("nan"), dtype=HF, device="cuda")
    good = torch.zeros(1, 1, 64, dtype=HF, device="cuda")
    at = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")  # noqa: E731
    lib.df_cache_append(nan, good, cache, table[:1], at(35), offsets([1]).cuda())
    assert bool(torch.isnan(lib.df_cache_attn(q[:1], cache, table[:1], at(38))).all())
    assert torch.equal(lib.df_cache_attn(q[:1], cache, table[:1], at(35)), lib.df_cache_attn(q[:1], cache, table[:1], at(35)))
    assert bool(torch.isfinite(lib.df_cache_attn(q[:1], cache, table[:1], at(35))).all())       # not yet among the tokens
    assert bool(torch.isfinite(lib.df_cache_attn(q[:1], cache, table[:1], at(38), window=2)).all())  # behind the window


def test_captured_step_replays_with_new_tokens(lib):
    """Append and attend captured once; lengths and tokens change from replay to replay."""
    heads, d, page, B = 2, 64, 16, 3
    calls = tokens([[30, 1, 47]], heads, d, BF, seed=10)
    cache, table, held = fill(lib, calls, heads, d, page)
    n_pages = cache.shape[0]
    bigger = lib.df_cache_new(n_pages + 3, heads, page, d)
    bigger[:n_pages] = cache
    table = torch.cat([table, torch.full((B, 1), -1, dtype=torch.int32, device="cuda")], dim=1)
    for b in range(B):
        table[b, int(-(-int(held[b]) // page))] = n_pages + b
    k, v = torch.zeros(B, 1, heads, d, dtype=BF, device="cuda"), torch.zeros(B, 1, heads, d, dtype=BF, device="cuda")
    q, after = torch.zeros(B, 1, 4, d, dtype=BF, device="cuda"), held + 1

    def step():
        lib.df_cache_append(k, v, bigger, table, held)
        return lib.df_cache_attn(q, bigger, table, after, max_length=64)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    g = torch.Generator().manual_seed(11)
    for _ in range(10):
        n, *new = [1] * B, *(torch.randn(B, heads, d, generator=g).to(BF) for _ in range(2))
        calls.append((n, *new))
        for t, x in zip((k, v), new):
            t.copy_(x.view(B, 1, heads, d))
        x = torch.randn(B, 1, 4, d, generator=g).to(BF)
        q.copy_(x)
        graph.replay()
        lens = [int(i) for i in after.tolist()]
        w = want_attn(np64(x).reshape(-1, 4, d), lens, [1] * B, oracles(calls, heads, d), True, 0, 0, d ** -0.5)
        check_forward(out.view(-1, 4, d), w, BF, d)
        held.add_(1)
        after.add_(1)


def test_offsets_beyond_32_bits(lib):
    """Pages that lie behind the first 4 GB of the cache."""
    heads, d, page, n_pages = 16, 128, 1 << 16, 20  # 269 MB a page
    cache = lib.df_cache_new(n_pages, heads, page, d)
    assert cache.numel() > 2 ** 32
    calls = tokens([[50]], heads, d, BF, seed=12)
    n, k, v = calls[0]
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    zero, held = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([50], dtype=torch.int32, device="cuda")
    lib.df_cache_append(k.cuda(), v.cuda(), cache, table, zero, offsets(n).cuda())
    got, _ = lib.df_cache_read(cache, table, held, rows=50, dtype=F32)
    both = oracles(calls, heads, d)
    assert np.array_equal(np64(got[0]), both[0][0].values())
    q = torch.randn(1, 1, heads, d).to(BF)
    w = want_attn(np64(q)[0], [50], [1], both, True, 0, 0, d ** -0.5)
    check_forward(lib.df_cache_attn(q.cuda(), cache, table, held, max_length=50)[0], w, BF, d)
