"""Queries and values at the ends of their types' ranges, attended to and read back."""

import numpy as np
import pytest
import torch

from _cache import fill, oracles, tokens
from _cross import U32, check_forward, np64
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


@pytest.mark.parametrize("B,H,Hk,d,Lq", [(2, 4, 2, 64, 1), (1, 8, 8, 32, 1), (2, 16, 2, 128, 3)])
@pytest.mark.parametrize("below", [17, 20, 23])
def test_small_digits_of_a_query_beside_a_large_one(lib, B, H, Hk, d, Lq, below):
    """A column that is 2^below of the others and whose keys are 0: the scores are the others', with all
    digits of theirs."""
    lens = [120, 50][:B]
    calls = []
    for n, k, v in tokens([lens], Hk, d, BF, seed=below):
        k = k.float() * 2.0 ** 6
        k[..., 0] = 0
        calls.append((n, k.to(BF), v))
    q = torch.randn(B, Lq, H, d, generator=torch.Generator().manual_seed(below)) * 2.0 ** -6
    q[..., 0] = 2.0 ** (below - 6)
    out, lse, w = attend(lib, calls, q.to(BF), Hk, d)
    check_forward(out, w, BF, d, lse)


@pytest.mark.parametrize("e", [-132, -126, -118, -110, -95, -94, -93, 0, 95])
def test_queries_of_any_exponent(lib, e):
    """bf16 queries from subnormal ones to where their keys are subnormal codes, scores of some 1."""
    d = 64
    up = min(max(-e, -97), 120)
    calls = [(n, (k.float() * 2.0 ** up).to(BF), v) for n, k, v in tokens([[90, 33]], 2, d, BF, seed=3)]
    q = (torch.randn(2, 2, 4, d, generator=torch.Generator().manual_seed(9)) * 2.0 ** e).to(BF)
    out, lse, w = attend(lib, calls, q, 2, d)
    check_forward(out, w, BF, d, lse)


def test_the_largest_query_of_all(lib):
    """The column of the type's largest value meets keys of 0."""
    d = 64
    (n, k, v), = tokens([[90]], 2, d, BF, seed=4)
    k = k.float() * 2.0 ** -96
    k[..., 5] = 0
    q = torch.randn(1, 1, 4, d, generator=torch.Generator().manual_seed(10)) * 2.0 ** 97
    q[..., 5] = torch.finfo(BF).max
    out, lse, w = attend(lib, [(n, k.to(BF), v)], q.to(BF), 2, d)
    # Columns around 2^-30 of the largest have some that lie below 2^-32 of it.  Those are off by half of fp16's
    # smallest step, 2^-25, where the largest is 2^15 at least, 2^-40 of it; a score by that many times the sum
    # of its key's columns, scaled; a weight by twice that (its own score, and the row's sum).
    off = d ** -0.5 * 2.0 ** -40 * float(torch.finfo(BF).max) * float(k.to(BF).double().abs().sum(-1).max()) * (1 + 2.0 ** -4)
    w["score_mass"] = w["score_mass"] + off / ((d + 4) * U32)  # (of which score_error takes 2 (d + 4) roundings)
    check_forward(out, w, BF, d, lse)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_finite_values_stay_finite(lib, dtype):
    """The largest values of the type: held, read back in every type and attended to."""
    d, top = 32, float(torch.finfo(dtype).max)
    v = torch.zeros(4, 1, d)
    v[0], v[1], v[2, 0, :8], v[3] = top, -top, top, top * torch.linspace(0.8, 1, d)
    v = v.to(dtype)
    calls = [([1], torch.zeros_like(v[:1]), v[i:i + 1]) for i in range(4)]
    cache, table, held = fill(lib, calls, 1, d, 16)
    want = oracles(calls, 1, d)[0][1].values()
    half = 2.0 ** -4  # of e4m3
    assert np.isfinite(want).all() and (np.abs(want - np64(v)) <= half * np.abs(np64(v))).all()
    for t in (F32, BF, HF):
        _, got = lib.df_cache_read(cache, table, held, rows=4, dtype=t)
        assert np.array_equal(np64(got[0]), np.clip(want, -65504, 65504) if t == HF else want)
    for i in range(4):
        # a window of one token: its values themselves
        out = lib.df_cache_attn(torch.ones(1, 1, 1, d, dtype=dtype, device="cuda"), cache, table,
                                torch.full_like(held, i + 1), window=1)
        got, ref = np64(out[0, 0, 0]), want[i, 0]
        ref = np.clip(ref, -65504, 65504) if dtype == HF else ref
        assert np.isfinite(got).all() and (np.abs(got - ref) <= torch.finfo(dtype).eps * np.abs(ref)).all()


@pytest.mark.parametrize("brought", [HF, BF])
def test_results_in_fp16_are_those_that_reading_back_gives(lib, brought):
    """fp16 results of held values beyond its range (65504 itself is held as 65536): +-65504, as they are read
    back; NaN stays NaN."""
    d = 32
    v = torch.zeros(5, 1, d)
    v[0, 0, :3] = torch.tensor([65504.0, -65504.0, 64000.0])
    v[1], v[2, 0, 4], v[3] = 65504.0, float("nan"), 1.0
    v[4] = torch.linspace(-1, 1, d) * (1e6 if brought == BF else 65504.0)
    calls = [([5], torch.zeros(5, 1, d, dtype=brought), v.to(brought))]
    cache, table, held = fill(lib, calls, 1, d, 16)
    read = np64(lib.df_cache_read(cache, table, held, rows=5, dtype=HF)[1])[0, :, 0]
    q = torch.ones(1, 1, 1, d, dtype=HF, device="cuda")
    for i in range(5):
        # a window of one token: its values themselves (the sum's reciprocal is an approximation: a step)
        got = np64(lib.df_cache_attn(q, cache, table, torch.full_like(held, i + 1), window=1))[0, 0, 0]
        nan = np.isnan(read[i])
        assert np.array_equal(np.isnan(got), nan) and np.isfinite(got[~nan]).all()
        assert (np.abs(got - read[i])[~nan] <= torch.finfo(HF).eps * np.abs(read[i][~nan])).all()
    # the mean of two that are held as 65536
    out = lib.df_cache_attn(q, cache, table, torch.full_like(held, 2), window=2)
    assert float(out[0, 0, 0, 0]) == 65504.0


def test_scores_beyond_the_range_are_not_a_number(lib):
    """+infinity among the scores that a query sees: NaN, also where the parts of a sequence are joined;
    -infinity is a weight of 0."""
    d, top = 32, float(torch.finfo(BF).max)
    x = torch.zeros(4, 1, d)
    x[0], x[1], x[2, 0, :8], x[3] = top, -top, top, top * torch.linspace(0.8, 1, d)
    x = x.to(BF)
    cache, table, held = fill(lib, [([1], x[i:i + 1], x[i:i + 1]) for i in range(4)], 1, d, 16)
    q, lse = torch.ones(1, 1, 1, d, dtype=BF, device="cuda"), torch.zeros(1, 1, 1, device="cuda")
    for i in range(4):
        out = lib.df_cache_attn(q, cache, table, torch.full_like(held, i + 1), window=1, lse=lse)
        if i == 1:
            assert bool((out == 0).all()) and float(lse) == float("-inf")
        else:
            assert bool(out.isnan().all()) and bool(lse.isnan().all())
    k, v = torch.zeros(3000, 1, d), torch.ones(3000, 1, d)
    k[1234] = top
    cache, table, held = fill(lib, [([3000], k.to(BF), v.to(BF))], 1, d, 16)
    both = torch.cat([q, -q], 2)
    for bound in (1, 3000):
        out = lib.df_cache_attn(both, cache, table, held, max_length=bound)[0, 0]
        assert bool(out[0].isnan().all()) and bool((out[1] == 1).all())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_token_that_is_not_a_number_leaves_its_block_alone(lib, dtype):
    """NaN and infinities appended behind 35 tokens: those are read and attended to as before, bit for bit."""
    d = 64
    calls = tokens([[35]], 2, d, dtype, seed=13)
    cache, table, held = fill(lib, calls, 2, d, 32, spare_pages=1)
    q = torch.randn(1, 1, 4, d, generator=torch.Generator().manual_seed(14)).to(dtype).cuda()
    before, rows = lib.df_cache_attn(q, cache, table, held), lib.df_cache_read(cache, table, held, rows=35)
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = torch.full((1, 1, 2, d), value, dtype=dtype, device="cuda")
        lib.df_cache_append(bad, bad, cache, table, held)
        assert torch.equal(lib.df_cache_attn(q, cache, table, held), before)
        assert all(torch.equal(a, b) for a, b in zip(lib.df_cache_read(cache, table, held, rows=35), rows))
        assert bool(lib.df_cache_attn(q, cache, table, held + 1).isnan().all())
        assert bool(lib.df_cache_read(cache, table, held + 1, rows=36)[0][:, 35].isnan().all())
