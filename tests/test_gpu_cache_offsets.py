"""Packed rows of the 8-bit cache's calls whose offsets do not begin at 0, or cannot be: nothing in
front of the first sequence, before the tensors or behind them is touched."""

import numpy as np
import pytest
import torch

from _cache import fill, offsets, oracles, tokens
from _cross import np64

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
GUARD = 12000  # rows of 7 on either side: more than any offset of these tests


def word(lib):
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def guarded(rows, heads, d, dtype):
    """(all rows, the `rows` in their middle), all 7."""
    every = torch.full((2 * GUARD + rows, heads, d), 7.0, dtype=dtype, device="cuda")
    return every, every[GUARD:GUARD + rows]


@pytest.mark.parametrize("first", [1, 15, 16, 17, 1000])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_read_leaves_the_rows_in_front_of_the_first_sequence(lib, first, dtype):
    heads, d, lens, behind = 2, 64, [37, 0, 130], 40
    calls = tokens([lens], heads, d, BF, seed=first)
    cache, table, held = fill(lib, calls, heads, d, 32)
    want = oracles(calls, heads, d)
    # the last sequence has more rows here than it holds
    n = [37, 0, 140]
    rows, status = first + sum(n) + behind, word(lib)
    cu = offsets(n).cuda() + first
    (every_k, k), (every_v, v) = guarded(rows, heads, d, dtype), guarded(rows, heads, d, dtype)
    lib.df_cache_read(cache, table, held, cu, out=(k, v), status=status)
    assert int(status.item()) == lib.DF_OK
    for i, (every, x) in enumerate(((every_k, k), (every_v, v))):
        assert bool((every[:GUARD + first] == 7).all()) and bool((every[GUARD + rows:] == 7).all())
        ref = np.concatenate([o[i].values() for o in want])
        at = first + 37 + 130
        assert np.array_equal(np64(x[first:at]), np64(torch.from_numpy(ref).to(dtype)))
        assert bool((x[at:] == 0).all())


@pytest.mark.parametrize("cu,rows,zeros", [  # zeros: from this row on (those behind the last sequence)
    ([10000, 10000], 100, 100), ([121, 80], 120, 80), ([121, 121], 120, 120), ([-1, 40], 120, 40), ([120, 50], 120, 50),
    ([2 ** 31 - 1, 2 ** 31 - 1], 120, 120), ([2 ** 31 - 1, -2 ** 31], 120, 0), ([-2 ** 31, 2 ** 31 - 1], 120, 120)])
def test_read_stays_within_its_rows_whatever_the_offsets(lib, cu, rows, zeros):
    heads, d = 2, 64
    calls = tokens([[50]], heads, d, BF, seed=rows)
    cache, table, held = fill(lib, calls, heads, d, 16)
    status = word(lib)
    (every_k, k), (every_v, v) = guarded(rows, heads, d, BF), guarded(rows, heads, d, BF)
    lib.df_cache_read(cache, table, held, ints(*cu), out=(k, v), status=status)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG
    for every, x in ((every_k, k), (every_v, v)):
        assert bool((every[:GUARD] == 7).all()) and bool((every[GUARD + rows:] == 7).all())
        assert bool((x[:zeros] == 7).all()) and bool((x[zeros:] == 0).all())


def with_rows_in_front(x, first):
    return torch.cat([torch.full((first, *x.shape[1:]), float("nan"), dtype=x.dtype), x]).cuda()


@pytest.mark.parametrize("first", [1, 16, 40, 1000])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_looks_at_pages_of_its_own_tokens_only(lib, first, dtype):
    """Rows in front of the first sequence are nobody's, and a page that a window has left behind may
    be gone from the table."""
    heads, d, page = 2, 64, 16
    calls = tokens([[600, 0, 70], [5, 0, 33]], heads, d, dtype, seed=first)
    cache, table, held = fill(lib, calls, heads, d, page)
    old = ints(600, 0, 70)
    # (the same pages: those of the whole, filled by the first call only)
    part = lib.df_cache_new(cache.shape[0], heads, page, d).fill_(0xFF)
    n, k, v = calls[0]
    lib.df_cache_append(k.cuda(), v.cuda(), part, table, torch.zeros_like(old), offsets(n).cuda())
    gone = table.clone()
    gone[0, :600 // page], gone[2, :70 // page] = -1, -1
    n, k, v = calls[1]
    status = word(lib)
    lib.df_cache_append(with_rows_in_front(k, first), with_rows_in_front(v, first), part, gone, old,
                        offsets(n).cuda() + first, status=status)
    assert int(status.item()) == lib.DF_OK and torch.equal(part, cache)


@pytest.mark.parametrize("first", [16, 64, 200])
def test_append_leaves_pages_that_are_another_sequences_by_now(lib, first):
    """The table of the first sequence still names, for tokens long gone, the page to which the second
    one appends in the same call, with values that raise its scale."""
    heads, d, B = 4, 64, 2
    g = torch.Generator().manual_seed(first)
    rows = lambda n, s: (torch.randn(n, heads, d, generator=g) * s).to(BF)  # noqa: E731
    old_k, old_v, k, v = rows(5, 1.0), rows(5, 1.0), rows(9, 300.0), rows(9, 300.0)
    held, n = ints(64, 5), [3, 6]
    stale, clean = ints(0, 0, 0, 0, 1, 0, -1, -1, -1, -1).view(B, 5), ints(-1, -1, -1, -1, 1, 0, -1, -1, -1, -1).view(B, 5)
    cache = lib.df_cache_new(2, heads, 16, d).fill_(0)
    lib.df_cache_append(old_k.cuda(), old_v.cuda(), cache, clean, ints(0, 0), offsets([0, 5]).cuda())
    want = cache.clone()
    lib.df_cache_append(k.cuda(), v.cuda(), want, clean, held, offsets(n).cuda())
    assert not torch.equal(want, cache)
    for _ in range(20):
        got, status = cache.clone(), word(lib)
        lib.df_cache_append(with_rows_in_front(k, first), with_rows_in_front(v, first), got, stale, held,
                            offsets(n).cuda() + first, status=status)
        assert int(status.item()) == lib.DF_OK and torch.equal(got, want)
