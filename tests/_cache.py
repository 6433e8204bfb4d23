"""Caches of the tests: random tokens, appended in parts through the library and to the oracle."""

import numpy as np
import torch

import oracle


def table_of(lengths, page, n_pages, seed, spare=0):
    """A page table in no order; entries behind the last page are -1."""
    need = [-(-n // page) for n in lengths]
    order = np.random.default_rng(seed).permutation(n_pages)[:sum(need)]
    table = np.full((len(lengths), max(max(need), 1) + spare), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table)


def tokens(parts, heads, d, dtype, seed, sigma=1.0):
    """Keys and values of each call: a list of (lengths, k, v) with packed rows."""
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(0.7 * torch.randn(2, heads, d, generator=g)) * sigma
    out = []
    for n in parts:
        both = [(torch.randn(sum(n), heads, d, generator=g) * size[i]).to(dtype) for i in range(2)]
        out.append((list(n), *both))
    return out


def offsets(n):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)


def oracles(calls, heads, d):
    """(keys, values) oracle of each sequence after the calls."""
    B = len(calls[0][0])
    both = [(oracle.CacheOracle(heads, d), oracle.CacheOracle(heads, d)) for _ in range(B)]
    for n, k, v in calls:
        at = np.concatenate([[0], np.cumsum(n)])
        for b in range(B):
            for o, x in zip(both[b], (k, v)):
                o.append(x[at[b]:at[b + 1]].double().numpy())
    return both


def fill(lib, calls, heads, d, page, seed=0, spare_pages=2, **more):
    """The cache after the calls: (cache, table, lengths) on the GPU."""
    total = np.sum([c[0] for c in calls], axis=0)
    n_pages = int(sum(-(-int(n) // page) for n in total)) + spare_pages
    cache = lib.df_cache_new(n_pages, heads, page, d)
    cache.fill_(0xFF)  # NaN codes and NaN scales where nothing is written
    table = table_of([int(n) for n in total], page, n_pages, seed).cuda()
    held = np.zeros(len(total), np.int64)
    for n, k, v in calls:
        lib.df_cache_append(k.cuda(), v.cuda(), cache, table, torch.tensor(held, dtype=torch.int32).cuda(),
                            offsets(n).cuda(), **more)
        held += np.asarray(n)
    return cache, table, torch.tensor(held, dtype=torch.int32).cuda()
