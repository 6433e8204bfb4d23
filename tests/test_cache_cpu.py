"""The 8-bit cache without a GPU: the oracle by its own definition, and the host refusals."""

import ctypes

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def binding():
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding as b
    return b


def test_codes_are_those_of_torch():
    assert np.array_equal(oracle.E4M3[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy())
    x = torch.cat([torch.randn(20000, generator=torch.Generator().manual_seed(0)) * s for s in (1e-3, 0.01, 1, 100)])
    x = torch.cat([x, torch.arange(0, 449) / 2.0 ** 10, torch.arange(0, 449).float()]).clamp(-448, 448).to(torch.bfloat16)
    x = torch.cat([x, -x]).float()
    assert np.array_equal(oracle.e4m3_codes(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scale_is_the_least_power_of_two():
    for top in (448.0, 448.5, 1.0, 0.875, 0.8751, 3e38, 1e-30, 2.0 ** -126):
        s = oracle.block_scale([top, -top / 2, np.nan, np.inf])
        assert top <= 448 * s and (top > 448 * s / 2 or s == 2.0 ** -100)
    assert oracle.block_scale(np.zeros(4)) == 2.0 ** -100


def test_appending_in_parts_rounds_no_worse_than_twice():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((45, 2, 32)) * np.exp(rng.standard_normal((45, 1, 1)))
    whole, parts = oracle.CacheOracle(2, 32).append(x), oracle.CacheOracle(2, 32)
    at = 0
    for n in (3, 1, 20, 0, 1, 20):
        parts.append(x[at:at + n])
        at += n
    a, b = whole.values(), parts.values()
    assert a.shape == x.shape and np.array_equal(whole.scale, parts.scale)
    step = whole.scale[np.arange(45) // 16][:, :, None] * 2.0 ** -9
    assert (np.abs(a - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step / 2)).all()
    assert (np.abs(b - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step)).all()


P = dict(cache=0x1000000, pages=0x20000, lengths=0x30000)


def _append(b, **over):
    a = dict(P, k=0x100000, v=0x200000, cu=None, B=2, Hk=3, n=5, total=10, d=64, dtype=0, n_pages=4, page=32, max_pages=2)
    a.update(over)
    p = lambda n: None if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    return b.raw_library.df_cache_append(p("k"), p("v"), p("cu"), a["B"], a["Hk"], a["n"], a["total"], a["d"], a["dtype"],
                                         p("cache"), a["n_pages"], a["page"], p("pages"), a["max_pages"], p("lengths"), None,
                                         None)


def _read(b, **over):
    a = dict(P, k=0x100000, v=0x200000, cu=None, B=2, Hk=3, n=5, total=10, d=64, dtype=0, n_pages=4, page=32, max_pages=2)
    a.update(over)
    p = lambda n: None if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    return b.raw_library.df_cache_read(p("cache"), a["n_pages"], a["page"], p("pages"), a["max_pages"], p("lengths"),
                                       p("cu"), a["B"], a["Hk"], a["n"], a["total"], a["d"], a["dtype"], p("k"), p("v"), None,
                                       None)


def _attn(b, **over):
    a = dict(P, q=0x100000, cu=None, B=2, H=6, Hk=3, Lq=5, total=10, d=64, scale=0.125, causal=1, window=0, sinks=0, dtype=0,
             n_pages=4, page=32, max_pages=2, max_length=64, out=0x200000, lse=None)
    a.update(over)
    p = lambda n: None if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    return b.raw_library.df_cache_attn(p("q"), p("cu"), a["B"], a["H"], a["Hk"], a["Lq"], a["total"], a["d"], a["scale"],
                                       a["causal"], a["window"], a["sinks"], a["dtype"], p("cache"), a["n_pages"], a["page"],
                                       p("pages"), a["max_pages"], p("lengths"), a["max_length"], p("out"), p("lse"), None,
                                       None)


SHARED = [  # arguments, status
    (dict(B=-1), 1), (dict(Hk=0), 1), (dict(d=0), 1), (dict(page=0), 1), (dict(n_pages=-1), 1), (dict(max_pages=-1), 1),
    (dict(total=11), 1), (dict(dtype=3), 1), (dict(cache=None), 1), (dict(pages=None), 1), (dict(lengths=None), 1),
    (dict(d=48), 2), (dict(d=160), 2), (dict(page=24), 2), (dict(max_pages=1 << 26), 2), (dict(cache=0x1000008), 3),
    (dict(pages=0x20002), 3), (dict(lengths=0x30001), 3), (dict(cu=0x40002, total=10), 3)]


@pytest.mark.parametrize("over,status", SHARED)
def test_entry_points_refuse_on_the_host(binding, over, status):
    for call in (_append, _read, _attn):
        assert call(binding, **over) == status, (call.__name__, over)


def test_each_call_refuses_its_own(binding):
    b = binding
    for call in (_append, _read):
        assert call(b, k=None) == b.DF_ERR_INVALID_ARG and call(b, v=None) == b.DF_ERR_INVALID_ARG
        assert call(b, k=0x100008) == b.DF_ERR_ALIGNMENT and call(b, n=-1) == b.DF_ERR_INVALID_ARG
        assert call(b, k=0x1000000) == b.DF_ERR_INVALID_ARG  # over the cache
        assert call(b, n=0, total=0, k=None, v=None) == b.DF_OK  # nothing to do
    assert _append(b, dtype=2) == b.DF_ERR_UNSUPPORTED
    assert _read(b, v=0x100010) == b.DF_ERR_INVALID_ARG  # over one another
    assert _append(b, pages=0x1000010) == b.DF_ERR_INVALID_ARG
    bad = [dict(H=7), dict(H=0), dict(Lq=-1), dict(max_length=-1), dict(scale=0.0), dict(scale=float("nan")),
           dict(window=-1), dict(sinks=-1), dict(causal=0, window=4), dict(q=None), dict(out=None), dict(out=0x100000),
           dict(lse=0x200000), dict(out=0x1000000)]
    for over in bad:
        assert _attn(b, **over) == b.DF_ERR_INVALID_ARG, over
    assert _attn(b, dtype=2) == b.DF_ERR_UNSUPPORTED and _attn(b, H=258, Hk=2) == b.DF_ERR_UNSUPPORTED
    assert _attn(b, lse=0x50002) == b.DF_ERR_ALIGNMENT and _attn(b, q=0x100008) == b.DF_ERR_ALIGNMENT
    assert _attn(b, Lq=0, total=0, q=None, out=None) == b.DF_OK


def test_bytes(binding):
    size = binding.raw_library.df_cache_bytes
    assert size(7, 3, 48, 96) == 7 * 3 * 3 * (32 * 96 + 16) and size(1, 1, 24, 64) == 0 and size(0, 1, 16, 64) == 0
    assert size(1 << 20, 64, 16, 128) == (1 << 26) * 4112  # beyond 32 bits


def test_binding_refuses(binding):
    b = binding
    cache = b.df_cache_new(4, 3, 32, 64, device="cpu")
    assert cache.shape == (4, 3, 2, 32 * 64 + 16) and cache.dtype == torch.uint8
    table, held, k = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 5, 3, 64)
    k = k.to(torch.bfloat16)
    for args in ((4, 3, 24, 64), (4, 3, 32, 40), (4, 0, 32, 64)):
        with pytest.raises(ValueError):
            b.df_cache_new(*args, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        b.df_cache_append(k, k, cache, table, held)
    shape = b._decoder._cache_shape
    assert shape(cache, table, held) == (2, 3, 64, 4, 32, 2)
    for bad in ((cache.float(), table, held), (cache[0], table, held), (cache[..., :-1], table, held),
                (cache, table.long(), held), (cache, table[0], held), (cache, table, held[:1]), (cache, table, held.long())):
        with pytest.raises(ValueError):
            shape(*bad)
    rows = b._decoder._cache_rows
    assert rows("k", k, None, 2) == (5, 10) and rows("k", k[0], held.new_zeros(3), 2) == (0, 5)
    for x, cu in ((k[0], None), (k, held.new_zeros(3)), (k[0], held), (k[:1], None)):
        with pytest.raises(ValueError):
            rows("k", x, cu, 2)
