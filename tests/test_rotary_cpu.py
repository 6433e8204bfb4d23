"""Rotary positions without a GPU: the oracle, the table of frequencies (a host function), and
the host refusals."""

import ctypes
import math

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


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(factor=4.0),
                                dict(factor=8.0, original_len=8192.0, low=1.0, high=4.0),
                                dict(factor=2.5, original_len=4096.0), dict(base=0.5)])
@pytest.mark.parametrize("rot", [2, 20, 64, 128])
def test_table_holds_the_frequencies(binding, rot, kw):
    table = binding.df_rotary_table(rot, device="cpu", **kw)
    assert table.dtype == torch.int64 and table.shape == (rot // 2,)
    for got, f in zip(table.tolist(), oracle.rotary_frequencies(rot, **kw)):
        turn = f / (2 * math.pi) % 1.0
        off = abs((got % 2 ** 64) / 2 ** 64 - turn)
        # the power, the product and the quotient round (53 digits)
        assert min(off, 1 - off) <= 8 * 2.0 ** -53 * f / (2 * math.pi) + 2.0 ** -64


def test_oracle_rotates_by_complex_numbers():
    rng = np.random.default_rng(0)
    x, angles = rng.standard_normal((3, 2, 10)), rng.standard_normal((3, 4))
    for inter in (False, True):
        y, _ = oracle.rotary(x, angles, inter, amplitude=1.5)
        a, b = (slice(0, 8, 2), slice(1, 8, 2)) if inter else (slice(0, 4), slice(4, 8))
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angles)[:, None] * 1.5
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag) and (y[..., 8:] == x[..., 8:]).all()
        back, _ = oracle.rotary(y, angles, inter, inverse=True, amplitude=1 / 1.5)
        assert np.allclose(back, x)


def _call(b, **over):
    a = dict(x=(0x100000, 0x200000), heads=(4, 2), xs=(256, 128), out=(0x300000, 0x400000), os=(256, 128),
             pos=0x500000, pos_64=0, T=5, d=64, rot=64, turns=0x600000, amp=1.0, dtype=0)
    a.update(over)
    p = lambda n: None if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    rows = [v for i in range(2) for v in (a["x"][i], a["heads"][i], a["xs"][i], a["out"][i], a["os"][i])]
    return b.raw_library.df_rotary(*rows, p("pos"), a["pos_64"], a["T"], a["d"], a["rot"], 0, 0, p("turns"), a["amp"],
                                   a["dtype"], None)


REFUSED = [
    (dict(T=-1), 1), (dict(heads=(4, -1)), 1), (dict(rot=0), 1), (dict(rot=63), 1), (dict(rot=66), 1),
    (dict(pos=None), 1), (dict(turns=None), 1), (dict(x=(None, 0x200000)), 1), (dict(out=(0x300000, None)), 1),
    (dict(heads=(0, 2)), 1), (dict(xs=(255, 128)), 1), (dict(os=(256, 127)), 1), (dict(xs=(256, -128)), 1),
    (dict(amp=float("nan")), 1), (dict(amp=float("inf")), 1), (dict(dtype=3), 1), (dict(pos=0x500002), 3),
    (dict(pos=0x500004, pos_64=1), 3), (dict(turns=0x600004), 3), (dict(x=(0x100001, 0x200000)), 3),
    # results over another input, over one another, over the positions; a shifted input
    (dict(out=(0x200000, 0x400000)), 1), (dict(out=(0x300000, 0x300100)), 1), (dict(out=(0x4fffc0, 0x400000)), 1),
    (dict(out=(0x100010, 0x400000)), 1), (dict(out=(0x100000, 0x400000), os=(512, 128)), 1)]


@pytest.mark.parametrize("over,status", REFUSED)
def test_refused_on_the_host(binding, over, status):
    assert _call(binding, **over) == status, over


def test_nothing_to_do(binding):
    assert _call(binding, T=0, pos=None, turns=None) == binding.DF_OK


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(base=0.0), dict(base=float("inf")), dict(factor=0.0),
                                dict(original_len=-1.0), dict(original_len=10.0, low=2.0, high=2.0)])
def test_table_refuses(binding, kw):
    with pytest.raises(binding.DFError):
        binding.df_rotary_table(**{"rot": 64, "device": "cpu", **kw})


def test_binding_refuses(binding):
    b = binding
    table = b.df_rotary_table(64, device="cpu")
    x, pos = torch.zeros(5, 4, 64), torch.zeros(5, dtype=torch.int32)
    bad = [((x, pos.float(), table), "positions"), ((x, pos[:4], table), "positions"), ((x, pos, table.int()), "table"),
           ((x.double(), pos, table), "bf16"), (((x, x, x), pos, table), "one tensor or two"),
           (((x, x[:4]), pos, table), "share"), ((x, pos, table), "CUDA")]
    for args, text in bad:
        with pytest.raises(ValueError, match=text):
            b.df_rotary(*args)
    with pytest.raises(ValueError, match="next to one another"):
        b._decoder._token_stride("x", torch.zeros(5, 64, 4).transpose(1, 2), 1)
    with pytest.raises(ValueError, match="constant distance"):
        b._decoder._token_stride("x", torch.zeros(5, 3, 4, 64)[:, :2], 2)
    assert b._decoder._token_stride("x", torch.zeros(5, 3, 12, 64)[:, :, 4:8], 2) == 12 * 64
    assert b._decoder._token_stride("x", torch.zeros(1, 3, 4, 64)[:, ::2], 2) == 2 * 4 * 64
