"""The decoder's calls and layers with a stream as argument: everything that they allocate
belongs to that stream (see test_streams_cpu.py, whose stand-ins these tests use)."""

import inspect

import pytest
import torch

from test_streams_cpu import dev, record  # noqa: F401 (the fixture)


def calls(b, e):
    q, cu = dev(6, 8, 64), dev(3, dtype=torch.int32)
    paged = dev(4, 8, 2, 32 * 64 + 16, dtype=torch.uint8), dev(2, 2, dtype=torch.int32), dev(2, dtype=torch.int32)
    at = dict(cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=4, max_seqlen_k=4, window=3, sinks=1)
    cfg = e.EncoderConfig(hidden=512, heads=8, layers=1, ffn=512)
    put = lambda w: {n: dev(*t.shape) for n, t in w.items()}  # noqa: E731
    own = e.SelfAttention(cfg, put(e.synthetic_self_weights(cfg, 4, device="cpu")), dev(32, dtype=torch.int64), key_heads=4)
    cross = e.CrossAttention(cfg, put(e.synthetic_cross_weights(cfg, device="cpu")))
    x, pos, x2, pos2 = dev(6, 512), dev(6, dtype=torch.int32), dev(2, 1, 512), dev(2, 1, dtype=torch.int32)
    small = dev(4, 4, 2, 32 * 64 + 16, dtype=torch.uint8), *paged[1:]
    return {
        "SelfAttention.prompt": lambda **s: own.prompt(x, pos, cu, 4, *small[:2], **s),
        "SelfAttention.step": lambda **s: own.step(x2, pos2, *small, **s),
        "CrossAttention.store": lambda **s: cross.store(x, *paged[:2], cu, **s),
        "CrossAttention.attend_stored": lambda **s: cross.attend_stored(dev(2, 512), *paged, **s),
        "df_self_attn_fwd": lambda **s: b.df_self_attn_fwd(q, q, q, with_stats=True, **at, **s),
        "df_self_attn_bwd": lambda **s: b.df_self_attn_bwd(q, q, q, q, b.CrossStats(dev(6, 8, dtype=torch.float32), q), q,
                                                           **at, **s),
        "df_rotary": lambda **s: b.df_rotary((q, q), dev(6, dtype=torch.int32), dev(32, dtype=torch.int64), **s),
        "df_cache_read": lambda **s: b.df_cache_read(*paged, rows=9, **s),
        "df_cache_attn": lambda **s: b.df_cache_attn(q, *paged, cu, max_seqlen_q=3, **s),
    }


NAMES = ["df_self_attn_fwd", "df_self_attn_bwd", "df_rotary", "df_cache_read", "df_cache_attn", "SelfAttention.prompt",
         "SelfAttention.step", "CrossAttention.store", "CrossAttention.attend_stored"]
NOTHING = {"df_cache_append"}  # allocates nothing


@pytest.fixture
def recorded(record, monkeypatch):  # noqa: F811
    b, e, seen = record
    from exact_attention_deberta_gb300 import decoder_binding
    if hasattr(decoder_binding, "torch"):
        monkeypatch.setattr(decoder_binding, "torch", b.torch)
    return b, e, seen


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream_given(recorded, name):
    b, e, seen = recorded
    call = calls(b, e)[name]
    seen.clear()
    call(stream=1234)
    assert seen and set(seen) == {1234}, seen


def test_every_call_with_a_stream_is_listed(recorded):
    from exact_attention_deberta_gb300 import decoder_binding as d
    takes = {n for n, f in vars(d).items() if inspect.isfunction(f) and not n.startswith("_") and
             "stream" in inspect.signature(f).parameters}
    assert takes - NOTHING <= set(NAMES)


def test_calls_are_reached_through_the_binding():
    from exact_attention_deberta_gb300 import binding, decoder_binding
    for name in decoder_binding.__all__:
        assert getattr(binding, name) is getattr(decoder_binding, name)
    with pytest.raises(AttributeError):
        binding.df_no_such_call
