"""The layers hand a status word on to the calls that report into it: ids outside the
vocabulary and bad offsets must not pass in silence.  Without a GPU: the binding's calls
are replaced by ones that record what they are given."""

import pytest
import torch


@pytest.fixture
def layers(monkeypatch):
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding, encoder
    got = {}

    def record(name, give):
        def call(*args, **kw):
            got.setdefault(name, []).append(kw.get("status"))
            return give(*args, **kw)
        monkeypatch.setattr(binding, name, call)

    record("df_embedding", lambda ids, table, **kw: torch.zeros(ids.numel(), table.shape[1]))
    record("df_linear", lambda x, w, *a, **kw: [torch.zeros(x.shape[0], w[0].shape[0]) for _ in w])
    record("df_cross_attn_fwd", lambda q, k, v, **kw: torch.zeros_like(q))
    monkeypatch.setattr(binding, "df_layernorm", lambda x, *a, **kw: x)
    cfg = encoder.EncoderConfig(hidden=256, heads=4, layers=0, vocab=9)
    enc = encoder.Encoder(cfg, [], encoder.synthetic_weights(cfg, device="cpu")[1])
    return enc, encoder.CrossAttention(cfg, encoder.synthetic_cross_weights(cfg, device="cpu")), got


def test_status_reaches_the_calls(layers):
    enc, cross, got = layers
    word, cu = torch.zeros(1, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32)
    x = enc.embed(torch.zeros(3, dtype=torch.int64), status=word)
    k, v = cross.project(x, status=word)
    cross.attend(x, k, v, cu, 3, cu, 3, status=word)
    assert {n: len(s) for n, s in got.items()} == {"df_embedding": 1, "df_linear": 3, "df_cross_attn_fwd": 1}
    assert all(s is word for calls in got.values() for s in calls)
