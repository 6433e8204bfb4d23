"""The SelfAttention layer with frequencies that are stretched for long contexts."""

import numpy as np
import pytest
import torch

import oracle
from _cache import offsets
from _cross import np64

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("amplitude,interleaved", [(1.0, False), (0.1 * np.log(4.0) + 1.0, False), (1.25, True)])
def test_rows_are_rotated_with_the_amplitude(lib, amplitude, interleaved):
    """The queries and keys of a prompt and of a step, and the keys that the cache holds."""
    from exact_attention_deberta_gb300 import encoder
    heads, d, n = 8, 64, 90
    cfg = encoder.EncoderConfig(hidden=heads * d, heads=heads)
    w = encoder.synthetic_self_weights(cfg, 4, seed=3)
    turns = lib.df_rotary_table(d, factor=4.0, original_len=4096.0)
    layer = encoder.SelfAttention(cfg, w, turns, key_heads=4, interleaved=interleaved, amplitude=amplitude)
    x = torch.randn(n + 1, cfg.hidden, generator=torch.Generator().manual_seed(4)).to(BF).cuda()
    pos = torch.arange(n + 1, dtype=torch.int32, device="cuda") + 9000
    cache, table = lib.df_cache_new(6, 4, 16, d), torch.arange(6, dtype=torch.int32, device="cuda").view(1, 6)
    prompt, step = [], []
    layer.prompt(x[:n], pos[:n], offsets([n]).cuda(), n, cache, table, trace=prompt)
    layer.step(x[n:].view(1, 1, -1), pos[n:].view(1, 1), cache, table,
               torch.tensor([n], dtype=torch.int32, device="cuda"), trace=step)
    angles = oracle.rotary_angles(pos.tolist(), turns.tolist())
    for t, rows in ((prompt[0], slice(0, n)), (step[0], slice(n, n + 1))):
        for name, h in (("q", heads), ("k", 4)):
            (plain,) = lib.df_linear(x[rows].contiguous(), [w["w_" + name]], [w["b_" + name]])
            ref, mass = oracle.rotary(np64(plain).reshape(-1, h, d), angles[rows], interleaved, amplitude=amplitude)
            got = np64(t[name]).reshape(ref.shape)
            # one rounding of the result, and the fp32 sine, cosine and products (2^-20 of the columns' mass)
            assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * mass).all()
    k, _ = lib.df_cache_read(cache, table, torch.tensor([n + 1], dtype=torch.int32, device="cuda"), rows=n + 1)
    rotated = np.concatenate([np64(prompt[0]["k"]), np64(step[0]["k"])[0]])
    assert (np.abs(np64(k[0]) - rotated) <= np.maximum(np.abs(rotated) * 2.0 ** -4, np.abs(rotated).max() * 2.0 ** -17)).all()
