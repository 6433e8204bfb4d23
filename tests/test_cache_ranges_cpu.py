"""The cache oracle at the top of bf16's range."""

import numpy as np
import torch

import oracle


def test_finite_values_are_held_as_finite_ones():
    top = torch.arange(1 << 15, dtype=torch.int32)[-129 * 128:].to(torch.int16).view(torch.bfloat16)
    x = top[top.isfinite()].double().numpy()
    assert x.max() == float(torch.finfo(torch.bfloat16).max)
    x = np.concatenate([x, -x]).reshape(-1, 1, 32)
    for rows in (x, np.concatenate([np.full((3, 1, 32), x.max()), x])):
        got = oracle.CacheOracle(1, 32).append(rows).values()
        scale = oracle.CacheOracle(1, 32).append(rows).scale[np.arange(len(rows)) // 16][:, :, None]
        assert (got.astype(np.float32) == got).all() and np.isfinite(got.astype(np.float32)).all()
        assert (np.abs(got - rows) <= np.maximum(2.0 ** -4 * np.abs(rows), 2.0 ** -10 * scale)).all()


def test_what_is_not_finite_is_not_a_number():
    x = np.array([np.inf, -np.inf, np.nan, 3.3e38]).reshape(4, 1, 1) * np.ones((1, 1, 32))
    got = oracle.CacheOracle(1, 32).append(x).values()
    assert np.isnan(got[:3]).all() and (got[3] == 240.0 * 2.0 ** 120).all()
