"""Oracle of the embedding lookup with scaling and of its table's gradient
(float64).  TEST INFRASTRUCTURE ONLY (see the package header)."""

from __future__ import annotations

import numpy as np


def embed(ids, table, scale):
    """scale * table[ids]; zeros where an id is outside the table."""
    ids = np.asarray(ids, dtype=np.int64)
    table = np.asarray(table, dtype=np.float64)
    inside = (ids >= 0) & (ids < table.shape[0])
    rows = table[np.where(inside, ids, 0)] * scale
    return np.where(inside[..., None], rows, 0.0)


def embed_grad(ids, dout, vocab, scale, padding_idx=None, grad=None):
    """(the gradient [vocab, N], the sum of |scale * dout| added to each entry,
    the number of rows added to each table row)."""
    ids = np.asarray(ids, dtype=np.int64).reshape(-1)
    dout = np.asarray(dout, dtype=np.float64).reshape(ids.size, -1)
    keep = (ids >= 0) & (ids < vocab)
    if padding_idx is not None:
        keep &= ids != padding_idx
    out = np.zeros((vocab, dout.shape[1])) if grad is None else np.array(grad, dtype=np.float64)
    mass = np.abs(out)
    count = np.zeros(vocab, dtype=np.int64)
    for t in np.nonzero(keep)[0]:
        out[ids[t]] += scale * dout[t]
        mass[ids[t]] += np.abs(scale * dout[t])
        count[ids[t]] += 1
    return out, mass, count
