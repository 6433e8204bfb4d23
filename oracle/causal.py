"""Oracle of causal attention with a sliding window and sinks and of its gradients, one
sequence and one query head after another in float64.  TEST INFRASTRUCTURE ONLY (see the
package header).  The queries of a sequence are the last of its tokens."""

from __future__ import annotations

import numpy as np


def visible(n, m, window=0, sinks=0):
    """[n, m]: whether query i, at position i + m - n, sees key j."""
    p, j = np.arange(n)[:, None] + (m - n), np.arange(m)[None, :]
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def causal_rows(q, k, v, valid, scale, window=0, sinks=0, dout=None):
    """One sequence: q [n, H, d], k and v [m, Hk, d], valid [m] (bool).  The dict of
    ``cross_rows``: results, and the masses that a tolerance counts roundings of."""
    n, H, d = q.shape
    m, Hk, _ = k.shape
    G = H // Hk
    z = lambda *s: np.zeros(s)  # noqa: E731
    r = dict(out=z(n, H, d), lse=np.full((n, H), -np.inf), out_mass=z(n, H, d), v_sum=z(n, H, d), score_mass=z(n, H))
    if dout is not None:
        r.update({name: z(n, H, d) for name in ("dq", "dq_mass", "dq_round")})
        r.update({name: z(m, Hk, d) for name in ("dk", "dv", "dk_mass", "dv_mass", "dk_round")})
    if n == 0 or m == 0:
        return r
    seen = visible(n, m, window, sinks) & np.asarray(valid, bool)[None, :]
    some = seen.any(axis=1)
    for h in range(H):
        hk = h // G
        Q, K, V = q[:, h].astype(np.float64), k[:, hk].astype(np.float64), v[:, hk].astype(np.float64)
        s = np.where(seen, scale * (Q @ K.T), -np.inf)
        top = np.where(some, s.max(axis=1), 0.0)[:, None]
        e = np.exp(s - top)
        total = np.where(some, e.sum(axis=1), 1.0)[:, None]
        p = e / total
        r["out"][:, h] = p @ V
        r["lse"][some, h] = (top + np.log(total))[some, 0]
        r["out_mass"][:, h] = p @ np.abs(V)
        r["v_sum"][:, h] = seen @ np.abs(V)
        r["score_mass"][:, h] = scale * np.where(seen, np.abs(Q) @ np.abs(K).T, 0.0).max(axis=1)
        if dout is None:
            continue
        g = dout[:, h].astype(np.float64)
        ds = p * (g @ V.T - (g * r["out"][:, h]).sum(axis=1, keepdims=True))
        ds_all = p * (np.abs(g) @ np.abs(V).T + (np.abs(g) * r["out_mass"][:, h]).sum(axis=1, keepdims=True))
        r["dq"][:, h] = scale * (ds @ K)
        r["dq_mass"][:, h] = scale * (ds_all @ np.abs(K))
        r["dq_round"][:, h] = scale * (np.abs(ds) @ np.abs(K))
        r["dk"][:, hk] += scale * (ds.T @ Q)
        r["dk_mass"][:, hk] += scale * (ds_all.T @ np.abs(Q))
        r["dk_round"][:, hk] += scale * (np.abs(ds).T @ np.abs(Q))
        r["dv"][:, hk] += p.T @ g
        r["dv_mass"][:, hk] += p.T @ np.abs(g)
    return r


def causal_batch(q, k, v, scale, window=0, sinks=0, key_mask=None, cu_q=None, cu_k=None, dout=None):
    """A batch in the layouts of the entry points: the same dict, its arrays laid out like q
    (or k); packed rows behind the last sequence are zeros (lse -inf)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    H, d = q.shape[-2:]
    Hk = k.shape[-2]
    B = (len(cu_q) - 1) if cu_q is not None else q.shape[0]
    q2, k2, v2 = q.reshape(-1, H, d), k.reshape(-1, Hk, d), v.reshape(-1, Hk, d)
    g2 = None if dout is None else np.asarray(dout, dtype=np.float64).reshape(-1, H, d)
    at_q = list(cu_q) if cu_q is not None else [b * q.shape[1] for b in range(B + 1)]
    at_k = list(cu_k) if cu_k is not None else [b * k.shape[1] for b in range(B + 1)]
    by_key = ("dk", "dv", "dk_mass", "dv_mass", "dk_round")
    full = {}
    for b in range(B):
        sq, sk = slice(at_q[b], at_q[b + 1]), slice(at_k[b], at_k[b + 1])
        valid = np.ones(at_k[b + 1] - at_k[b], bool) if key_mask is None else np.asarray(key_mask[b]) != 0
        r = causal_rows(q2[sq], k2[sk], v2[sk], valid, scale, window, sinks, None if g2 is None else g2[sq])
        for name, x in r.items():
            rows = k2 if name in by_key else q2
            if name not in full:
                full[name] = np.full((rows.shape[0],) + x.shape[1:], -np.inf if name == "lse" else 0.0)
            full[name][sk if name in by_key else sq] = x
    return {name: x.reshape((k if name in by_key else q).shape[:-2] + x.shape[1:]) for name, x in full.items()}
