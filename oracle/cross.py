"""Oracle of cross attention (queries of one length against keys and values of
another, shared key heads) and of its gradients, one sequence and one query head
after another in float64.  TEST INFRASTRUCTURE ONLY (see the package header).

Every function also returns the magnitudes that a tolerance counts roundings of:
sums of absolute values in the place of the sums themselves."""

from __future__ import annotations

import numpy as np


def cross_rows(q, k, v, valid, scale, dout=None):
    """One sequence: q [n, H, d], k and v [m, Hk, d], valid [m] (bool).

    Returns a dict: out [n, H, d], lse [n, H], out_mass = sum_j p_ij |v_j|,
    v_sum = sum over valid j of |v_j| [n, H, d], score_mass [n, H] = max_j
    scale sum_c |q_ic k_jc|; with dout also dq, dk, dv and their masses."""
    n, H, d = q.shape
    m, Hk, _ = k.shape
    G = H // Hk
    z = lambda *s: np.zeros(s)  # noqa: E731
    r = dict(out=z(n, H, d), lse=np.full((n, H), -np.inf), out_mass=z(n, H, d), v_sum=z(n, H, d), score_mass=z(n, H))
    if dout is not None:
        r.update({name: z(n, H, d) for name in ("dq", "dq_mass")})
        r.update({name: z(m, Hk, d) for name in ("dk", "dv", "dk_mass", "dv_mass")})
        r["ds_mass"] = z(n, H)
    at = np.nonzero(valid)[0]
    if at.size == 0 or n == 0:
        return r
    for h in range(H):
        hk = h // G
        Q, K, V = q[:, h].astype(np.float64), k[at, hk].astype(np.float64), v[at, hk].astype(np.float64)
        s = scale * (Q @ K.T)
        top = s.max(axis=1, keepdims=True)
        e = np.exp(s - top)
        total = e.sum(axis=1, keepdims=True)
        p = e / total
        r["out"][:, h] = p @ V
        r["lse"][:, h] = (top + np.log(total))[:, 0]
        r["out_mass"][:, h] = p @ np.abs(V)
        r["v_sum"][:, h] = np.abs(V).sum(axis=0)
        r["score_mass"][:, h] = scale * (np.abs(Q) @ np.abs(K).T).max(axis=1)
        if dout is None:
            continue
        g = dout[:, h].astype(np.float64)
        dp = g @ V.T
        row = (g * r["out"][:, h]).sum(axis=1, keepdims=True)
        ds = p * (dp - row)
        # what a relative error of the scores and of dP, D can move dS by
        ds_all = p * (np.abs(g) @ np.abs(V).T + (np.abs(g) * r["out_mass"][:, h]).sum(axis=1, keepdims=True))
        r["dq"][:, h] = scale * (ds @ K)
        r["dq_mass"][:, h] = scale * (ds_all @ np.abs(K))
        r["dk"][at, hk] += scale * (ds.T @ Q)
        r["dk_mass"][at, hk] += scale * (ds_all.T @ np.abs(Q))
        r["dv"][at, hk] += p.T @ g
        r["dv_mass"][at, hk] += p.T @ np.abs(g)
        # the rounding of dS itself to 16 bits, by gradient
        r.setdefault("dq_round", np.zeros((n, H, d)))[:, h] = scale * (np.abs(ds) @ np.abs(K))
        r.setdefault("dk_round", np.zeros((m, Hk, d)))[at, hk] += scale * (np.abs(ds).T @ np.abs(Q))
    return r


def cross_batch(q, k, v, scale, key_mask=None, cu_q=None, cu_k=None, dout=None):
    """A batch in the layouts of the entry points: the same dict, its arrays laid
    out like q (or k); packed rows behind the last sequence are zeros (lse -inf)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    H, d = q.shape[-2:]
    Hk = k.shape[-2]
    B = (len(cu_q) - 1) if cu_q is not None else q.shape[0]
    q2, k2, v2 = q.reshape(-1, H, d), k.reshape(-1, Hk, d), v.reshape(-1, Hk, d)
    g2 = None if dout is None else np.asarray(dout, dtype=np.float64).reshape(-1, H, d)
    at_q = list(cu_q) if cu_q is not None else [b * q.shape[1] for b in range(B + 1)]
    at_k = list(cu_k) if cu_k is not None else [b * k.shape[1] for b in range(B + 1)]
    full = {}
    by_key = ("dk", "dv", "dk_mass", "dv_mass", "dk_round")
    for b in range(B):
        sq, sk = slice(at_q[b], at_q[b + 1]), slice(at_k[b], at_k[b + 1])
        valid = np.ones(at_k[b + 1] - at_k[b], bool) if key_mask is None else np.asarray(key_mask[b]) != 0
        r = cross_rows(q2[sq], k2[sk], v2[sk], valid, scale, None if g2 is None else g2[sq])
        for name, x in r.items():
            rows = k2 if name in by_key else q2
            if name not in full:
                fill = -np.inf if name == "lse" else 0.0
                full[name] = np.full((rows.shape[0],) + x.shape[1:], fill)
            full[name][sk if name in by_key else sq] = x
    lead = lambda x, like: x.reshape(like.shape[:-2] + x.shape[1:])  # noqa: E731
    return {name: lead(x, k if name in by_key else q) for name, x in full.items()}
