"""Inputs and bounds shared by the cross-attention tests."""

from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24  # one fp32 rounding


def inputs(B, H, Hk, d, Lq, Lk, dtype, q="padded", k="full", seed=0, sigma=1.0, nq=None, nk=None):
    """A seeded batch: dict of host tensors (q, k, v, dout, key_mask, cu_q, cu_k).
    `nq`, `nk` give the lengths; drawn in [0, L] otherwise."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed + 1)
    nq = nq if nq is not None else [int(x) for x in rng.integers(0, Lq + 1, B)]
    nk = nk if nk is not None else [int(x) for x in rng.integers(0, Lk + 1, B)]

    def normal(*shape):
        return (torch.randn(*shape, generator=g) * sigma).to(dtype)

    cu = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32)  # noqa: E731
    x = dict(key_mask=None, cu_q=None, cu_k=None)
    q_rows = (B, Lq)
    if q == "packed":
        x["cu_q"] = cu(nq)
        q_rows = (int(sum(nq)),)
    k_rows = (B, Lk)
    if k == "packed":
        x["cu_k"] = cu(nk)
        k_rows = (int(sum(nk)),)
    elif k == "masked":
        m = (np.arange(Lk)[None, :] < np.asarray(nk)[:, None]) & (rng.random((B, Lk)) < 0.9)
        x["key_mask"] = torch.from_numpy(m.astype(np.uint8))
    x["q"], x["k"], x["v"], x["dout"] = normal(*q_rows, H, d), normal(*k_rows, Hk, d), normal(*k_rows, Hk, d), \
        normal(*q_rows, H, d)
    x["Lq"], x["Lk"] = Lq, Lk
    return x


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def want(oracle, x, scale, with_grad=False):
    lists = {n: None if x[n] is None else x[n].cpu().numpy() for n in ("key_mask", "cu_q", "cu_k")}
    return oracle.cross_batch(np64(x["q"]), np64(x["k"]), np64(x["v"]), scale, lists["key_mask"], lists["cu_q"],
                              lists["cu_k"], np64(x["dout"]) if with_grad else None)


def call(binding, x, dev, scale=None, **more):
    return binding.df_cross_attn_fwd(dev["q"], dev["k"], dev["v"], key_mask=dev["key_mask"], cu_seqlens_q=dev["cu_q"],
                                     cu_seqlens_k=dev["cu_k"], max_seqlen_q=x["Lq"], max_seqlen_k=x["Lk"],
                                     scale=scale, **more)


def to_dev(x):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def score_error(w, d):
    """Relative error of a weight exp(s_ij - lse_i): the score is a sum of d products
    accumulated in fp32, scaled and rebased (a few more roundings of values up to
    |s| + 8 log 2), and both the weight and the row's sum carry it; the hardware's
    exp2 adds at most 2^-22 to each."""
    return 2 * (d + 4) * U32 * (w["score_mass"] + 6.0) + 4 * 2.0 ** -22


def out_bound(w, dtype, d):
    """The weights are rounded to the type (half a step each) and the row's sum is
    not, the products are summed in fp32, the result is rounded to the type.  fp16
    weights below its normal range are off by half a step of 2^-24."""
    half = torch.finfo(dtype).eps / 2
    e = score_error(w, d)[..., None]
    low = 2.0 ** -25 * w["v_sum"] if dtype == torch.float16 else 0.0
    p_part = (half * (1 + half) + e) * w["out_mass"] * 1.01 + low
    return p_part, half * (np.abs(w["out"]) + p_part)


def check_forward(out, w, dtype, d, lse=None, out_lo=None):
    got = np64(out)
    assert np.isfinite(got).all()
    p_part, rounding = out_bound(w, dtype, d)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-37
    err = np.abs(got - w["out"])
    assert (err <= p_part + rounding + tiny).all(), float((err - p_part - rounding).max())
    if lse is not None:
        l, e = np64(lse), score_error(w, d)
        empty = np.isinf(w["lse"])
        assert (l[empty] == -np.inf).all()
        # the sum itself is right to e; its logarithm, and the product with ln 2, round
        tol = e[~empty] + 8 * U32 * (np.abs(w["lse"][~empty]) + 6)
        assert (np.abs(l[~empty] - w["lse"][~empty]) <= tol).all()
    if out_lo is not None:
        lo = np64(out_lo)
        half = torch.finfo(dtype).eps / 2
        assert (np.abs(lo) <= half * np.abs(got) * 1.01 + tiny).all()
        # together they carry the fp32 result: the rounding to the type is gone
        assert (np.abs(got + lo - w["out"]) <= p_part + half * rounding + tiny).all()


def call_bwd(binding, x, dev, out, stats, scale=None, **more):
    return binding.df_cross_attn_bwd(dev["q"], dev["k"], dev["v"], out, stats, dev["dout"], key_mask=dev["key_mask"],
                                     cu_seqlens_q=dev["cu_q"], cu_seqlens_k=dev["cu_k"], max_seqlen_q=x["Lq"],
                                     max_seqlen_k=x["Lk"], scale=scale, **more)


def check_backward(grads, w, dtype, d):
    """Three roundings to the type meet in a gradient: of the operand (the weight, or
    dS), of the forward's weights through D, of the result; everything else is fp32.

    Entry by entry each is counted at its worst, half a step of every term.  The
    terms' signs are independent, so over a whole gradient each rounding weighs at
    most half a step of its norm: three halves in all (and the fp32 part, for
    gradients that are themselves differences that cancel)."""
    half = torch.finfo(dtype).eps / 2
    fp32 = float(score_error(w, d).max()) + (d + 4) * U32
    # fp16: results below its normal range are off by half a step of 2^-24
    tiny = 2.0 ** -25 if dtype == torch.float16 else 1e-37
    for name, t in zip(("dq", "dk", "dv"), grads):
        got, ref = np64(t), w[name]
        assert np.isfinite(got).all(), name
        err, mass = np.abs(got - ref), w[name + "_mass"]
        if name == "dv":
            terms = (half + fp32) * mass
        else:
            terms = half * w[name + "_round"] + (half + fp32) * mass
        assert (err <= 1.01 * terms + half * (np.abs(ref) + terms) + tiny).all(), name
        norm = lambda z: float(np.sqrt((z ** 2).sum()))  # noqa: E731
        assert norm(err) <= 3 * half * norm(ref) + 4 * fp32 * norm(mass) + tiny * np.sqrt(err.size), \
            (name, norm(err), norm(ref))
