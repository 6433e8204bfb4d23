"""Workloads of the cross-attention and embedding operators.

Each case is one call (or one training step) as a program that builds a decoder
or a reader on top of the encoder makes it: target tokens are looked up in an
embedding table, the decoder's queries attend to the encoder's states, and in
training the gradients come back.  ``run`` computes a case either in plain
torch operations in 32 bits or, with ``own`` set, through the framework.
"""

import itertools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the token ids of one short request, looked up before its first layer
        {"name": "embed_one_request", "op": "embed", "T": 48, "N": 768, "V": 128100, "dtype": "bf16",
         "scale": 1.0, "pad": -1},
        # a packed batch of 16 documents of 8192 tokens, embeddings scaled by sqrt(width)
        {"name": "embed_long_batch", "op": "embed", "T": 131072, "N": 768, "V": 128100, "dtype": "bf16",
         "scale": math.sqrt(768.0), "pad": -1},
        # gradient of a padded batch's embeddings: a third of the ids are the padding id
        {"name": "embed_grad_padded", "op": "embed_grad", "T": 8192, "N": 1024, "V": 50021, "dtype": "fp16",
         "scale": 1.0, "pad": 0},
        # gradient of the long packed batch
        {"name": "embed_grad_long_batch", "op": "embed_grad", "T": 131072, "N": 768, "V": 128100,
         "dtype": "bf16", "scale": math.sqrt(768.0), "pad": -1},
        # a few short targets against short padded encoder states, one source empty
        {"name": "cross_short_padded", "op": "cross", "B": 4, "H": 12, "Hk": 12, "d": 64, "Lq": 33, "Lk": 200,
         "dtype": "fp16", "q": "padded", "k": "masked", "empty": True},
        # a ragged packed batch with shared key heads
        {"name": "cross_packed_shared", "op": "cross", "B": 64, "H": 16, "Hk": 4, "d": 128, "Lq": 512,
         "Lk": 2048, "dtype": "bf16", "q": "packed", "k": "packed", "empty": False},
        # long documents read by long targets
        {"name": "cross_long", "op": "cross", "B": 16, "H": 12, "Hk": 12, "d": 64, "Lq": 2048, "Lk": 8192,
         "dtype": "bf16", "q": "padded", "k": "full", "empty": False},
        # generation: one query token per sequence, one request
        {"name": "cross_token_one", "op": "cross", "B": 1, "H": 12, "Hk": 12, "d": 64, "Lq": 1, "Lk": 512,
         "dtype": "bf16", "q": "padded", "k": "full", "empty": False},
        # generation: 64 requests over ragged long documents
        {"name": "cross_token_batch", "op": "cross", "B": 64, "H": 24, "Hk": 24, "d": 64, "Lq": 1, "Lk": 8192,
         "dtype": "bf16", "q": "padded", "k": "packed", "empty": False},
        # training steps: short padded batch with holes in the mask, ragged packed
        # batch with shared key heads, long documents
        {"name": "cross_train_padded", "op": "cross_train", "B": 4, "H": 12, "Hk": 12, "d": 64, "Lq": 77,
         "Lk": 300, "dtype": "fp16", "q": "padded", "k": "masked", "empty": True},
        {"name": "cross_train_packed_shared", "op": "cross_train", "B": 64, "H": 16, "Hk": 4, "d": 128,
         "Lq": 512, "Lk": 2048, "dtype": "bf16", "q": "packed", "k": "packed", "empty": False},
        {"name": "cross_train_long", "op": "cross_train", "B": 8, "H": 12, "Hk": 12, "d": 64, "Lq": 2048,
         "Lk": 8192, "dtype": "bf16", "q": "padded", "k": "full", "empty": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "cross", "cross", "cross_token", "cross_train", "cross_train"])
    if op in ("embed", "embed_grad"):
        return {"op": op, "T": _log_int(rng, 1, 131072), "N": 8 * _log_int(rng, 4, 128),
                "V": _log_int(rng, 2, 100000), "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "scale": rng.choice([1.0, 0.5, 27.7]), "pad": rng.choice([-1, 0, 1])}
    token = op == "cross_token"
    op = "cross" if token else op
    hk = rng.choice([1, 2, 4, 8, 12])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    c = {"op": op, "B": _log_int(rng, 1, 48), "H": hk * group, "Hk": hk, "d": rng.choice([32, 64, 64, 96, 128, 128]),
         "Lq": 1 if token else _log_int(rng, 2, 2048), "Lk": _log_int(rng, 1, 8192),
         "dtype": rng.choice(["bf16", "bf16", "fp16"]), "q": rng.choice(["padded", "packed"]),
         "k": rng.choice(["full", "masked", "packed"]), "empty": rng.random() < 0.25}
    if token:
        c["q"] = "padded"
    if op == "cross_train":
        # over a single key the gradients of q and k are zero but for rounding
        c["Lk"] = max(c["Lk"], 16)
    # no dearer than the largest listed cases: the batch first, then the lengths
    top = 4.0e11 if op == "cross_train" else 2.0e11
    while 4.0 * c["B"] * c["H"] * c["Lq"] * c["Lk"] * c["d"] > top or c["B"] * c["Lk"] * hk * c["d"] > 2.0e8:
        if c["B"] > 1:
            c["B"] = (c["B"] + 1) // 2
        else:
            c["Lq"], c["Lk"] = (c["Lq"] + 1) // 2, max((c["Lk"] + 1) // 2, 16)
    return c


# ---------------------------------------------------------------------------
# inputs


def _lengths_on_host(case):
    """Lengths decide the shapes of packed tensors: they are drawn once per case,
    the same for every seed, so that its inputs have the same shapes and work."""
    g = torch.Generator().manual_seed(1000003 + case["B"] * 7919 + case["Lq"] * 31 + case["Lk"])

    def one(longest, empty):
        low = max(1, longest // 4)
        x = torch.randint(low, longest + 1, (case["B"],), generator=g)
        if empty and case["B"] > 1:
            x[-1] = 0
        return [int(v) for v in x]

    nq = one(case["Lq"], case["empty"]) if case["q"] == "packed" else [case["Lq"]] * case["B"]
    nk = one(case["Lk"], case["empty"]) if case["k"] != "full" else [case["Lk"]] * case["B"]
    return nq, nk


def _offsets(lengths):
    return [0] + list(itertools.accumulate(lengths))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    if case["op"] in ("embed", "embed_grad"):
        T, N, V = case["T"], case["N"], case["V"]
        # token frequencies fall about as 1 / rank, as in running text
        u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(V + 1.0)) - 1.0).to(torch.int64).clamp(0, V - 1)
        pad = case["pad"] if case["pad"] < V else -1
        if pad >= 0:
            ids[torch.rand(T, generator=g, device="cuda") < 1.0 / 3.0] = pad
        s = {"op": case["op"], "ids": ids.to(torch.int32), "V": V, "scale": case["scale"], "pad": pad}
        if case["op"] == "embed":
            s["table"] = normal(V, N, std=0.02)
        else:
            s["dout"] = normal(T, N, std=0.1)
        return s

    B, H, Hk, d, Lq, Lk = (case[n] for n in ("B", "H", "Hk", "d", "Lq", "Lk"))
    nq, nk = _lengths_on_host(case)
    cu_q, cu_k = _offsets(nq), _offsets(nk)
    s = {"op": case["op"], "Lq": Lq, "Lk": Lk, "cu_q": None, "cu_k": None, "mask": None}
    if case["q"] == "packed":
        q_rows = (cu_q[-1],)
        s["cu_q"] = torch.tensor(cu_q, dtype=torch.int32, device="cuda")
    else:
        q_rows = (B, Lq)
    if case["k"] == "packed":
        k_rows = (cu_k[-1],)
        s["cu_k"] = torch.tensor(cu_k, dtype=torch.int32, device="cuda")
    else:
        k_rows = (B, Lk)
    s["q"] = normal(*q_rows, H, d)
    s["k"], s["v"] = normal(*k_rows, Hk, d), normal(*k_rows, Hk, d)
    if case["k"] == "masked":
        n = torch.tensor(nk, device="cuda")[:, None]
        at = torch.arange(Lk, device="cuda")[None, :]
        # right padding, and one key in 32 taken out inside the text
        holes = torch.rand(B, Lk, generator=g, device="cuda") < 1.0 / 32.0
        s["mask"] = ((at < n) & ~(holes & (at > 0))).to(torch.uint8)
    if case["op"] == "cross_train":
        s["dout"] = normal(*q_rows, H, d)
    return s


# ---------------------------------------------------------------------------
# the plain form


def _rows(x, cu, longest):
    """[B, L, heads, d] in 32 bits and the rows' validity [B, L]: packed rows are
    taken apart by index, padded ones are as they are."""
    if cu is None:
        return x.float(), torch.ones(x.shape[:2], dtype=torch.bool, device=x.device), None
    at = torch.arange(longest, device=x.device)[None, :]
    valid = at < (cu[1:] - cu[:-1])[:, None]
    idx = (cu[:-1, None].long() + at).clamp(max=x.shape[0] - 1)
    return x[idx].float(), valid, idx


def _repack(x, valid, rows):
    """The valid rows of [B, L, heads, d] one after another."""
    out = torch.zeros((rows,) + tuple(x.shape[2:]), dtype=x.dtype, device=x.device)
    flat = x[valid]
    out[: flat.shape[0]] = flat
    return out


def _plain_cross(s):
    q, qv, _ = _rows(s["q"], s["cu_q"], s["Lq"])
    k, kv, _ = _rows(s["k"], s["cu_k"], s["Lk"])
    v, _, _ = _rows(s["v"], s["cu_k"], s["Lk"])
    if s["mask"] is not None:
        kv = kv & (s["mask"] != 0)
    B, Lq, H, d = q.shape
    Lk, Hk = k.shape[1], k.shape[2]
    G = H // Hk
    # the query rows of the heads that share a key head stand one after another
    q2 = q.view(B, Lq, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * Lq, d)
    k2, v2 = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    v2 = torch.where(kv[:, None, :, None], v2, torch.zeros((), device=v.device))
    scale = 1.0 / math.sqrt(d)
    p = torch.matmul(q2, k2.transpose(2, 3))
    p.mul_(scale)
    p.masked_fill_(~kv[:, None, None, :], -math.inf)
    m = p.amax(dim=3, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p.sub_(m).exp_()
    total = p.sum(dim=3, keepdim=True)
    p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = torch.matmul(p, v2)

    def back(x):  # [B, Hk, G Lq, d] -> the layout of q, in its type
        x = x.view(B, Hk, G, Lq, d).permute(0, 3, 1, 2, 4).reshape(B, Lq, H, d)
        x = x if s["cu_q"] is None else _repack(x, qv, s["q"].shape[0])
        return x.to(s["q"].dtype)

    if s["op"] == "cross":
        return back(o)
    do, _, _ = _rows(s["dout"], s["cu_q"], s["Lq"])
    do = torch.where(qv[:, :, None, None], do, torch.zeros((), device=do.device))
    do2 = do.view(B, Lq, Hk, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * Lq, d)
    dv = torch.matmul(p.transpose(2, 3), do2)
    ds = torch.matmul(do2, v2.transpose(2, 3))
    ds.sub_((do2 * o).sum(dim=3, keepdim=True)).mul_(p).mul_(scale)
    k2 = torch.where(kv[:, None, :, None], k2, torch.zeros((), device=k.device))
    dq = torch.matmul(ds, k2)
    dk = torch.matmul(ds.transpose(2, 3), q2)

    def back_k(x):
        x = x.permute(0, 2, 1, 3)
        x = x if s["cu_k"] is None else _repack(x, kv, s["k"].shape[0])
        return x.to(s["k"].dtype)

    return {"out": back(o), "dq": back(dq), "dk": back_k(dk), "dv": back_k(dv)}


def _plain_embed(s):
    return (s["table"][s["ids"].long()].float() * s["scale"]).to(s["table"].dtype)


def _plain_embed_grad(s):
    ids, dout = s["ids"].long(), s["dout"].double() * s["scale"]
    if s["pad"] >= 0:
        dout = torch.where((ids == s["pad"])[:, None], torch.zeros((), dtype=dout.dtype, device=dout.device), dout)
    # rows of frequent tokens are sums of thousands of terms: added in 64 bits
    out = torch.zeros(s["V"], dout.shape[1], dtype=torch.float64, device=dout.device)
    return out.index_add_(0, ids, dout).float()


def run(s):
    if own:
        from exact_attention_deberta_gb300 import binding
        if s["op"] == "embed":
            return binding.df_embedding(s["ids"], s["table"], scale=s["scale"])
        if s["op"] == "embed_grad":
            return binding.df_embedding_bwd(s["ids"], s["dout"], s["V"], scale=s["scale"],
                                            padding_idx=None if s["pad"] < 0 else s["pad"])
        kw = dict(key_mask=s["mask"], cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"],
                  max_seqlen_q=s["Lq"], max_seqlen_k=s["Lk"])
        if s["op"] == "cross":
            return binding.df_cross_attn_fwd(s["q"], s["k"], s["v"], **kw)
        out, stats = binding.df_cross_attn_fwd(s["q"], s["k"], s["v"], with_stats=True, **kw)
        dq, dk, dv = binding.df_cross_attn_bwd(s["q"], s["k"], s["v"], out, stats, s["dout"], **kw)
        return {"out": out, "dq": dq, "dk": dk, "dv": dv}
    if s["op"] == "embed":
        return _plain_embed(s)
    if s["op"] == "embed_grad":
        return _plain_embed_grad(s)
    return _plain_cross(s)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("embed", "embed_grad"):
        T, N, V = case["T"], case["N"], case["V"]
        # rows of the table that the ids reach, for frequencies that fall as 1 / rank
        r = torch.arange(1, V + 1, dtype=torch.float64)
        hit = float((1.0 - torch.exp(T * torch.log1p(-torch.log1p(1.0 / r) / math.log(V + 1.0)))).sum())
        if case["op"] == "embed":
            return {"bytes": 4.0 * T + size * N * (hit + T), "flops": 1.0 * T * N}
        kept = T * (2.0 / 3.0 if 0 <= case["pad"] < V else 1.0)
        return {"bytes": 4.0 * T + size * N * kept + 4.0 * V * N, "flops": 1.0 * kept * N}
    nq, nk = _lengths_on_host(case)
    H, Hk, d = case["H"], case["Hk"], case["d"]
    rows_q = sum(nq) * H * d * 2.0
    rows_k = sum(nk) * Hk * d * 2.0
    pairs = float(sum(a * b for a, b in zip(nq, nk))) * H * d
    if case["op"] == "cross":
        return {"bytes": 2 * rows_q + 2 * rows_k, "flops": 4.0 * pairs}
    # forward, then its gradient: q, k, v, dout in, out, dq, dk, dv out; two
    # products forward, five back
    return {"bytes": 4 * rows_q + 4 * rows_k, "flops": 14.0 * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence and one key head after another


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        return s["table"].double().index_select(0, s["ids"].long()) * s["scale"]
    if case["op"] == "embed_grad":
        out = torch.zeros(s["V"], s["dout"].shape[1], dtype=torch.float64, device="cuda")
        keep = s["ids"] != s["pad"]
        ids, rows = s["ids"][keep].long(), s["dout"][keep].double()
        return out.index_add_(0, ids, rows).mul_(s["scale"])
    nq, nk = _lengths_on_host(case)
    H, Hk, d = case["H"], case["Hk"], case["d"]
    G = H // Hk
    q, k, v = (s[n].reshape(-1, s[n].shape[-2], d) for n in ("q", "k", "v"))
    train = case["op"] == "cross_train"
    do = s["dout"].reshape(-1, H, d) if train else None
    out, dq = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    dk, dv = (torch.zeros(k.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    at_q = s["cu_q"].tolist() if s["cu_q"] is not None else [b * case["Lq"] for b in range(case["B"] + 1)]
    at_k = s["cu_k"].tolist() if s["cu_k"] is not None else [b * case["Lk"] for b in range(case["B"] + 1)]
    for b in range(case["B"]):
        rq = slice(at_q[b], at_q[b + 1])
        rk = torch.arange(at_k[b], at_k[b + 1], device="cuda")
        if s["mask"] is not None:
            rk = rk[s["mask"][b] != 0]
        n, m = at_q[b + 1] - at_q[b], rk.numel()
        if n == 0 or m == 0:
            continue
        for h in range(Hk):
            qs = q[rq, h * G:(h + 1) * G].double().reshape(n * G, d)
            ks, vs = k[rk, h].double(), v[rk, h].double()
            p = torch.softmax(qs @ ks.T / math.sqrt(d), dim=1)
            o = p @ vs
            out[rq, h * G:(h + 1) * G] = o.view(n, G, d)
            if not train:
                continue
            g = do[rq, h * G:(h + 1) * G].double().reshape(n * G, d)
            dv[rk, h] = p.T @ g
            dp = g @ vs.T
            dp -= (g * o).sum(dim=1, keepdim=True)
            dp *= p
            dp /= math.sqrt(d)
            dq[rq, h * G:(h + 1) * G] = (dp @ ks).view(n, G, d)
            dk[rk, h] = dp.T @ qs
    out, dq = out.view(s["q"].shape), dq.view(s["q"].shape)
    if not train:
        return out
    return {"out": out, "dq": dq, "dk": dk.view(s["k"].shape), "dv": dv.view(s["k"].shape)}
