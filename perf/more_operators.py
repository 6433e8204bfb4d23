"""Workloads of a decoder's own attention beside the encoder: rotary positions,
causal attention with a sliding window and sinks, and the 8-bit paged cache.

Each case is one call (or one training step) as a program that trains, prompts or
generates with a decoder makes it.  ``run`` computes a case either in plain torch
operations in 32 bits or, with ``own`` set, through the framework.

The cache's record of 16 tokens of one head (32 d + 16 bytes): the keys' e4m3 codes
as [d / 32][16][32], the values' likewise, the keys' and the values' scale (float32),
8 bytes unused; pages are [n_pages, heads, page / 16, 32 d + 16].
"""

import itertools
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 16


def listed():
    return [
        # queries and keys of a packed batch of 16 documents of 8192 tokens, positions
        # stretched to four times the length that the frequencies were made for
        {"name": "rotary_long_batch", "op": "rotary", "T": 131072, "H": 12, "Hk": 12, "d": 64, "rot": 64,
         "inter": False, "inverse": False, "dtype": "bf16", "far": 32768, "factor": 4.0},
        # the gradient of a part of each head in interleaved pairs, shared key heads
        {"name": "rotary_grad_part", "op": "rotary", "T": 8191, "H": 16, "Hk": 4, "d": 128, "rot": 48,
         "inter": True, "inverse": True, "dtype": "fp16", "far": 8192, "factor": 1.0},
        # a few short right-padded prompts, one of them empty
        {"name": "self_short_padded", "op": "self", "B": 4, "H": 12, "Hk": 12, "d": 64, "Lq": 77, "Lk": 77,
         "dtype": "fp16", "layout": "masked", "empty": True, "window": 0, "sinks": 0},
        # prompts of long documents, each token sees the last 1024 and the first 4
        {"name": "self_window_long", "op": "self", "B": 16, "H": 12, "Hk": 12, "d": 64, "Lq": 8192, "Lk": 8192,
         "dtype": "bf16", "layout": "full", "empty": False, "window": 1024, "sinks": 4},
        # training steps: a ragged packed batch with shared key heads, every earlier
        # token visible; long documents with a window
        {"name": "self_train_packed_shared", "op": "self_train", "B": 64, "H": 16, "Hk": 4, "d": 128, "Lq": 2048,
         "Lk": 2048, "dtype": "bf16", "layout": "packed", "empty": False, "window": 0, "sinks": 0},
        {"name": "self_train_window", "op": "self_train", "B": 8, "H": 12, "Hk": 12, "d": 64, "Lq": 8192,
         "Lk": 8192, "dtype": "bf16", "layout": "full", "empty": False, "window": 1024, "sinks": 16},
        # ragged prompts stored in an empty cache and read back for the next chunk
        {"name": "cache_store_prompt", "op": "cache_store", "B": 64, "Hk": 12, "d": 64, "old": 0, "new": 8192,
         "page": 64, "dtype": "bf16"},
        # one token added to each of 64 short sequences, whose rows are then read
        {"name": "cache_store_step", "op": "cache_store", "B": 64, "Hk": 8, "d": 128, "old": 499, "new": 1,
         "page": 16, "dtype": "fp16"},
        # generation: one request, one token
        {"name": "cache_token_one", "op": "cache", "B": 1, "H": 12, "Hk": 12, "d": 64, "Lq": 1, "L": 512, "page": 64,
         "dtype": "bf16", "causal": True, "window": 0, "sinks": 0},
        # generation: 64 requests over ragged long caches
        {"name": "cache_token_batch", "op": "cache", "B": 64, "H": 24, "Hk": 24, "d": 64, "Lq": 1, "L": 8192,
         "page": 64, "dtype": "bf16", "causal": True, "window": 0, "sinks": 0},
        # four proposed tokens for each of 16 long requests, shared key heads, a window
        {"name": "cache_few_window", "op": "cache", "B": 16, "H": 32, "Hk": 8, "d": 128, "Lq": 4, "L": 32768,
         "page": 16, "dtype": "bf16", "causal": True, "window": 4096, "sinks": 16},
        # one token per request reads the encoder's states, held in 8 bits
        {"name": "cache_states", "op": "cache", "B": 64, "H": 16, "Hk": 4, "d": 128, "Lq": 1, "L": 4096, "page": 128,
         "dtype": "fp16", "causal": False, "window": 0, "sinks": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "self", "self", "self_train", "self_train", "cache_store", "cache", "cache"])
    hk = rng.choice([1, 2, 4, 8, 12])
    group = rng.choice([1, 1, 2, 3, 4, 8])
    if op == "rotary":
        d = rng.choice([32, 64, 64, 80, 96, 128, 128])
        c = {"op": op, "T": _log_int(rng, 1, 131072), "H": hk * group, "Hk": hk, "d": d,
             "rot": rng.choice([d, d, d // 2, 2 * rng.randint(1, d // 2)]), "inter": rng.random() < 0.5,
             "inverse": rng.random() < 0.4, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
             "far": _log_int(rng, 2, 4000000), "factor": rng.choice([1.0, 1.0, 2.0, 8.0])}
        while c["T"] * (c["H"] + c["Hk"]) * d * (4 if c["dtype"] == "fp32" else 2) > 4.1e8:
            c["T"] = (c["T"] + 1) // 2
        return c
    if op in ("self", "self_train"):
        c = {"op": op, "B": _log_int(rng, 1, 48), "H": hk * group, "Hk": hk,
             "d": rng.choice([32, 64, 64, 96, 128, 128]), "Lq": 1, "Lk": _log_int(rng, 2, 8192),
             "dtype": rng.choice(["bf16", "bf16", "fp16"]), "layout": rng.choice(["full", "masked", "packed"]),
             "empty": rng.random() < 0.25, "window": rng.choice([0, 0, 1, 1, 1]), "sinks": 0}
        if op == "self_train":
            # over a single key the gradients of q and k are zero but for rounding
            c["Lk"] = max(c["Lk"], 16)
        if c["window"]:
            c["window"] = _log_int(rng, 8, c["Lk"] + 8)
            c["sinks"] = rng.choice([0, 1, 4, 16, 200])
        while c["B"] * c["H"] * _pairs([c["Lk"]], [c["Lk"]], c["window"], c["sinks"]) * c["d"] > 1.0e11:
            if c["B"] > 1:
                c["B"] = (c["B"] + 1) // 2
            else:
                c["Lk"] = (c["Lk"] + 1) // 2
        # the queries are all tokens, or the last part of them
        c["Lq"] = c["Lk"] if rng.random() < 0.6 else max(1, c["Lk"] // rng.choice([2, 3, 8]))
        return c
    d = rng.choice([32, 64, 64, 96, 128, 128])
    page = rng.choice([16, 16, 32, 64, 64, 128, 256, 48])
    B = _log_int(rng, 1, 64)
    if op == "cache_store":
        c = {"op": op, "B": B, "Hk": hk, "d": d, "old": rng.choice([0, _log_int(rng, 1, 2000)]),
             "new": rng.choice([1, _log_int(rng, 1, 8192)]), "page": page, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
        while c["B"] * (c["old"] + c["new"]) * hk * d > 2.5e8:
            c["B"], c["new"] = (c["B"] + 1) // 2, (c["new"] + 1) // 2
        return c
    c = {"op": op, "B": B, "H": hk * group, "Hk": hk, "d": d, "Lq": rng.choice([1, 1, 1, 2, 4, 7, 16]),
         "L": _log_int(rng, 1, 32768), "page": page, "dtype": rng.choice(["bf16", "bf16", "fp16"]),
         "causal": rng.random() < 0.75, "window": 0, "sinks": 0}
    c["L"] = max(c["L"], c["Lq"])
    if c["causal"] and rng.random() < 0.5:
        c["window"], c["sinks"] = _log_int(rng, 8, c["L"] + 8), rng.choice([0, 1, 4, 16, 100])
    while c["B"] * c["L"] * hk * d > 4.0e8 or 4.0 * c["B"] * c["L"] * c["Lq"] * c["H"] * d > 4.0e10:
        if c["B"] > 1:
            c["B"] = (c["B"] + 1) // 2
        else:
            c["L"] = max((c["L"] + 1) // 2, c["Lq"])
    return c


# ---------------------------------------------------------------------------
# inputs


def _ragged(n, longest, salt, shortest=None):
    """Lengths decide the shapes of packed tensors: they are drawn once per case, the
    same for every seed, so that its inputs have the same shapes and work."""
    g = torch.Generator().manual_seed(1000003 + n * 7919 + longest * 31 + salt)
    low = max(1, longest // 4) if shortest is None else shortest
    return [int(v) for v in torch.randint(low, longest + 1, (n,), generator=g)]


def _self_lengths(case):
    """Queries and keys of each sequence."""
    B, Lq, Lk = case["B"], case["Lq"], case["Lk"]
    if case["layout"] != "packed":
        return [Lq] * B, [Lk] * B
    nk = _ragged(B, Lk, 1)
    nq = [max(1, n * Lq // Lk) for n in nk]
    if case["empty"] and B > 1:
        nq[-1] = nk[-1] = 0
    return nq, nk


def _cache_lengths(case):
    """Tokens of each sequence before the call, and the call's own."""
    if case["op"] == "cache":
        n = _ragged(case["B"], case["L"], 2, max(case["Lq"], case["L"] // 4))
        return n, [case["Lq"]] * case["B"]
    old = _ragged(case["B"], case["old"], 3) if case["old"] else [0] * case["B"]
    return old, _ragged(case["B"], case["new"], 4)


def _offsets(lengths):
    return [0] + list(itertools.accumulate(lengths))


def _pairs(nq, nk, window, sinks):
    """Visible (query, key) pairs."""
    total = 0
    for a, b in zip(nq, nk):
        p = torch.arange(b - a, b, dtype=torch.int64)
        p = p[p >= 0]
        seen = p + 1
        if window:
            low = (p + 1 - window).clamp(min=0)
            seen = p + 1 - low + torch.minimum(low, torch.full_like(low, sinks))
        total += int(seen.sum())
    return float(total)


def _frequencies(rot, factor, far):
    """Per pair, radians a position; 64 bits.  Long contexts: pairs that turn often within
    the original length keep their frequency, slow ones are divided by `factor`."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f
    turns = f * (far / factor) / (2.0 * math.pi)
    keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor)


def _records(k, v):
    """Keys and values [blocks, heads, 16, d] in 32 bits to the cache's records."""
    nb, heads, _, d = k.shape
    rec = torch.zeros(nb, heads, 32 * d + 16, dtype=torch.uint8, device=k.device)
    for i, x in enumerate((k, v)):
        scale = _block_scale(x.abs().amax(dim=(2, 3)))
        code = (x / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        code = code.view(nb, heads, BLOCK, d // 32, 32).transpose(2, 3).reshape(nb, heads, 16 * d)
        rec[:, :, 16 * d * i:16 * d * (i + 1)] = code
        rec[:, :, 32 * d + 4 * i:32 * d + 4 * i + 4] = scale.contiguous().view(torch.uint8).view(nb, heads, 4)
    return rec


def _block_scale(top):
    """The least power of two, 2^-100 or more, with top <= 448 of it."""
    m, e = torch.frexp(top)  # top = m 2^e, 448 = 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(top > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    if case["op"] == "rotary":
        T = case["T"]
        # documents one after another, the first one from a late position
        first = int(torch.randint(0, case["far"], (1,), generator=g, device="cuda"))
        pos = (torch.arange(T, device="cuda") + first) % case["far"]
        s = {"op": "rotary", "x": [normal(T, h, case["d"]) for h in (case["H"], case["Hk"])],
             "pos": pos.to(torch.int32), "inter": case["inter"], "inverse": case["inverse"], "rot": case["rot"],
             "amplitude": 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0}
        if own:
            from exact_attention_deberta_gb300 import binding
            s["table"] = binding.df_rotary_table(case["rot"], base=10000.0, factor=case["factor"],
                                                 original_len=case["far"] / case["factor"], low=1.0, high=32.0)
        else:
            s["freq"] = _frequencies(case["rot"], case["factor"], case["far"]).cuda()
        return s
    if case["op"] in ("self", "self_train"):
        B, H, Hk, d, Lq, Lk = (case[n] for n in ("B", "H", "Hk", "d", "Lq", "Lk"))
        nq, nk = _self_lengths(case)
        s = {"op": case["op"], "Lq": Lq, "Lk": Lk, "cu_q": None, "cu_k": None, "mask": None, "nq": nq, "nk": nk,
             "window": case["window"], "sinks": case["sinks"]}
        if case["layout"] == "packed":
            q_rows, k_rows = (sum(nq),), (sum(nk),)
            s["cu_q"], s["cu_k"] = (torch.tensor(_offsets(n), dtype=torch.int32, device="cuda") for n in (nq, nk))
        else:
            q_rows, k_rows = (B, Lq), (B, Lk)
        s["q"] = normal(*q_rows, H, d)
        s["k"], s["v"] = normal(*k_rows, Hk, d), normal(*k_rows, Hk, d)
        if case["layout"] == "masked":
            n = torch.tensor(_ragged(B, Lk, 5), device="cuda")
            if case["empty"] and B > 1:
                n[-1] = 0
            at = torch.arange(Lk, device="cuda")[None, :]
            s["mask"] = (at < n[:, None]).to(torch.uint8)
        if case["op"] == "self_train":
            s["dout"] = normal(*q_rows, H, d)
        return s
    B, Hk, d, page = (case[n] for n in ("B", "Hk", "d", "page"))
    held, new = _cache_lengths(case)
    store = case["op"] == "cache_store"
    ends = [a + b for a, b in zip(held, new)] if store else held
    need = [(n + page - 1) // page for n in ends]
    n_pages = sum(need) + 1
    # pages come in no order, as a pool hands them out
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    # channels differ in size, as a projection's do
    size = torch.exp(0.5 * torch.randn(2, Hk, 1, d, generator=g, device="cuda"))
    per = page // BLOCK
    cache = torch.empty(n_pages, Hk, per, 32 * d + 16, dtype=torch.uint8, device="cuda")
    some = max(1, (1 << 25) // (Hk * BLOCK * d * per))  # pages at a time
    for p0 in range(0, n_pages, some):
        n = min(some, n_pages - p0)
        kv = [torch.randn(n * per, Hk, BLOCK, d, generator=g, device="cuda") * size[i] for i in range(2)]
        cache[p0:p0 + n] = _records(*kv).view(n, per, Hk, -1).transpose(1, 2)
    s = {"op": case["op"], "cache": cache, "table": table, "page": page, "d": d,
         "held": torch.tensor(held, dtype=torch.int32, device="cuda"), "dtype": dt}
    if store:
        rows = sum(new)
        s["k"], s["v"] = ((torch.randn(rows, Hk, d, generator=g, device="cuda") * size[i, :, 0]).to(dt) for i in range(2))
        s["cu"] = torch.tensor(_offsets(new), dtype=torch.int32, device="cuda")
        s["ends"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["cu_all"] = torch.tensor(_offsets(ends), dtype=torch.int32, device="cuda")
        s["new"], s["total"], s["n"] = max(new), sum(ends), (held, new)
        return s
    s["q"] = normal(B, case["Lq"], case["H"], d)
    s.update(n=held, L=max(held), causal=case["causal"], window=case["window"], sinks=case["sinks"])
    return s


# ---------------------------------------------------------------------------
# the plain form


def _plain_rotary(s):
    # far positions: the angles in 64 bits
    angle = s["pos"].double()[:, None] * s["freq"]
    cos = (torch.cos(angle) * s["amplitude"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["amplitude"]).float()[:, None, :]
    if s["inverse"]:
        sin = -sin
    r, out = s["rot"], []
    for x in s["x"]:
        y = x.float()
        head = y[..., :r]
        a, b = (head[..., 0::2], head[..., 1::2]) if s["inter"] else (head[..., :r // 2], head[..., r // 2:])
        turned = (a * cos - b * sin, b * cos + a * sin)
        turned = torch.stack(turned, dim=-1).flatten(-2) if s["inter"] else torch.cat(turned, dim=-1)
        out.append(torch.cat((turned, y[..., r:]), dim=-1).to(x.dtype))
    return out


def _seen(p, keys, window, sinks):
    """[queries, keys]: which of the keys (positions) the queries at positions p see."""
    seen = keys[None, :] <= p[:, None]
    if window:
        seen &= (keys[None, :] > p[:, None] - window) | (keys[None, :] < sinks)
    return seen


def _plain_self(s, rows=1024):
    """Sequence after sequence, some query rows at a time, over the keys that those can see."""
    q, k, v = s["q"], s["k"], s["v"]
    H, d = q.shape[-2:]
    Hk = k.shape[-2]
    G, scale, dev = H // Hk, 1.0 / math.sqrt(d), q.device
    train = s["op"] == "self_train"
    q, k, v = q.reshape(-1, H, d), k.reshape(-1, Hk, d), v.reshape(-1, Hk, d)
    out = torch.zeros_like(q)
    if train:
        do = s["dout"].reshape(-1, H, d)
        dq = torch.zeros_like(q)
        dk, dv = (torch.zeros(k.shape, dtype=torch.float32, device=dev) for _ in range(2))
    cq, ck = _offsets(s["nq"]), _offsets(s["nk"])
    for b, (n, m) in enumerate(zip(s["nq"], s["nk"])):
        kb = k[ck[b]:ck[b + 1]].float().transpose(0, 1)  # [Hk, m, d]
        vb = v[ck[b]:ck[b + 1]].float().transpose(0, 1)
        counts = None
        if s["mask"] is not None:
            counts = s["mask"][b] != 0
            vb = torch.where(counts[None, :, None], vb, torch.zeros((), device=dev))
        for i0 in range(0, n, rows):
            i1 = min(n, i0 + rows)
            p = torch.arange(i0, i1, device=dev) + (m - n)
            hi = i1 + m - n
            if hi <= 0:
                continue
            lo = max(0, i0 + m - n + 1 - s["window"]) if s["window"] else 0
            head = min(s["sinks"], lo)
            keys = torch.cat((torch.arange(head, device=dev), torch.arange(lo, hi, device=dev)))
            seen = _seen(p, keys, s["window"], s["sinks"])
            if counts is not None:
                seen = seen & counts[keys][None, :]
            seen = seen.repeat(G, 1)  # the query heads that share a key head stand one after another
            kk, vv = kb[:, keys], vb[:, keys]

            def rows_of(x):
                x = x[cq[b] + i0:cq[b] + i1].float()
                return x.view(i1 - i0, Hk, G, d).permute(1, 2, 0, 3).reshape(Hk, G * (i1 - i0), d)

            def back(x):
                return x.view(Hk, G, i1 - i0, d).permute(2, 0, 1, 3).reshape(i1 - i0, H, d).to(q.dtype)

            qq = rows_of(q)
            w = torch.matmul(qq, kk.transpose(1, 2))
            w.mul_(scale)
            w.masked_fill_(~seen, -math.inf)
            top = w.amax(dim=2, keepdim=True)
            top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
            w.sub_(top).exp_()
            total = w.sum(dim=2, keepdim=True)
            w.div_(torch.where(total > 0, total, torch.ones_like(total)))
            o = torch.matmul(w, vv)
            out[cq[b] + i0:cq[b] + i1] = back(o)
            if not train:
                continue
            gg = rows_of(do)
            dvv = torch.matmul(w.transpose(1, 2), gg)
            ds = torch.matmul(gg, vv.transpose(1, 2))
            ds.sub_((gg * o).sum(dim=2, keepdim=True)).mul_(w).mul_(scale)
            dq[cq[b] + i0:cq[b] + i1] = back(torch.matmul(ds, kk))
            dkk = torch.matmul(ds.transpose(1, 2), qq)
            # (the keys of a part are the sinks and a run)
            for dst, src in ((dk, dkk), (dv, dvv)):
                src = src.transpose(0, 1)
                dst[ck[b]:ck[b] + head] += src[:head]
                dst[ck[b] + lo:ck[b] + hi] += src[head:]
    out = out.view(s["q"].shape)
    if not train:
        return out
    return {"out": out, "dq": dq.view(s["q"].shape), "dk": dk.to(k.dtype).view(s["k"].shape),
            "dv": dv.to(v.dtype).view(s["v"].shape)}


def _plain_rows(s, b, lo, hi):
    """Keys and values of sequence b at positions lo .. hi - 1 in 32 bits, [heads, hi - lo, d]."""
    page, d, cache = s["page"], s["d"], s["cache"]
    heads = cache.shape[1]
    p0, p1 = lo // page, (hi + page - 1) // page
    rec = cache[s["table"][b, p0:p1].long()].transpose(0, 1).reshape(heads, -1, 32 * d + 16)
    scale = rec[..., 32 * d:32 * d + 8].contiguous().view(torch.float32)
    both = []
    for i in range(2):
        x = rec[..., 16 * d * i:16 * d * (i + 1)].contiguous().view(torch.float8_e4m3fn).float()
        x = x * scale[..., i:i + 1]
        x = x.view(heads, -1, d // 32, BLOCK, 32).transpose(2, 3).reshape(heads, -1, d)
        both.append(x[:, lo - p0 * page:hi - p0 * page])
    return both


def _plain_cache(s):
    q = s["q"]
    B, n, H, d = q.shape
    Hk = s["cache"].shape[1]
    G, scale, dev = H // Hk, 1.0 / math.sqrt(d), q.device
    out = torch.zeros_like(q)
    for b, m in enumerate(s["n"]):
        lo = max(0, m - n + 1 - s["window"]) if s["window"] else 0
        head = min(s["sinks"], lo)
        k, v = _plain_rows(s, b, lo, m)
        keys = torch.arange(lo, m, device=dev)
        if head:
            ks, vs = _plain_rows(s, b, 0, head)
            k, v = torch.cat((ks, k), dim=1), torch.cat((vs, v), dim=1)
            keys = torch.cat((torch.arange(head, device=dev), keys))
        qq = q[b].float().view(n, Hk, G, d).permute(1, 2, 0, 3).reshape(Hk, G * n, d)
        w = torch.matmul(qq, k.transpose(1, 2)).mul_(scale)
        if s["causal"]:
            seen = _seen(torch.arange(m - n, m, device=dev), keys, s["window"], s["sinks"])
            w.masked_fill_(~seen.repeat(G, 1), -math.inf)
        w.sub_(w.amax(dim=2, keepdim=True)).exp_()
        w.div_(w.sum(dim=2, keepdim=True))
        o = torch.matmul(w, v)
        out[b] = o.view(Hk, G, n, d).permute(2, 0, 1, 3).reshape(n, H, d).to(q.dtype)
    return out


def _plain_store(s):
    """The rows that the cache holds after the new ones are added, block by block."""
    d, dt = s["d"], s["dtype"]
    heads = s["cache"].shape[1]
    held, new = s["n"]
    cu, cu_all = _offsets(new), _offsets([a + b for a, b in zip(held, new)])
    out = [torch.empty(s["total"], heads, d, dtype=dt, device=s["k"].device) for _ in range(2)]
    for b, (m, n) in enumerate(zip(held, new)):
        kept = m % BLOCK
        base = m - kept
        if base:
            for o, x in zip(out, _plain_rows(s, b, 0, base)):
                o[cu_all[b]:cu_all[b] + base] = x.transpose(0, 1).to(dt)
        part = _plain_rows(s, b, base, m) if kept else None
        scales = None
        if kept:
            rec = s["cache"][s["table"][b, base // s["page"]].long(), :, (base % s["page"]) // BLOCK]
            scales = rec[:, 32 * d:32 * d + 8].contiguous().view(torch.float32)
        for i, x in enumerate((s["k"], s["v"])):
            rows = x[cu[b]:cu[b + 1]].float().transpose(0, 1)  # [heads, n, d]
            if kept:
                rows = torch.cat((part[i], rows), dim=1)
            pad = -rows.shape[1] % BLOCK
            full = torch.nn.functional.pad(rows, (0, 0, 0, pad)).view(heads, -1, BLOCK, d)
            fresh = full.abs()
            if kept:
                # the block's scale stays or grows: older rows count by the scale that they have
                fresh = fresh.clone()
                fresh[:, 0, :kept] = 0
            scale = _block_scale(fresh.amax(dim=(2, 3)))
            if kept:
                scale[:, 0] = torch.maximum(scale[:, 0], scales[:, i])
            scale = scale[:, :, None, None]
            value = (full / scale).to(torch.float8_e4m3fn).float() * scale
            value = value.reshape(heads, -1, d)[:, :kept + n]
            out[i][cu_all[b] + base:cu_all[b + 1]] = value.transpose(0, 1).to(dt)
    return out


def run(s):
    if own:
        from exact_attention_deberta_gb300 import binding
        if s["op"] == "rotary":
            return binding.df_rotary(s["x"], s["pos"], s["table"], interleaved=s["inter"], inverse=s["inverse"],
                                     amplitude=s["amplitude"])
        if s["op"] in ("self", "self_train"):
            kw = dict(key_mask=s["mask"], cu_seqlens_q=s["cu_q"], cu_seqlens_k=s["cu_k"], max_seqlen_q=s["Lq"],
                      max_seqlen_k=s["Lk"], window=s["window"], sinks=s["sinks"])
            if s["op"] == "self":
                return binding.df_self_attn_fwd(s["q"], s["k"], s["v"], **kw)
            out, stats = binding.df_self_attn_fwd(s["q"], s["k"], s["v"], with_stats=True, **kw)
            dq, dk, dv = binding.df_self_attn_bwd(s["q"], s["k"], s["v"], out, stats, s["dout"], **kw)
            return {"out": out, "dq": dq, "dk": dk, "dv": dv}
        if s["op"] == "cache_store":
            binding.df_cache_append(s["k"], s["v"], s["cache"], s["table"], s["held"], s["cu"])
            return binding.df_cache_read(s["cache"], s["table"], s["ends"], s["cu_all"], rows=s["total"],
                                         dtype=s["dtype"])
        return binding.df_cache_attn(s["q"], s["cache"], s["table"], s["held"], max_length=s["L"], causal=s["causal"],
                                     window=s["window"], sinks=s["sinks"])
    if s["op"] == "rotary":
        return _plain_rotary(s)
    if s["op"] in ("self", "self_train"):
        return _plain_self(s)
    return _plain_store(s) if s["op"] == "cache_store" else _plain_cache(s)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rotary":
        rows = float(case["T"]) * (case["H"] + case["Hk"])
        return {"bytes": 2.0 * rows * case["d"] * size + 4.0 * case["T"], "flops": 3.0 * rows * case["rot"]}
    if case["op"] in ("self", "self_train"):
        nq, nk = _self_lengths(case)
        H, Hk, d = case["H"], case["Hk"], case["d"]
        if case["layout"] == "masked":
            # keys behind a sequence's length are not read; its padded rows see all of the others
            nk = [n for n in _ragged(case["B"], case["Lk"], 5)]
            if case["empty"] and case["B"] > 1:
                nk[-1] = 0
            pairs = 0.0
            for n in nk:
                p = torch.arange(case["Lk"] - case["Lq"], case["Lk"], dtype=torch.int64)
                top = torch.minimum(p + 1, torch.tensor(n))
                low = (p + 1 - case["window"]).clamp(min=0) if case["window"] else torch.zeros_like(p)
                pairs += float(((top - low).clamp(min=0) + torch.minimum(torch.minimum(low, top),
                                torch.tensor(case["sinks"]))).sum())
        else:
            pairs = _pairs(nq, nk, case["window"], case["sinks"])
        rows_q, rows_k = sum(nq) * H * d * 2.0, sum(nk) * Hk * d * 2.0
        if case["op"] == "self":
            return {"bytes": 2 * rows_q + 2 * rows_k, "flops": 4.0 * pairs * H * d}
        return {"bytes": 4 * rows_q + 4 * rows_k, "flops": 14.0 * pairs * H * d}
    held, new = _cache_lengths(case)
    Hk, d = case["Hk"], case["d"]
    if case["op"] == "cache_store":
        # the new rows in 16 bits in, as 8 bits out; all rows in 8 bits in, in 16 out
        rows, every = float(sum(new)) * Hk * d, float(sum(held) + sum(new)) * Hk * d
        return {"bytes": 2 * (3.0 * rows + 3.0 * every), "flops": 4.0 * rows + 2.0 * every}
    n, H = case["Lq"], case["H"]
    keys = 0.0
    for m in held:
        low = max(0, m - n + 1 - case["window"]) if case["window"] else 0
        keys += m - low + min(low, case["sinks"])
    pairs = _pairs(new, held, case["window"], case["sinks"]) if case["causal"] else float(sum(held) * n)
    return {"bytes": keys * Hk * (2.0 * d + 0.5) + 4.0 * case["B"] * n * H * d, "flops": 4.0 * pairs * H * d}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _exact_codes():
    """The values of the 256 e4m3 codes."""
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(math.nan if (c & 127) == 127 else -x if c & 128 else x)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def _power(e):
    """2^e in 64 bits, by its bits (no function that could round)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_round(x):
    """Nearest e4m3 value, ties to the even code, for |x| <= 448."""
    _, e = torch.frexp(x)
    step = _power((e - 4).clamp(min=-9))
    return torch.round(x / step) * step


def _exact_read(s, b, n):
    """Positions 0 .. n - 1 of sequence b from the records, [n, heads, d], token after token."""
    cache, page, d, codes = s["cache"], s["page"], s["d"], _exact_codes()
    pos = torch.arange(n, device="cuda")
    rec = cache[s["table"][b][pos // page].long(), :, (pos % page) // BLOCK]  # [n, heads, bytes]
    col = torch.arange(d, device="cuda")
    where = (col // 32 * 512 + col % 32)[None, None, :] + (pos % BLOCK * 32)[:, None, None]
    where = where.expand(n, cache.shape[1], d)
    return [codes[rec.gather(2, where + 16 * d * i).long()] *
            rec[..., 32 * d + 4 * i:32 * d + 4 * i + 4].contiguous().view(torch.float32).double() for i in range(2)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        r, out = case["rot"], []
        freq = _frequencies(r, case["factor"], case["far"]).cuda()
        z = torch.polar(torch.full((case["T"], r // 2), s["amplitude"], dtype=torch.float64, device="cuda"),
                        s["pos"].double()[:, None] * freq)
        z = z.conj() if case["inverse"] else z
        at = torch.arange(r // 2, device="cuda")
        a, b = (2 * at, 2 * at + 1) if case["inter"] else (at, at + r // 2)
        for x in s["x"]:
            y = x.double()
            w = torch.complex(y[..., a], y[..., b]) * z[:, None, :]
            y[..., a], y[..., b] = w.real, w.imag
            out.append(y)
        return out
    if case["op"] in ("self", "self_train"):
        H, Hk, d = case["H"], case["Hk"], case["d"]
        G, train = H // Hk, case["op"] == "self_train"
        cost = float(sum(a * b for a, b in zip(s["nq"], s["nk"]))) * H * d * (14.0 if train else 4.0)
        if cost > 1.2e13:
            return None
        q, k, v = (s[n].reshape(-1, s[n].shape[-2], d) for n in ("q", "k", "v"))
        do = s["dout"].reshape(-1, H, d) if train else None
        out, dq = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
        dk, dv = (torch.zeros(k.shape, dtype=torch.float64, device="cuda") for _ in range(2))
        cq, ck = _offsets(s["nq"]), _offsets(s["nk"])
        for b, (n, m) in enumerate(zip(s["nq"], s["nk"])):
            if n == 0 or m == 0:
                continue
            i = torch.arange(n, device="cuda")[:, None] + (m - n)
            j = torch.arange(m, device="cuda")[None, :]
            hidden = j > i
            if case["window"]:
                hidden = hidden | ((i - j >= case["window"]) & (j >= case["sinks"]))
            if s["mask"] is not None:
                hidden = hidden | (s["mask"][b] == 0)[None, :]
            none = hidden.all(dim=1)
            for h in range(H):
                qs, ks, vs = q[cq[b]:cq[b + 1], h].double(), k[ck[b]:ck[b + 1], h // G].double(), \
                    v[ck[b]:ck[b + 1], h // G].double()
                p = torch.softmax((qs @ ks.T / math.sqrt(d)).masked_fill(hidden, -math.inf), dim=1)
                p = p.masked_fill(none[:, None], 0.0)
                o = p @ vs
                out[cq[b]:cq[b + 1], h] = o
                if not train:
                    continue
                gs = do[cq[b]:cq[b + 1], h].double()
                dv[ck[b]:ck[b + 1], h // G] += p.T @ gs
                dp = gs @ vs.T
                dp -= (gs * o).sum(dim=1, keepdim=True)
                dp *= p
                dp /= math.sqrt(d)
                dq[cq[b]:cq[b + 1], h] = dp @ ks
                dk[ck[b]:ck[b + 1], h // G] += dp.T @ qs
        if not train:
            return out.view(s["q"].shape)
        return {"out": out.view(s["q"].shape), "dq": dq.view(s["q"].shape), "dk": dk.view(s["k"].shape),
                "dv": dv.view(s["v"].shape)}
    if case["op"] == "cache_store":
        held, new = s["n"]
        cu, both = _offsets(new), [[], []]
        for b, (m, n) in enumerate(zip(held, new)):
            old = _exact_read(s, b, m) if m else None
            for i, x in enumerate((s["k"], s["v"])):
                rows = x[cu[b]:cu[b + 1]].double()
                if m:
                    rows = torch.cat((old[i], rows))
                first = m // BLOCK  # the first block that takes new rows
                rows, done = rows[first * BLOCK:], rows[:first * BLOCK]
                blk = torch.arange(rows.shape[0], device="cuda") // BLOCK
                top = torch.zeros(int(blk[-1]) + 1, rows.shape[1], dtype=torch.float64, device="cuda")
                kept = m - first * BLOCK
                top.index_reduce_(0, blk[kept:], rows[kept:].abs().amax(dim=2), "amax")
                # top / 448 <= 2^e
                part, e = torch.frexp(top / 7.0)
                e = torch.where(part > 0.5, e, e - 1) - 6
                unit = _power(torch.where(top > 0, e, -100).clamp(min=-100))
                # (the quotient is rounded, by less than the distance of two inputs)
                if kept:
                    rec = s["cache"][s["table"][b, m // case["page"]].long(), :, (m % case["page"]) // BLOCK]
                    at = 32 * case["d"] + 4 * i
                    unit[0] = torch.maximum(unit[0], rec[:, at:at + 4].contiguous().view(torch.float32).double()[:, 0])
                u = unit[blk][:, :, None]
                both[i].append(torch.cat((done, _exact_round(rows / u) * u)))
        return [torch.cat(x) for x in both]
    H, Hk, d, n = case["H"], case["Hk"], case["d"], case["Lq"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, m in enumerate(s["n"]):
        k, v = (x.repeat_interleave(H // Hk, dim=1) for x in _exact_read(s, b, m))
        w = torch.einsum("ihc,jhc->hij", s["q"][b].double(), k) / math.sqrt(d)
        if case["causal"]:
            i = torch.arange(m - n, m, device="cuda")[:, None]
            j = torch.arange(m, device="cuda")[None, :]
            hidden = j > i
            if case["window"]:
                hidden = hidden | ((i - j >= case["window"]) & (j >= case["sinks"]))
            w = w.masked_fill(hidden, -math.inf)
        out[b] = torch.einsum("hij,jhc->ihc", torch.softmax(w, dim=2), v)
    return out
