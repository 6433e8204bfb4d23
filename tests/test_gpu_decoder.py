"""The decoder's operators together, as they are used: a training step through rotary positions
and causal attention, prompts and generation through a SelfAttention layer and its cache, and a
CrossAttention layer that reads stored states."""

import numpy as np
import pytest
import torch

import oracle
from _cache import offsets, table_of
from _cross import check_forward, np64

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype,d,rot,interleaved", [(BF, 64, 64, False), (HF, 128, 48, True)])
def test_training_step_through_positions_and_attention(lib, dtype, d, rot, interleaved):
    """Gradients of q, k before their rotation, against float64 through the rounded rotated rows:
    what the call's own rounding of those adds is bounded by the attention's tests."""
    g = torch.Generator().manual_seed(d)
    H, Hk, lens = 4, 2, [150, 31, 260]
    T = sum(lens)
    q, k, v, do = (torch.randn(T, h, d, generator=g).to(dtype) for h in (H, Hk, Hk, H))
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32)
    cu = offsets(lens).cuda()
    table = lib.df_rotary_table(rot)
    kw = dict(cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=max(lens), max_seqlen_k=max(lens), window=70, sinks=2)
    at = pos.cuda()
    qr, kr = lib.df_rotary((q.cuda(), k.cuda()), at, table, interleaved=interleaved)
    out, stats = lib.df_self_attn_fwd(qr, kr, v.cuda(), with_stats=True, **kw)
    dqr, dkr, dv = lib.df_self_attn_bwd(qr, kr, v.cuda(), out, stats, do.cuda(), **kw)
    dq, dk = lib.df_rotary((dqr, dkr), at, table, interleaved=interleaved, inverse=True)
    w = oracle.causal_batch(np64(qr), np64(kr), np64(v), d ** -0.5, 70, 2, cu_q=cu.cpu().numpy(), cu_k=cu.cpu().numpy(),
                            dout=np64(do))
    check_forward(out, w, dtype, d, stats.lse, stats.out_lo)
    angles = oracle.rotary_angles(pos.tolist(), table.tolist())
    half = torch.finfo(dtype).eps / 2
    for got, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        ref = w[name] if name == "dv" else oracle.rotary(w[name], angles, interleaved, inverse=True)[0]
        norm = lambda z: float(np.sqrt((z ** 2).sum()))  # noqa: E731
        # the backward's three roundings, half a step each (as its own test counts them), and
        # one more of the rotated gradient
        assert norm(np64(got) - ref) <= 4 * half * norm(ref) + 1e-4 * norm(w[name + "_mass"]), name


def held(lib, cache, table, lengths):
    """The cache's tokens of each sequence, in float64."""
    n = [int(x) for x in lengths.tolist()]
    k, v = lib.df_cache_read(cache, table, lengths, offsets(n).cuda(), rows=sum(n), dtype=torch.float32)
    ends = np.cumsum(n)[:-1]
    return list(zip(np.split(np64(k), ends), np.split(np64(v), ends)))


@pytest.mark.parametrize("heads,key_heads,window,sinks,n", [(8, 8, 0, 0, 1), (8, 4, 60, 3, 2)])
def test_prompt_and_generation(lib, heads, key_heads, window, sinks, n):
    from exact_attention_deberta_gb300 import encoder
    cfg = encoder.EncoderConfig(hidden=64 * heads, heads=heads)
    layer = encoder.SelfAttention(cfg, encoder.synthetic_self_weights(cfg, key_heads, seed=1), lib.df_rotary_table(64),
                                  key_heads=key_heads, window=window, sinks=sinks)
    lens, page, steps, B = [130, 17, 64], 16, 20, 3
    g = torch.Generator().manual_seed(2)
    T = sum(lens)
    x = torch.randn(T, cfg.hidden, generator=g).to(BF).cuda()
    pos = torch.cat([torch.arange(m) for m in lens]).to(torch.int32).cuda()
    cu = offsets(lens).cuda()
    ends = [m + steps * n for m in lens]
    n_pages = sum(-(-m // page) for m in ends) + 1
    cache, table = lib.df_cache_new(n_pages, key_heads, page, 64), table_of(ends, page, n_pages, 3).cuda()
    cache.fill_(0xFF)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    trace = []
    y = layer.prompt(x, pos, cu, max(lens), cache, table, status=status, trace=trace)
    assert torch.equal(layer.prompt(x, pos, cu, max(lens)), y) and bool(torch.isfinite(y).all())
    t = trace[0]
    w = oracle.causal_batch(np64(t["q"]), np64(t["k"]), np64(t["v"]), 0.125, window, sinks, cu_q=cu.cpu().numpy(),
                            cu_k=cu.cpu().numpy())
    check_forward(t["ctx"], w, BF, 64)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # what is held: the rotated keys and the values within half a code of their block's scale
    at = 0
    for (kk, vv), m in zip(held(lib, cache, table, lengths), lens):
        for got, ref in ((kk, np64(t["k"])[at:at + m]), (vv, np64(t["v"])[at:at + m])):
            assert (np.abs(got - ref) <= np.maximum(np.abs(ref) * 2.0 ** -4, np.abs(ref).max() * 2.0 ** -17)).all()
        at += m
    for _ in range(steps):
        z = torch.randn(B, n, cfg.hidden, generator=g).to(BF).cuda()
        p = (lengths[:, None] + torch.arange(n, device="cuda", dtype=torch.int32)[None, :]).contiguous()
        trace = []
        y = layer.step(z, p, cache, table, lengths, status=status, trace=trace)
        lengths += n
        assert y.shape == z.shape and bool(torch.isfinite(y).all())
    t = trace[0]
    rows = [oracle.causal_rows(np64(t["q"][b]), *held(lib, cache, table, lengths)[b], np.ones(int(lengths[b]), bool), 0.125,
                               window, sinks) for b in range(B)]
    w = {name: np.concatenate([r[name] for r in rows]) for name in rows[0]}
    check_forward(t["ctx"].view(-1, heads, 64), w, BF, 64)
    assert int(status.item()) == lib.DF_OK


def test_generation_continues_the_prompt(lib):
    """The last token of a prompt, given as a step after the others, comes out as in the prompt
    but for the cache's 8 bits."""
    from exact_attention_deberta_gb300 import encoder
    cfg = encoder.EncoderConfig(hidden=512, heads=8)
    layer = encoder.SelfAttention(cfg, encoder.synthetic_self_weights(cfg, seed=4), lib.df_rotary_table(64), window=40, sinks=2)
    x = torch.randn(100, 512, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    ta, tb = [], []
    layer.prompt(x, pos, offsets([100]).cuda(), 100, trace=ta)
    cache, table = lib.df_cache_new(8, 8, 16, 64), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    layer.prompt(x[:99].contiguous(), pos[:99].contiguous(), offsets([99]).cuda(), 99, cache, table)
    layer.step(x[99:].view(1, 1, 512).contiguous(), pos[99:].view(1, 1).contiguous(), cache, table,
               torch.tensor([99], dtype=torch.int32, device="cuda"), trace=tb)
    q, k, v = (np64(ta[0][n]) for n in "qkv")
    w = oracle.causal_rows(q[99:], k, v, np.ones(100, bool), 0.125, 40, 2)
    got = np64(tb[0]["ctx"])[0]
    # codes are off by 2^-4 of a value at most: scores by 2^-4 of their mass, values by theirs
    s = 2.0 ** -4 * w["score_mass"]
    bound = (np.exp(2 * s)[..., None] * (1 + 2.0 ** -4) - 1) * w["out_mass"] + 2.0 ** -8 * np.abs(w["out"]) + 2.0 ** -8 * w["out_mass"]
    assert (np.abs(got - w["out"]) <= bound).all()


@pytest.mark.parametrize("rows", [1, 3])
def test_cross_attention_to_stored_states(lib, rows):
    from exact_attention_deberta_gb300 import encoder
    cfg = encoder.EncoderConfig(hidden=512, heads=8)
    layer = encoder.CrossAttention(cfg, encoder.synthetic_cross_weights(cfg, seed=6))
    lens, page = [200, 0, 77], 32
    g = torch.Generator().manual_seed(7)
    states = torch.randn(sum(lens), 512, generator=g).to(BF).cuda()
    n_pages = 12
    cache, table = lib.df_cache_new(n_pages, 8, page, 64), table_of(lens, page, n_pages, 8).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    layer.store(states, cache, table, offsets(lens).cuda(), status=status)
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x = torch.randn(3 * rows, 512, generator=g).to(BF).cuda()
    cu = offsets([rows] * 3).cuda()
    y = layer.attend_stored(x, cache, table, lengths, cu if rows > 1 else None, rows, status=status)
    # the same layer on the values that the cache stands for, as 16-bit keys
    k, v = lib.df_cache_read(cache, table, lengths, offsets(lens).cuda(), rows=sum(lens))
    ref = layer.attend(x, k, v, cu, rows, offsets(lens).cuda(), 200)
    # both round weights and results to 16 bits: a step or two of the normalised rows
    assert float((y.float() - ref.float()).abs().max()) <= 4 * 2.0 ** -8 * float(ref.float().abs().max())
    assert int(status.item()) == lib.DF_OK


def test_calls_on_a_side_stream_with_current_allocations(lib):
    """Given streams: the results are those of the default stream, whatever runs there meanwhile."""
    q = torch.randn(2, 1, 8, 64, device="cuda").to(BF)
    k, v = torch.randn(2, 90, 8, 64, device="cuda").to(BF), torch.randn(2, 90, 8, 64, device="cuda").to(BF)
    table, rot = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6), lib.df_rotary_table(64)
    zero, held90 = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.full((2,), 90, dtype=torch.int32, device="cuda")
    pos = torch.arange(180, dtype=torch.int32, device="cuda").view(2, 90)

    def chain(**s):
        cache = lib.df_cache_new(12, 8, 16, 64)
        kr = lib.df_rotary(k, pos, rot, **s)
        lib.df_cache_append(kr, v, cache, table, zero, **s)
        a = lib.df_cache_attn(q, cache, table, held90, **s)
        kk, vv = lib.df_cache_read(cache, table, held90, rows=90, **s)
        return a, lib.df_self_attn_fwd(q, kk, vv, window=30, **s)

    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
    with torch.cuda.stream(side):
        got = chain(stream=side)
    del junk
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
