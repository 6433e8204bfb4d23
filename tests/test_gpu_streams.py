"""The encoder's and the reader's layers, and the calls around them, on a stream that
is given as an argument: freed blocks of theirs are not handed out to the current
stream while the given one still runs."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
def test_layers_on_a_stream_given_as_an_argument(lib, handle):
    from exact_attention_deberta_gb300.encoder import (CrossAttention, Encoder, EncoderConfig,
                                                       synthetic_cross_weights, synthetic_weights)
    cfg = EncoderConfig(hidden=512, heads=8, layers=2, ffn=1024, vocab=3000)
    layers, shared = synthetic_weights(cfg, seed=1)
    enc, cross = Encoder(cfg, layers, shared), CrossAttention(cfg, synthetic_cross_weights(cfg, seed=2))
    g = torch.Generator().manual_seed(3)
    src, tgt = torch.randint(0, 3000, (4000,), generator=g).cuda(), torch.randint(0, 3000, (900,), generator=g).cuda()
    cu_k = torch.tensor([0, 1500, 1600, 4000], dtype=torch.int32).cuda()
    cu_q = torch.tensor([0, 300, 500, 900], dtype=torch.int32).cuda()
    mask = (torch.rand(3, 400, generator=g) < 0.8).to(torch.uint8).cuda()
    rows = torch.randn(3, 400, 512, generator=g).to(torch.bfloat16).cuda()

    def run(**on):
        x = enc.embed(src, **on)
        states = enc(x, cu_k, 2400, **on)
        k, v = cross.project(states, **on)
        out = cross.attend(enc.embed(tgt, **on), k, v, cu_q, 400, cu_k, 2400, **on)
        packed, cu, info = lib.pack_padded_with_info(rows, mask, **on)
        back, _ = lib.unpack_packed(packed, cu, 400, info, **on)
        return x, states, k, v, out, packed, back

    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = sorted({t.numel() for t in want} | {4000 * 1024, 900 * 512, 4000 * 3 * 512})
    for _ in range(4):
        got = run(stream=side.cuda_stream if handle else side)
        # blocks of the same sizes on the current stream, written at once
        junk = [torch.full((n,), 9.0, dtype=torch.bfloat16, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 4 * len(sizes)


def test_the_default_stream_as_a_handle(lib):
    # its handle is 0: what is called on it runs there and belongs to it, whatever the
    # current stream is
    default, side = torch.cuda.default_stream(), torch.cuda.Stream()
    assert default.cuda_stream == 0
    x = torch.zeros(4, device="cuda")
    with torch.cuda.stream(side):
        for given in (0, default, default.cuda_stream):
            with lib._current(given, x):
                assert torch.cuda.current_stream() == default
        assert torch.cuda.current_stream() == side
    # ordered behind the work already there: the ids are written on the default stream
    table = torch.randn(50, 64, device="cuda")
    ids = torch.zeros(1 << 20, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        with torch.cuda.stream(default):
            torch.cuda._sleep(20_000_000)
            ids.fill_(7)
        out = lib.df_embedding(ids, table, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out[-1], table[7]) and bool((out == table[7]).all())
