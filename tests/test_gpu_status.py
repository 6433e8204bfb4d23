"""What the encoder's and the reader's layers report through a status word."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_layers_report_bad_ids_and_offsets(lib):
    from exact_attention_deberta_gb300.encoder import (CrossAttention, Encoder, EncoderConfig,
                                                       synthetic_cross_weights, synthetic_weights)
    cfg = EncoderConfig(hidden=256, heads=4, layers=0, vocab=50)
    enc = Encoder(cfg, *synthetic_weights(cfg))
    cross = CrossAttention(cfg, synthetic_cross_weights(cfg))
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = (torch.arange(40) % 50).cuda()
    x = enc.embed(ids, status=word)
    k, v = cross.project(x, status=word)
    cu = torch.tensor([0, 15, 40], dtype=torch.int32).cuda()
    good = cross.attend(x, k, v, cu, 25, cu, 25, status=word)
    assert int(word.item()) == lib.DF_OK
    assert torch.equal(good, cross.attend(x, k, v, cu, 25, cu, 25))
    ids[7] = 50
    enc.embed(ids, status=word)
    assert int(word.item()) == lib.DF_ERR_INVALID_ARG
    for bad in ([0, 15, 41], [0, 41, 40], [-1, 15, 40]):
        bad = torch.tensor(bad, dtype=torch.int32).cuda()
        for q_cu, k_cu in ((bad, cu), (cu, bad)):
            word.zero_()
            cross.attend(x, k, v, q_cu, 25, k_cu, 25, status=word)
            assert int(word.item()) == lib.DF_ERR_INVALID_ARG
