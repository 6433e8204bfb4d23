"""Cross-attention gradients beside a dout that is not finite: rows and keys that have no
part in it keep their results, and keys that do not count get zeros all the same."""

import pytest
import torch

from _cross import call, call_bwd, inputs, to_dev

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d,G", [(64, 1), (128, 2)])
def test_keys_that_do_not_count_get_zeros(lib, d, G, dtype, junk):
    x = inputs(3, 2 * G, 2, d, 70, 300, dtype, "padded", "masked", seed=d, nk=[300, 40, 131])
    dev = to_dev(x)
    out, stats = call(lib, x, dev, with_stats=True)
    clean = call_bwd(lib, x, dev, out, stats)
    dev["dout"][0, 7, 0, 3] = junk
    dirty = call_bwd(lib, x, dev, out, stats)
    off = dev["key_mask"] == 0
    for c, t in zip(clean[1:], dirty[1:]):
        assert int((t[off] != 0).sum()) == 0
        assert torch.equal(t[1:], c[1:])  # the other sequences
        assert torch.equal(t[0, :, 1], c[0, :, 1])  # the other key head
        assert bool((~t[0, :, 0].isfinite()).any(dim=-1)[~off[0]].all())
    rest = torch.ones(3, 70, 2 * G, dtype=torch.bool, device="cuda")
    rest[0, 7, 0] = False
    assert torch.equal(dirty[0][rest], clean[0][rest]) and not bool(dirty[0][0, 7, 0].isfinite().all())
