"""Embedding calls of many tokens: the lookup's four rows per warp, which begin at 256 tokens
for each SM, and the gradient's chunks of 32 sorted entries, in every type, against
the float64 oracle with bounds counted in roundings."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
U32 = 2.0 ** -24


def _switch():
    return 4 * 64 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("more", [-1, 0, 1, 2, 3, 29])
@pytest.mark.parametrize("dtype,wide,N", [(BF, False, 264), (HF, True, 8), (FP, False, 40), (FP, True, 264)])
def test_lookup_of_many_tokens(lib, more, dtype, wide, N):
    T, V = _switch() + more, 3001
    rng = np.random.default_rng(T + N)
    ids = rng.integers(0, V, T)
    # ids outside the table at every place of a group of four, among the first and the last
    for at in (0, 5, 10, 15, T - 1, T - 2, T - 7, T - 12):
        ids[at] = rng.choice([-1, V, 2 ** 31 - 1, -2 ** 31])
    if wide:
        ids[21] = 2 ** 40 + 3
    table = torch.randn(V, N, generator=torch.Generator().manual_seed(N)).to(dtype)
    table[0] = float("nan")  # the row that stands in for an id outside
    ids[ids == 0] = 1
    dev = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    room = torch.full((T + 64, N), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lib.df_embedding(dev, table.cuda(), scale=1.7, out=room[:T], status=status)
    table[0] = 0.0
    want = oracle.embed(ids, table.double().numpy(), float(np.float32(1.7)))
    info = torch.finfo(dtype)
    tol = (info.eps / 2 + 2 * U32) * np.abs(want) + info.tiny * info.eps / 2
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    assert bool((room[T:] == 7.0).all()) and int(status.item()) == lib.DF_ERR_INVALID_ARG
    status.zero_()
    lib.df_embedding(dev[40:T - 40].contiguous(), table.cuda(), status=status)
    assert int(status.item()) == lib.DF_OK


@pytest.mark.parametrize("T,V", [(32769, 700), (40007, 60000), (65537, 90)])
@pytest.mark.parametrize("dtype,N", [(HF, 264), (FP, 264), (BF, 520), (FP, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_of_many_tokens(lib, T, V, dtype, N, accumulate):
    rng = np.random.default_rng(T + N)
    ids = np.where(rng.random(T) < 0.4, 3, rng.integers(0, V, T))  # one id in long runs
    dout = torch.randn(T, N, generator=torch.Generator().manual_seed(T)).to(dtype)
    base = torch.randn(V, N, generator=torch.Generator().manual_seed(1)) if accumulate else torch.full((V, N), float("nan"))
    grad = lib.df_embedding_bwd(torch.from_numpy(ids).cuda(), dout.cuda(), V, scale=0.75, padding_idx=5, grad=base.cuda(),
                                accumulate=accumulate)
    d = dout.double() * 0.75
    d[torch.from_numpy(ids == 5)] = 0.0
    at = torch.from_numpy(ids)
    zero = lambda: (base.double() if accumulate else torch.zeros(V, N, dtype=torch.float64))  # noqa: E731
    want, mass = zero().index_add_(0, at, d), zero().abs().index_add_(0, at, d.abs())
    count = torch.bincount(at, minlength=V)[:, None]
    # n additions in fp32 of partial sums that `mass` bounds, the product with the scale, the sum
    # with the base
    tol = (count + 2) * U32 * mass * (1 + 1e-3) + 1e-37
    assert bool(((grad.cpu().double() - want).abs() <= tol).all())
