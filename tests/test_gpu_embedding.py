"""GPU parity of the embedding lookup and of its table's gradient against the
float64 oracle on the same rounded inputs, with bounds counted in roundings."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
U32 = 2.0 ** -24  # one fp32 rounding


def _np(t):
    return t.double().cpu().numpy()


def _ids(T, V, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    if kind == "same":
        return np.full(T, V - 1, dtype=np.int64)
    if kind == "all":
        return rng.permutation(np.arange(T, dtype=np.int64) % V)
    few = rng.integers(0, min(V, 3), T)  # a few very frequent ids among rare ones
    return np.where(rng.random(T) < 0.5, few, rng.integers(0, V, T)).astype(np.int64)


def _check_lookup(out, ids, table, scale):
    want = oracle.embed(ids, _np(table), scale)
    info = torch.finfo(table.dtype)
    # the fp32 product, then the rounding to the type (below its normal range an
    # absolute half step)
    tol = (info.eps / 2 + 2 * U32) * np.abs(want) + info.tiny * info.eps / 2
    assert (np.abs(_np(out) - want) <= tol).all()


def _check_grad(got, ids, dout, V, scale, pad, base=None):
    want, mass, count = oracle.embed_grad(ids, _np(dout) if isinstance(dout, torch.Tensor) else dout, V,
                                          float(np.float32(scale)), pad, base)
    # n additions in fp32, the product with the scale and the sum with the base:
    # at most (n + 2) roundings of partial sums that `mass` bounds
    tol = (count[:, None] + 2) * U32 * mass * (1 + 1e-3) + 1e-37
    err = np.abs(_np(got) - want)
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("T,N,V,dtype,scale", [
    (1, 8, 1, BF, 1.0), (1, 768, 1000, FP, 0.5), (48, 768, 5000, BF, 1.0), (333, 520, 77, HF, 27.7),
    (1000, 2056, 10, FP, -1.5), (4097, 72, 40000, BF, 3.0)])
@pytest.mark.parametrize("wide", [False, True])
def test_lookup_matches_oracle(lib, T, N, V, dtype, scale, wide):
    ids = _ids(T, V, T + N)
    g = torch.Generator().manual_seed(N)
    table = torch.randn(V, N, generator=g).to(dtype).cuda()
    dev = torch.from_numpy(ids).to(torch.int64 if wide else torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lib.df_embedding(dev, table, scale=scale, status=status)
    _check_lookup(out, ids, table, float(np.float32(scale)))
    assert int(status.item()) == lib.DF_OK


def test_lookup_shapes_and_ids_outside_the_table(lib):
    table = torch.randn(9, 64).cuda()
    ids = torch.tensor([[0, 8, -1], [9, 3, 2 ** 33]], dtype=torch.int64).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lib.df_embedding(ids, table, status=status)
    assert tuple(out.shape) == (2, 3, 64)
    _check_lookup(out, ids.cpu().numpy(), table, 1.0)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG
    assert tuple(lib.df_embedding(ids[:, :0].contiguous(), table).shape) == (2, 0, 64)
    with pytest.raises(lib.DFError):
        lib.df_embedding(ids, torch.zeros(4, 12).cuda())
    with pytest.raises(ValueError):
        lib.df_embedding(ids, table, out=torch.empty(2, 3, 64, dtype=HF, device="cuda"))
    with pytest.raises(ValueError):
        lib.df_embedding(ids.t(), table)


GRADS = [  # T, N, V, dtype, scale, padding id, kind of ids
    (1, 8, 1, BF, 1.0, None, "mixed"), (31, 264, 5, FP, 0.5, None, "mixed"), (32, 64, 2, HF, 1.0, 1, "mixed"),
    (33, 256, 3, BF, 2.0, 0, "mixed"), (2048, 24, 100, FP, 1.0, None, "all"), (2049, 768, 1023, BF, 27.7, 1, "mixed"),
    (5000, 520, 1024, HF, 1.0, None, "mixed"), (3000, 768, 50021, BF, 1.0, 0, "mixed"),
    (9000, 40, 4, BF, 1.0, None, "same"), (4096, 8, 1100000, FP, 1.0, 7, "mixed"), (700, 72, 700, HF, 1.0, None, "all"),
    (64, 64, 9, FP, 1.0, 8, "same")]


@pytest.mark.parametrize("T,N,V,dtype,scale,pad,kind", GRADS)
def test_gradient_matches_oracle(lib, T, N, V, dtype, scale, pad, kind):
    ids = _ids(T, V, T + V, kind)
    g = torch.Generator().manual_seed(T)
    dout = torch.randn(T, N, generator=g).to(dtype).cuda()
    dev = torch.from_numpy(ids).to(torch.int32 if T % 2 else torch.int64).cuda()
    ws = torch.full((lib.df_embedding_bwd_workspace_size(T, N, V),), 0xFF, dtype=torch.uint8, device="cuda")
    grad = torch.full((V, N), float("nan"), device="cuda")
    lib.df_embedding_bwd(dev, dout, V, scale=scale, padding_idx=pad, grad=grad, workspace=ws)
    _check_grad(grad, ids, dout, V, scale, pad)
    again = lib.df_embedding_bwd(dev, dout, V, scale=scale, padding_idx=pad)
    assert torch.equal(grad, again)


def test_gradient_is_added_to_where_asked(lib):
    T, N, V = 700, 136, 60
    ids = _ids(T, V, 3)
    ids[ids == 11] = 12
    dout = torch.randn(T, N).to(BF).cuda()
    base = torch.randn(V, N).cuda()
    base[11] = float("nan")  # a row that no token reaches is not touched
    grad = base.clone()
    got = lib.df_embedding_bwd(torch.from_numpy(ids).cuda(), dout, V, scale=0.5, grad=grad, accumulate=True)
    assert got.data_ptr() == grad.data_ptr()
    assert torch.isnan(grad[11]).all()
    grad[11], base[11] = 0.0, 0.0
    _check_grad(grad, ids, dout, V, 0.5, None, _np(base))
    with pytest.raises(ValueError, match="accumulate"):
        lib.df_embedding_bwd(torch.from_numpy(ids).cuda(), dout, V, accumulate=True)


@pytest.mark.parametrize("T", [1, 2048, 2049, 8192, 8193, 65536, 65537])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_around_the_sorts_limits(lib, T, accumulate):
    # whole sums of small integers are exact in fp32, whatever their order
    N, V = 8, 3001
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, V, (T,), generator=g)
    dout = torch.randint(-4, 5, (T, N), generator=g).to(BF)
    want = torch.zeros(V, N, dtype=torch.float64).index_add_(0, ids, dout.double())
    grad = torch.full((V, N), 3.0, device="cuda")
    lib.df_embedding_bwd(ids.cuda(), dout.cuda(), V, grad=grad, accumulate=accumulate)
    assert torch.equal(grad.cpu().double(), want + 3.0 if accumulate else want)


def test_padding_and_outside_rows_may_hold_anything(lib):
    ids = np.array([3, 0, -7, 5, 0, 3, 99, 5], dtype=np.int64)
    dout = torch.randn(8, 64)
    clean = _np(dout)
    for t in (1, 2, 4, 6):
        dout[t] = float("nan") if t % 2 else float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grad = lib.df_embedding_bwd(torch.from_numpy(ids).cuda(), dout.cuda(), 9, padding_idx=0, status=status)
    _check_grad(grad, ids, clean, 9, 1.0, 0)
    assert int(status.item()) == lib.DF_ERR_INVALID_ARG
    empty = lib.df_embedding_bwd(torch.zeros(0, dtype=torch.int32).cuda(), torch.zeros(0, 64).cuda(), 9)
    assert tuple(empty.shape) == (9, 64) and int((empty != 0).sum()) == 0


def test_other_stream_and_captured_replay(lib):
    T, N, V = 3000, 256, 2000
    ids = torch.from_numpy(_ids(T, V, 8)).cuda()
    dout = torch.randn(T, N).to(BF).cuda()
    table = torch.randn(V, N).to(BF).cuda()
    ws = torch.empty(lib.df_embedding_bwd_workspace_size(T, N, V), dtype=torch.uint8, device="cuda")
    grad, out = torch.empty(V, N, device="cuda"), torch.empty(T, N, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lib.df_embedding(ids, table, out=out)
        lib.df_embedding_bwd(ids, dout, V, grad=grad, workspace=ws)
    new = _ids(T, V, 9, "all")
    ids.copy_(torch.from_numpy(new))
    dout.copy_(torch.randn(T, N))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    _check_lookup(out, new, table, 1.0)
    _check_grad(grad, new, dout, V, 1.0, None)
    with torch.cuda.stream(side):
        other = lib.df_embedding_bwd(ids, dout, V)
    side.synchronize()
    assert torch.equal(other, grad)


def test_ids_that_change_meanwhile_do_no_harm(lib):
    # which of the ids a gradient counts is then open, but nothing is read or written
    # outside the tensors, and the next call is right
    T, N, V = 40000, 64, 5000
    g = torch.Generator().manual_seed(2)
    dout = torch.randn(T, N, generator=g).to(torch.bfloat16).cuda()
    choices = [torch.randint(0, V, (T,), generator=g).cuda(), torch.full((T,), 3, device="cuda"),
               torch.full((T,), 1 << 40, device="cuda")]
    ids = choices[0].clone()
    guard = torch.zeros(V + 64, N, device="cuda")
    guard[V:] = 7.0
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k in range(30):
        lib.df_embedding_bwd(ids, dout, V, grad=guard[:V])
        with torch.cuda.stream(other):
            for c in choices:
                ids.copy_(c)
    torch.cuda.synchronize()
    assert bool((guard[V:] == 7.0).all())
    ids.copy_(choices[0])
    torch.cuda.synchronize()
    got = lib.df_embedding_bwd(ids, dout, V, grad=guard[:V])
    assert torch.equal(got, lib.df_embedding_bwd(choices[0], dout, V))


def test_offsets_beyond_32_bits(lib):
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    N = 2048
    V = (1 << 32) // N + 40
    table = torch.zeros(V, N, dtype=BF, device="cuda")
    table[-40:] = torch.randn(40, N, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    ids = torch.cat([torch.arange(V - 40, V), torch.arange(V - 20, V), torch.zeros(3, dtype=torch.int64)]).cuda()
    out = lib.df_embedding(ids, table)
    assert torch.equal(out, table[ids])
    grad = lib.df_embedding_bwd(ids, out, V)
    want = torch.zeros(40, N, device="cuda")
    want += table[-40:].float()
    want[20:] *= 2
    assert torch.equal(grad[-40:], want) and int(grad[:-40].count_nonzero()) == 0
    del grad
    # and many tokens: those behind 2^32 values of dout reach two rows
    T = V
    ids = torch.full((T,), 5, dtype=torch.int32, device="cuda")
    ids[-40:] = 7
    grad = lib.df_embedding_bwd(ids, table, 9)
    assert int(grad[:7].count_nonzero()) == 0 and int(grad[8].count_nonzero()) == 0
    # 40 additions, of partial sums below 64
    assert torch.allclose(grad[7].double(), table[-40:].double().sum(0), rtol=0, atol=40 * 64 * 2.0 ** -24)
