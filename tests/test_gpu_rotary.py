"""GPU parity of rotary positions against the float64 oracle (angles from the same table, by
exact integers), within bounds counted in roundings."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def check(got, x, angles, dtype, **kw):
    y, mass = oracle.rotary(x.double().cpu().numpy(), angles, **kw)
    half = torch.finfo(dtype).eps / 2
    # sine and cosine: CUDA's 2 units of the last place (2^-24 each way of values below one:
    # 2^-23), the amplitude, the products and the sum: 2^-24 each; the angle is cut at 2^-32 turns
    inner = mass * (2.0 ** -22 + 3 * 2.0 ** -24 + 2.0 ** -29)
    tiny = 2.0 ** -25 if dtype == HF else 0.0
    err = np.abs(got.double().cpu().numpy() - y)
    assert (err <= inner + half * (np.abs(y) + inner) * (mass > 0) + tiny * (mass > 0)).all(), float(err.max())


CASES = [  # T, heads, d, rot, dtype
    (1, (1,), 64, 64, BF), (5, (12, 12), 64, 64, HF), (77, (4, 1), 128, 128, BF), (33, (3, 1), 80, 20, BF),
    (19, (2, 2), 80, 40, HF), (300, (8, 2), 96, 48, BF), (7, (3, 5), 24, 6, F32), (64, (5,), 128, 32, F32),
    (9, (2, 1), 33, 32, BF), (9, (2, 3), 5, 2, HF), (11, (17, 9), 64, 30, F32), (4000, (12, 12), 64, 64, BF)]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,heads,d,rot,dtype", CASES)
def test_matches_oracle(lib, T, heads, d, rot, dtype, interleaved, inverse):
    g = torch.Generator().manual_seed(T + d + rot)
    xs = [torch.randn(T, h, d, generator=g).to(dtype).cuda() for h in heads]
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    table = lib.df_rotary_table(rot, factor=2.0, original_len=1000.0)
    outs = lib.df_rotary(xs, pos.cuda(), table, interleaved=interleaved, inverse=inverse, amplitude=1.25)
    angles = oracle.rotary_angles(pos.tolist(), table.tolist())
    for x, y in zip(xs, outs):
        check(y, x, angles, dtype, interleaved=interleaved, inverse=inverse, amplitude=1.25)
        assert torch.equal(y[..., rot:], x[..., rot:])
    one = lib.df_rotary(xs[0], pos.cuda(), table, interleaved=interleaved, inverse=inverse, amplitude=1.25)
    assert torch.equal(one, outs[0])
    kept = [x.clone() for x in xs]
    same = lib.df_rotary(kept, pos.cuda(), table, interleaved=interleaved, inverse=inverse, amplitude=1.25, out=kept)
    assert all(a is b and torch.equal(a, o) for a, b, o in zip(same, kept, outs))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_and_negative_positions(lib, dtype):
    pos = torch.tensor([0, 1, -1, -12345, 4_000_001, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 3, -2 ** 62, 2 ** 63 - 1])
    g = torch.Generator().manual_seed(1)
    x = torch.randn(10, 3, 64, generator=g).to(dtype).cuda()
    table = lib.df_rotary_table(64)
    got = lib.df_rotary(x, pos.cuda(), table)
    check(got, x, oracle.rotary_angles(pos.tolist(), table.tolist()), dtype)
    small = pos[:7].to(torch.int32)
    assert torch.equal(lib.df_rotary(x[:7], small.cuda(), table), got[:7])


def test_every_eighth_of_a_turn(lib):
    # a table of exact turns: positions land on, next to and between the quarters
    table = torch.tensor([2 ** 61, 2 ** 61 - 1, 2 ** 29 + 1, -2 ** 62], dtype=torch.int64, device="cuda")
    pos = torch.arange(-20, 20, dtype=torch.int64, device="cuda")
    x = torch.randn(40, 2, 8, generator=torch.Generator().manual_seed(2)).cuda()
    check(lib.df_rotary(x, pos, table), x, oracle.rotary_angles(pos.tolist(), table.tolist()), F32)


def test_parts_of_a_fused_projection(lib):
    T, H, Hk, d = 50, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(2, T, (H + 2 * Hk) * d, generator=g).to(BF).cuda()
    parts = lambda t: (t[..., :H * d].unflatten(-1, (H, d)), t[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d)))  # noqa: E731
    pos = torch.arange(2 * T, dtype=torch.int64, device="cuda").view(2, T)
    table = lib.df_rotary_table(d)
    want = lib.df_rotary([t.contiguous() for t in parts(qkv)], pos, table)
    got = lib.df_rotary(parts(qkv), pos, table)
    assert all(o.is_contiguous() and torch.equal(o, w) for o, w in zip(got, want))
    mine = qkv.clone()
    lib.df_rotary(parts(mine), pos, table, out=parts(mine))
    assert all(torch.equal(o, w) for o, w in zip(parts(mine), want))
    assert torch.equal(mine[..., (H + Hk) * d:], qkv[..., (H + Hk) * d:])  # what lies between is left alone
    odd = torch.randn(T * 3 * d + 1, generator=g).to(BF).cuda()[1:].view(T, 3, d)  # rows off 16 bytes
    assert torch.equal(lib.df_rotary(odd, pos[0], table), lib.df_rotary(odd.clone(), pos[0], table))
    with pytest.raises(lib.DFError):
        lib.df_rotary(odd[1:], pos[0, 1:], table, out=odd[:-1])


def test_inverse_is_the_gradient(lib):
    g = torch.Generator().manual_seed(4)
    x, dy, step = (torch.randn(20, 3, 64, generator=g).cuda() for _ in range(3))
    pos = torch.arange(20, dtype=torch.int32, device="cuda") * 97
    table = lib.df_rotary_table(48)
    kw = dict(interleaved=True, amplitude=1.3)
    dx = lib.df_rotary(dy, pos, table, inverse=True, **kw)
    up, down = (lib.df_rotary(x + s * step, pos, table, **kw) for s in (0.5, -0.5))
    diff = ((up.double() - down.double()) * dy.double()).sum()  # linear: the difference is exact but for roundings
    total = (dx.double() * step.double()).sum()
    mass = float((dy.double().abs() * (x.double().abs() + step.double().abs())).sum()) * 2 * 1.3
    assert abs(float(diff - total)) <= 10 * 2.0 ** -24 * 2 * mass


def test_no_tokens_and_a_captured_call(lib):
    table = lib.df_rotary_table(64)
    empty = lib.df_rotary(torch.zeros(0, 3, 64, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), table)
    assert empty.shape == (0, 3, 64)
    x, pos = torch.randn(9, 3, 64, device="cuda"), torch.arange(9, device="cuda")
    lib.df_rotary(x, pos, table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lib.df_rotary(x, pos, table)
    x.copy_(torch.randn(9, 3, 64, device="cuda"))
    pos.add_(1000)
    graph.replay()
    assert torch.equal(y, lib.df_rotary(x, pos, table))
