"""Results that overlap an input, or one another, are refused on the host: the kernels read
an input while other blocks already write results, so the outcome would be silently wrong."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding
    return binding


# B = 2, H = 4, Hk = 2, Lq = 5, Lk = 9, d = 64, bf16
BYTES = dict(q=5120, k=4608, v=4608, out=5120, lo=5120, lse=160, dout=5120, dq=5120, dk=4608, dv=4608, mask=18,
             cu_q=12, cu_k=12, ws=10 * 4 * 8)
AT = {n: 0x100000 * (i + 1) for i, n in enumerate(BYTES)}


def fwd(b, **over):
    a = {**AT, "mask": None, "cu_q": None, "cu_k": None, **over}
    p = lambda n: None if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    return b.raw_library.df_cross_attn_fwd(p("q"), p("k"), p("v"), p("mask"), p("cu_q"), p("cu_k"), 2, 4, 2, 5, 9, 10, 18,
                                           64, 0.125, 0, p("out"), p("lo"), p("lse"), None, None)


def bwd(b, **over):
    a = {**AT, "mask": None, "cu_q": None, "cu_k": None, **over}
    p = lambda n: None if a[n] is None else ctypes.c_void_p(a[n])  # noqa: E731
    return b.raw_library.df_cross_attn_bwd(p("q"), p("k"), p("v"), p("out"), p("lo"), p("lse"), p("dout"), p("mask"),
                                           p("cu_q"), p("cu_k"), 2, 4, 2, 5, 9, 10, 18, 64, 0.125, 0, p("dq"), p("dk"),
                                           p("dv"), None, p("ws"), 1 << 16, None)


READ = {fwd: ("q", "k", "v"), bwd: ("q", "k", "v", "out", "lo", "lse", "dout")}
WRITTEN = {fwd: ("out", "lo", "lse"), bwd: ("dq", "dk", "dv", "ws")}


@pytest.mark.parametrize("call", [fwd, bwd])
def test_cross_attention(lib, call):
    step = {"ws": 256}
    for w in WRITTEN[call]:
        for r in READ[call] + tuple(x for x in WRITTEN[call] if x != w):
            for at in (AT[r], AT[r] + (BYTES[r] - 1) // 256 * 256,  # its start, its last bytes
                       AT[r] - (BYTES[w] - 1) // step.get(w, 16) * step.get(w, 16)):  # w's last bytes on its first
                assert call(lib, **{w: at}) == lib.DF_ERR_INVALID_ARG, (w, r, hex(at))
        for r in ("mask", "cu_q", "cu_k"):
            given = {r: AT[w] + (BYTES[w] - 4)} if r != "mask" else {r: AT[w] + BYTES[w] - 1}
            assert call(lib, **given) == lib.DF_ERR_INVALID_ARG, (w, r)


def test_embedding(lib):
    b, p = lib, ctypes.c_void_p
    T, V, N = 4, 10, 64  # ids 16 bytes, table and grad 1280 and 2560, rows 512

    def lookup(ids=0x10000, table=0x20000, out=0x30000):
        return b.raw_library.df_embedding(p(ids), 0, T, p(table), V, N, 1.0, p(out), 0, None, None)

    def grad(ids=0x10000, dout=0x20000, grad=0x30000, ws=0x40000):
        return b.raw_library.df_embedding_bwd(p(ids), 0, T, p(dout), V, N, 1.0, -1, 0, p(grad), 0, None, p(ws), 1 << 20,
                                              None)

    for at in (0x10000, 0x20000, 0x20000 + 1264, 0x20000 - 496, 0x10000 - 496):
        assert lookup(out=at) == b.DF_ERR_INVALID_ARG, hex(at)
    for at in (0x10000, 0x20000, 0x20000 + 496, 0x20000 - 2544, 0x10000 - 2544, 0x40000, 0x40000 - 2544):
        assert grad(grad=at) == b.DF_ERR_INVALID_ARG, hex(at)
    for at in (0x10000, 0x20000, 0x20000 + 256, 0x30000 + 2304):
        assert grad(ws=at) == b.DF_ERR_INVALID_ARG, hex(at)
