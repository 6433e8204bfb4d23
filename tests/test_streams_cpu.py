"""With a stream as an argument, everything that a call or a layer allocates has to
belong to that stream: a block of the current stream's pool would be handed out
again while the given stream still uses it.  Checked without a GPU: the library's
entry points are replaced by ones that do nothing, the tensors say that they are on a
device, and every allocation is recorded with the stream that is current then."""

import contextlib

import pytest
import torch

BF = torch.bfloat16


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def dev(*shape, dtype=BF):
    return torch.Tensor._make_subclass(OnDevice, torch.zeros(*shape, dtype=dtype))


@pytest.fixture
def record(monkeypatch):
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding, encoder

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 1024
            return lambda *a: 0

    current, seen = [None], []

    @contextlib.contextmanager
    def use(stream, like=None):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "_current", use)
    monkeypatch.setattr(binding, "_stream", lambda stream: stream)
    monkeypatch.setattr(binding, "_call_on", lambda idx, fn, *a: 0)

    class Torch:  # torch, with allocations recorded
        def __getattr__(self, name):
            return getattr(torch, name)

        def empty(self, *shape, **kw):
            seen.append(current[0])
            if "size" not in kw and len(shape) == 1 and not isinstance(shape[0], int):
                shape = tuple(shape[0])
            return dev(*shape, dtype=kw.get("dtype", torch.float32))

        def zeros(self, *shape, **kw):
            return self.empty(*shape, **kw)

        def empty_like(self, t):
            return self.empty(*t.shape, dtype=t.dtype)

    monkeypatch.setattr(binding, "torch", Torch())
    monkeypatch.setattr(encoder, "torch", Torch())
    return binding, encoder, seen


def calls(b, e):
    x, w = dev(6, 512), dev(512, 512)
    q, pos, cu = dev(6, 8, 64), dev(512, 8, 64), dev(3, dtype=torch.int32)
    mask, ids = dev(2, 3, dtype=torch.uint8), dev(6, dtype=torch.int64)
    at = dict(cu_seqlens=cu, max_seqlen=4)
    cross = dict(cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=4, max_seqlen_k=4)
    info = b.PackedInfo(2, 3, cu, ids, dev(6, dtype=torch.int32), cu, 6, 3)
    cfg = e.EncoderConfig(hidden=512, heads=8, layers=1, ffn=512, vocab=5)
    layers, shared = ({n: dev(*t.shape) for n, t in w.items()} for w in (
        e.synthetic_weights(cfg, device="cpu")[0][0], e.synthetic_weights(cfg, device="cpu")[1]))
    enc = e.Encoder(cfg, [layers], shared)
    layer = e.CrossAttention(cfg, {n: dev(*t.shape) for n, t in e.synthetic_cross_weights(cfg, device="cpu").items()})
    return {
        "df_attn_fwd": lambda **s: b.df_attn_fwd(q, q, q, pos, pos, **at, **s),
        "df_attn_fwd_fp32_fast": lambda **s: b.df_attn_fwd_fp32_fast(*[t.float() for t in (q, q, q, pos, pos)], **at, **s),
        "df_attn_bwd": lambda **s: b.df_attn_bwd(q, q, q, pos, pos, q, **at, **s),
        "df_attn_fwd_host": lambda **s: b.df_attn_fwd_host(*[torch.zeros(t.shape, dtype=BF) for t in (q, q, q, pos, pos)],
                                                           cu_seqlens=torch.zeros(3, dtype=torch.int32), max_seqlen=4,
                                                           out=torch.zeros(q.shape, dtype=BF), **s),
        "df_attn_plan": lambda **s: b.df_attn_plan(q, q, pos, pos, **at, **s),
        "df_rel_index_table": lambda **s: b.df_rel_index_table(256, 512, 256, 9, **s),
        "df_pack_info": lambda **s: b.df_pack_info(mask, **s),
        "pack_padded_with_info": lambda **s: b.pack_padded_with_info(dev(2, 3, 8), mask, **s),
        "unpack_packed": lambda **s: b.unpack_packed(dev(6, 8), cu, 3, info, **s),
        "df_linear": lambda **s: b.df_linear(x, [w], **s),
        "qkv_projection": lambda **s: b.qkv_projection(x, dev(1536, 512), None, 8, **s),
        "rel_projection": lambda **s: b.rel_projection(x, w, None, w, None, 8, **s),
        "df_layernorm": lambda **s: b.df_layernorm(x, dev(512), dev(512), **s),
        "df_embedding": lambda **s: b.df_embedding(ids, dev(5, 512), **s),
        "df_embedding_bwd": lambda **s: b.df_embedding_bwd(ids, x, 5, **s),
        "df_cross_attn_fwd": lambda **s: b.df_cross_attn_fwd(q, q, q, with_stats=True, **cross, **s),
        "df_cross_attn_bwd": lambda **s: b.df_cross_attn_bwd(q, q, q, q, b.CrossStats(dev(6, 8, dtype=torch.float32), q), q,
                                                             **cross, **s),
        "Encoder.embed": lambda **s: enc.embed(ids, **s),
        "Encoder": lambda **s: enc(x, cu, 4, **s),
        "CrossAttention.project": lambda **s: layer.project(x, **s),
        "CrossAttention.attend": lambda **s: layer.attend(x, q, q, cu, 4, cu, 4, **s),
    }


NAMES = ["df_attn_fwd", "df_attn_fwd_fp32_fast", "df_attn_bwd", "df_attn_fwd_host", "df_attn_plan", "df_rel_index_table",
         "df_pack_info", "pack_padded_with_info", "unpack_packed", "df_linear", "qkv_projection", "rel_projection",
         "df_layernorm", "df_embedding", "df_embedding_bwd", "df_cross_attn_fwd", "df_cross_attn_bwd", "Encoder.embed",
         "Encoder", "CrossAttention.project", "CrossAttention.attend"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream_given(record, name):
    b, e, seen = record
    call = calls(b, e)[name]
    seen.clear()
    call(stream=1234)
    assert seen and set(seen) == {1234}, seen


def test_a_stream_may_be_given_by_position(record):
    b, _, seen = record
    b.df_pack_info(dev(2, 3, dtype=torch.uint8), 1234)
    b.df_rel_index_table(256, 512, 256, 9, None, 1234)
    assert set(seen) == {1234}


def test_every_call_with_a_stream_is_listed(record):
    import inspect
    b, _, _ = record
    waits = {"df_attn_noalloc_get_device_status", "df_attn_get_device_status", "df_attn_fwd_noalloc"}  # allocate nothing
    takes = {n for n, f in vars(b).items() if inspect.isfunction(f) and not n.startswith("_") and
             "stream" in inspect.signature(f).parameters}
    assert takes - waits <= set(NAMES)


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_streams_handles(monkeypatch, handle):
    # (an external stream of handle 0 would be a new stream of torch's)
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: f"external {handle}")
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert binding._current(handle, None) == "default"
    assert binding._current(64, None) == "external 64"


def test_a_stream_of_another_device_is_refused(monkeypatch):
    from exact_attention_deberta_gb300.build import build
    build()
    from exact_attention_deberta_gb300 import binding

    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 64

    class Here(OnDevice):
        device = torch.device("cuda", 0)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    x = torch.Tensor._make_subclass(Here, torch.zeros(2, 512))
    with pytest.raises(ValueError, match="device"):
        binding._current(Stream(), x)
    with pytest.raises(ValueError, match="device"):
        binding.df_layernorm(x, x, x, stream=Stream())
    Here.device = Stream.device
    assert isinstance(binding._current(Stream(), x), Stream)
