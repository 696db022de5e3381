"""Calls that allocate for the caller: what they allocate belongs to the stream they launch on."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_quant_gb300 as tlq  # noqa: E402


class Recorded:
    """Stands for a CUDA tensor; notes the stream context it was made in and the streams it is recorded on."""

    def __init__(self, shape, dtype, on):
        self.shape, self.dtype, self.on, self.kept_for = tuple(shape), dtype, on, []
        self.device = "cuda"

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def record_stream(self, s):
        self.kept_for.append(s)


@pytest.fixture
def fake(monkeypatch):
    made, now, launched = [], ["caller's"], []

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(shape, dtype=None, device=None):
        made.append(Recorded((shape,) if isinstance(shape, int) else shape, dtype, now[-1]))
        return made[-1]

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, t.dtype))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h: "handle %d" % h)
    for name in ("tl_quant_gemm_ws", "tl_pack_weights", "tl_quant_gemm_swiglu", "tl_interleave_rows",
                 "tl_requant_int4_to_int2", "tl_kv4_attention", "tl_lora_add", "tl_unpack_weights", "tl_dequant_fp16"):
        monkeypatch.setattr(tlq, name, lambda *a, **k: launched.append(a))
    monkeypatch.setattr(tlq, "tl_quant_gemm_workspace_size", lambda *a: 64)
    monkeypatch.setattr(tlq, "tl_kv4_attention_workspace_size", lambda *a: 64)
    return made, launched


def t(*shape):
    return Recorded(shape, torch.float16, "caller's")


class Cache:
    heads, head_dim = 2, 64
    blocks = t(1, 2, 64)
    attention_workspace = tlq.KV4Cache.attention_workspace


CALLS = {
    "quant_gemm": lambda s: tlq.quant_gemm(t(4, 128), t(64, 16), t(64, 1), t(64, 1), 4, 128, stream=s),
    "pack_weights": lambda s: tlq.pack_weights(t(64, 128), 4, stream=s),
    "quant_gemm_swiglu": lambda s: tlq.quant_gemm_swiglu(t(4, 128), t(64, 16), t(64, 1), t(64, 1), 4, 128, stream=s),
    "interleave_rows": lambda s: tlq.interleave_rows(t(4, 8), t(4, 8), s),
    "requant_int4_to_int2": lambda s: tlq.requant_int4_to_int2(t(64, 16), t(64, 1), t(64, 1), 128, stream=s),
    "kv4_attention": lambda s: tlq.kv4_attention(Cache(), t(3, 4, 64), t(2), t(1), t(1, 4), 3, stream=s),
    "lora_add": lambda s: tlq.lora_add(t(3, 64), t(1, 8, 64), t(1, 32, 8), t(1), t(2), t(1), 3, t(3, 32), stream=s),
    "unpack_weights": lambda s: tlq.unpack_weights(t(64, 16), 128, 4, stream=s),
    "dequant_fp16": lambda s: tlq.dequant_fp16(t(64, 16), t(64, 1), t(64, 1), 4, 128, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream,on", [(None, "caller's"), ("side", "side"), (77, "handle 77"), (0, "default")])
def test_what_a_call_allocates_is_of_its_stream(fake, name, stream, on):
    made, launched = fake
    out = CALLS[name](stream)
    assert len(launched) == 1 and made and all(m.on == on for m in made)
    for x in out if isinstance(out, tuple) else (out,):  # the caller's stream may use what it is given
        assert x in made and x.kept_for == ([] if stream is None else ["caller's"])


@pytest.mark.gpu
@pytest.mark.parametrize("adds", [1, 150])
def test_temporaries_are_not_handed_out_while_in_use(lib, adds):
    """A call on a busy side stream; the caller's stream allocates and fills what it can get meanwhile."""
    from test_serve_corners_gpu import Batch

    b = Batch(lib, [900, 700, 300], [adds] * 3, 8, 2, 128, 128)
    want = b.run()
    side = torch.cuda.Stream()
    ws_bytes = b.cache.attention_workspace(8, adds).numel()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)  # about 20 ms before the call begins
        got = lib.kv4_attention(b.cache, b.q, b.start, b.seq, b.table, adds, stream=handle)
        junk = [torch.full((ws_bytes,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        junk += [torch.full_like(b.q, float("nan")) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del junk
