"""Host-side refusals of the rotations, the shared prefix and sampling: every bad argument is answered before
anything is launched (the addresses below are never read)."""
import ctypes

import pytest

from test_serve_abi import BAD_CACHES, M, cache, pytestmark, tlq  # noqa: F401


def rope(tlq, table=32 * M, positions=1000, rot=128, interleaved=0, axes=1, sections=(64, 0, 0)):
    return tlq._Rope(table, positions, rot, interleaved, axes, (ctypes.c_int * 3)(*sections))


def ref(x):
    return None if x is None else ctypes.byref(x)


def qk(tlq, r="default", pos=1 * M, q=2 * M, ldq=1024, hq=8, qw=3 * M, qo=4 * M, ldqo=1024, k=5 * M, ldk=256, hk=2,
       kw=6 * M, ko=7 * M, ldko=256, d=128, eps=1e-6, tokens=4):
    r = rope(tlq) if r == "default" else r
    return tlq.load().tl_qk_norm_rope(ref(r), pos, q, ldq, hq, qw, qo, ldqo, k, ldk, hk, kw, ko, ldko, d, eps, tokens,
                                      None)


BAD_ROPES = [(dict(rot=8), "rot_dim"), (dict(rot=24), "rot_dim"), (dict(rot=256), "rot_dim"), (dict(positions=0), "num_positions"),
             (dict(positions=(1 << 30) + 1), "num_positions"), (dict(axes=0), "axes"), (dict(axes=4), "axes"),
             (dict(sections=(63, 0, 0)), "sections"), (dict(axes=2, sections=(64, 1, 0)), "sections"),
             (dict(axes=2, sections=(65, -1, 0)), "sections"), (dict(table=None), "null"), (dict(table=32 * M + 8), "aligned")]


@pytest.mark.parametrize("bad,word", BAD_ROPES)
def test_rope_refusals(tlq, bad, word):  # noqa: F811
    for call in (lambda r: qk(tlq, r), lambda r: append(tlq, r=r)):
        assert call(rope(tlq, **bad)) == tlq.TLQ_EINVAL
        assert word in tlq.tl_last_error()


@pytest.mark.parametrize("bad,word", [
    (dict(tokens=-1), "tokens"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(d=0), "head_dim"), (dict(hq=-1), "q_heads"), (dict(hk=5000), "k_heads"), (dict(q=None), "null"),
    (dict(qo=None), "null"), (dict(k=None), "null"), (dict(ko=None), "null"), (dict(pos=None), "null"),
    (dict(ldq=1016), "ldq"), (dict(ldqo=1028), "ldq"), (dict(ldk=248), "ldk"), (dict(ldko=260), "ldk"),
    (dict(q=2 * M + 8), "aligned"), (dict(qw=3 * M + 2), "aligned"), (dict(ko=7 * M + 4), "aligned"),
    (dict(pos=1 * M + 2), "aligned"), (dict(qo=2 * M + 16), "overlap"), (dict(qo=2 * M, ldqo=1032), "overlap"),
    (dict(qo=5 * M), "overlap"), (dict(ko=4 * M), "overlap"), (dict(ko=4 * M + 512), "overlap"), (dict(qo=3 * M), "overlap"),
    (dict(ko=1 * M), "overlap"), (dict(qo=32 * M + 1024), "overlap"), (dict(ko=6 * M + 128), "overlap")])
def test_norm_rope_refusals(tlq, bad, word):  # noqa: F811
    assert qk(tlq, **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


def test_norm_rope_unsupported(tlq):  # noqa: F811
    assert qk(tlq, d=96) == tlq.TLQ_EUNSUPPORTED
    big = dict(ldq=4096 * 128, hq=4096, ldqo=4096 * 128, q=1 << 50, qo=1 << 52, hk=0, tokens=1 << 20, pos=1 << 54)
    assert qk(tlq, **big) == tlq.TLQ_EUNSUPPORTED


def append(tlq, c="default", r="default", pos=1 * M, k=2 * M, ldk=512, kw=3 * M, v=4 * M, ldv=512, slots=5 * M, q=6 * M,
           ldq=1024, hq=8, qw=7 * M, qo=8 * M, ldqo=1024, eps=1e-6, tokens=4):
    c = cache(tlq) if c == "default" else c
    r = rope(tlq) if r == "default" else r
    return tlq.load().tl_kv4_append_rope(ref(c), ref(r), pos, k, ldk, kw, v, ldv, slots, q, ldq, hq, qw, qo, ldqo, eps,
                                         tokens, None)


@pytest.mark.parametrize("bad,word", [
    (dict(tokens=-1), "tokens"), (dict(eps=-1.0), "eps"), (dict(k=None), "null"), (dict(v=None), "null"),
    (dict(slots=None), "null"), (dict(q=None), "null"), (dict(qo=None), "null"), (dict(pos=None), "null"),
    (dict(ldk=504), "ldk"), (dict(ldv=516), "ldv"), (dict(ldq=1000), "ldq"), (dict(ldqo=1025), "ldq"),
    (dict(k=2 * M + 8), "aligned"), (dict(v=4 * M + 2), "aligned"), (dict(slots=5 * M + 4), "aligned"),
    (dict(kw=3 * M + 8), "aligned"), (dict(qo=6 * M + 16), "overlap"), (dict(qo=2 * M + 512), "overlap"),
    (dict(qo=4 * M), "overlap"), (dict(qo=5 * M), "overlap"), (dict(qo=3 * M), "overlap"), (dict(qo=1 * M), "overlap"),
    (dict(qo=64 * M), "overlap"), (dict(k=64 * M), "overlap"), (dict(v=64 * M + 1024), "overlap"),
    (dict(slots=64 * M), "overlap"), (dict(q=64 * M), "overlap"), (dict(kw=64 * M), "overlap"), (dict(pos=64 * M), "overlap")])
def test_append_rope_refusals(tlq, bad, word):  # noqa: F811
    assert append(tlq, **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


@pytest.mark.parametrize("bad,word", BAD_CACHES)
def test_cache_refusals(tlq, bad, word):  # noqa: F811
    for call in (append, prefix):
        assert call(tlq, cache(tlq, **bad)) == tlq.TLQ_EINVAL
        assert word in tlq.tl_last_error()
        assert call(tlq, None) == tlq.TLQ_EINVAL
        assert call(tlq, cache(tlq, head_dim=256, group=128)) == tlq.TLQ_EUNSUPPORTED


def test_a_head_of_64_takes_no_rope_of_128(tlq):  # noqa: F811
    assert append(tlq, cache(tlq, head_dim=64, group=64)) == tlq.TLQ_EINVAL
    assert "rot_dim" in tlq.tl_last_error()


def prefix(tlq, c="default", q=1 * M, ldq=1024, hq=8, out=2 * M, ldo=1024, qs=3 * M, lens=4 * M, table=5 * M, ldt=4,
           plen=6 * M, ptable=7 * M, pages=9, b=2, t=6, max_q=3, scale=0.1, ws=256 * M, wsb=64 * M):
    c = cache(tlq) if c == "default" else c
    return tlq.load().tl_kv4_attention_prefix(ref(c), q, ldq, hq, out, ldo, qs, lens, table, ldt, plen, ptable, pages, b, t,
                                              max_q, scale, ws, wsb, None)


@pytest.mark.parametrize("bad,word", [
    (dict(q=None), "null"), (dict(out=None), "null"), (dict(qs=None), "null"), (dict(lens=None), "null"),
    (dict(table=None), "null"), (dict(plen=None), "null"), (dict(ptable=None), "null"), (dict(pages=-1), "prefix_pages"),
    (dict(hq=0), "q_heads"), (dict(hq=6), "q_heads"), (dict(b=-1), "requests"), (dict(t=-1), "tokens"),
    (dict(max_q=-1), "max_q"), (dict(scale=float("nan")), "scale"), (dict(ldt=0), "ld_table"), (dict(ldq=1016), "ldq"),
    (dict(ldo=1028), "ldo"), (dict(q=1 * M + 8), "aligned"), (dict(out=2 * M + 4), "aligned"), (dict(plen=6 * M + 2), "aligned"),
    (dict(ws=256 * M + 8), "aligned"), (dict(ws=None), "workspace"), (dict(wsb=64), "workspace"), (dict(out=1 * M + 64), "overlap"),
    (dict(out=64 * M), "overlap"), (dict(out=6 * M), "overlap"), (dict(out=7 * M + 16), "overlap"), (dict(out=5 * M), "overlap"),
    (dict(ws=1 * M), "overlap"), (dict(ws=6 * M - 1024), "overlap"), (dict(ws=64 * M - 1024), "overlap")])
def test_prefix_refusals(tlq, bad, word):  # noqa: F811
    assert prefix(tlq, **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


def test_prefix_workspace(tlq):  # noqa: F811
    size = tlq.tl_kv4_attention_prefix_workspace_size
    sizes = [size(8, 4, 128, t, 1) for t in (0, 1, 7, 64, 4096)]
    assert sizes == sorted(sizes) and sizes[0] >= tlq.tl_kv4_attention_workspace_size(8, 4, 128, 1)
    # the sums of every row on both sides
    assert sizes[3] - sizes[0] >= 2 * 64 * 8 * 130 * 4
    for bad in ((0, 4, 128, 1, 1), (8, 0, 128, 1, 1), (7, 4, 128, 1, 1), (8, 4, 96, 1, 1), (8, 4, 128, -1, 1), (8, 4, 128, 1, -1)):
        assert size(*bad) == 0
    assert prefix(tlq, wsb=size(8, 4, 128, 6, 3) - 1) == tlq.TLQ_EINVAL
    assert "workspace" in tlq.tl_last_error()
    assert prefix(tlq, t=1 << 30, max_q=1, ldq=1024, wsb=1 << 62) == tlq.TLQ_EUNSUPPORTED


def sample(tlq, x=16 * M, half=1, ld=1000, rows=4, vocab=1000, u=1 * M, t=2 * M, k=3 * M, p=4 * M, mp=5 * M, tokens=6 * M,
           logs=7 * M):
    return tlq.load().tl_sample(x, half, ld, rows, vocab, u, t, k, p, mp, tokens, logs, None)


@pytest.mark.parametrize("bad,word", [
    (dict(rows=-1), "rows"), (dict(vocab=0), "vocab"), (dict(half=2), "fp16"), (dict(x=None), "null"), (dict(u=None), "null"),
    (dict(tokens=None), "null"), (dict(ld=999), "ld="), (dict(x=16 * M + 1), "aligned"), (dict(x=16 * M + 2, half=0), "aligned"),
    (dict(u=1 * M + 2), "aligned"), (dict(tokens=6 * M + 1), "aligned"), (dict(logs=7 * M + 2), "aligned"),
    (dict(tokens=16 * M + 4), "overlap"), (dict(logs=1 * M), "overlap"), (dict(tokens=2 * M + 8), "overlap"),
    (dict(tokens=3 * M), "overlap"), (dict(logs=4 * M), "overlap"), (dict(logs=5 * M + 12), "overlap"), (dict(logs=6 * M + 4), "overlap")])
def test_sample_refusals(tlq, bad, word):  # noqa: F811
    assert sample(tlq, **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


def test_sample_unsupported(tlq):  # noqa: F811
    assert sample(tlq, vocab=(1 << 20) + 1, ld=1 << 21) == tlq.TLQ_EUNSUPPORTED
    assert sample(tlq, rows=1 << 28) == tlq.TLQ_EUNSUPPORTED


@pytest.mark.parametrize("bad,word", [(dict(f=None), "null"), (dict(t=None), "null"), (dict(n=0), "num_positions"),
                                      (dict(n=(1 << 30) + 1), "num_positions"), (dict(rot=24), "rot_dim"), (dict(rot=512), "rot_dim"),
                                      (dict(scale=float("inf")), "scale"), (dict(t=2 * M + 8), "aligned"),
                                      (dict(f=1 * M + 4), "aligned"), (dict(t=1 * M), "overlap")])
def test_table_refusals(tlq, bad, word):  # noqa: F811
    a = dict(f=1 * M, n=100, rot=64, scale=1.0, t=2 * M)
    a.update(bad)
    assert tlq.load().tl_rope_table(a["f"], a["n"], a["rot"], a["scale"], a["t"], None) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


def test_nothing_to_do_is_no_launch(tlq):  # noqa: F811
    """Empty calls return without touching the device (there may be none)."""
    assert qk(tlq, tokens=0) == tlq.TLQ_OK
    assert qk(tlq, hq=0, hk=0, q=None, qo=None, k=None, ko=None) == tlq.TLQ_OK
    assert append(tlq, tokens=0) == tlq.TLQ_OK
    for empty in (dict(b=0), dict(t=0), dict(max_q=0)):
        assert prefix(tlq, **empty) == tlq.TLQ_OK
    assert sample(tlq, rows=0) == tlq.TLQ_OK


BINDING = ["norm_rope", "append_rope", "sample", "attention_prefix"]


@pytest.fixture(scope="module")
def module(tmp_path_factory):
    """The C API module with every entry point usleep(first argument), as in test_binding."""
    import importlib.util
    import shutil

    import test_binding as tb
    import weight_only_int4_quant_gb300 as lib

    lib.build()
    path = str(tmp_path_factory.mktemp("binding") / "_tlq_binding.so")
    shutil.copy(lib._BINDING_PATH, path)
    spec = importlib.util.spec_from_file_location("_tlq_binding", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    m.bind(tb.F16, tb.F32, tb.I32, tb.I64, tb.U8, lambda: 0, lambda d: 0, *[usleep] * 5)
    m.bind_step(*[usleep] * 4)
    return m, tb


def calls(m, tb):
    """(arguments, the function) of each; addresses first, so that usleep gets a short time."""
    T, h, i, f = tb.Tensor, tb.F16, tb.I32, tb.F32
    q, k, w = T((2, 4, 64), h), T((2, 2, 64), h), T((64,), h)
    pos, slots = T((2,), i), T((2,), tb.I64)
    return {
        "norm_rope": [1000, 1, q, k, pos, q, k, w, None, 1e-6, None],
        "append_rope": [1000, 2, 64, 2000, 1, k, k, pos, slots, w, q, q, w, 1e-6, None],
        "sample": [T((3, 50), f, 1000), T((3,), f), T((3,), i), T((3,), f), T((3,), i), None, T((3,), f), T((3,), f), None],
        "attention_prefix": [1000, 64, q, q, T((4,), i), T((3,), i), T((3, 4), i), T((1,), i), T((5,), i), 1, 0.5,
                             T((64,), tb.U8), None],
    }


@pytest.mark.parametrize("name", BINDING)
def test_the_short_way_calls(module, name):
    m, tb = module
    assert getattr(m, name)(*calls(m, tb)[name]) == 0


@pytest.mark.parametrize("name,at,bad", [
    ("norm_rope", 2, "type"), ("norm_rope", 4, "short"), ("norm_rope", 5, None), ("norm_rope", 6, "type"), ("norm_rope", 7, "short"),
    ("norm_rope", 9, 1), ("append_rope", 5, "type"), ("append_rope", 6, "short"), ("append_rope", 8, "short"),
    ("append_rope", 9, "short"), ("append_rope", 11, None), ("append_rope", 13, 0), ("sample", 0, "type"), ("sample", 1, None),
    ("sample", 2, "short"), ("sample", 3, "type"), ("sample", 7, "short"), ("attention_prefix", 2, "type"),
    ("attention_prefix", 3, "short"), ("attention_prefix", 4, "short"), ("attention_prefix", 7, None), ("attention_prefix", 8, "type"),
    ("attention_prefix", 10, 1), ("attention_prefix", 11, None)])
def test_the_short_way_gives_way(module, name, at, bad):
    """What is not as it should be comes back with -1, without a call and without an exception."""
    m, tb = module
    a = calls(m, tb)[name]
    if bad == "type":
        a[at] = tb.Tensor(a[at].shape, object())
    elif bad == "short":
        shape = a[at].shape
        a[at] = tb.Tensor((shape[0] + 1,) + shape[1:], a[at].dtype)
    else:
        a[at] = bad
    assert getattr(m, name)(*a) == -1


def test_positions_of_several_axes(module):
    m, tb = module
    a = calls(m, tb)["norm_rope"]
    a[1] = 3
    for shape, want in (((3, 2), 0), ((2, 3), -1), ((6,), -1), ((3, 3), -1)):
        a[4] = tb.Tensor(shape, tb.I32)
        assert m.norm_rope(*a) == want
    a[0] = None  # no rope: positions are not looked at
    assert m.norm_rope(*a[:4], None, *a[5:]) == 0


DEVICES = """
import ctypes, sys
sys.modules["torch"] = None
import weight_only_int4_quant_gb300 as tlq
lib, fake, M = tlq.load(), ctypes.CDLL(None), 1 << 20
G = 1 << 36

def prefix(d=128, group=128, t=2):
    c = tlq._KV4Cache(64 * M, 10, 4, d, 16, group)
    return lib.tl_kv4_attention_prefix(ctypes.byref(c), M, 1024, 8, 16 * M, 1024, 3 * M, 4 * M, 5 * M, 4, 6 * M, 7 * M, 9, 2, t,
                                       t, 0.1, G, G, None)

def sample(half, vocab):
    return lib.tl_sample(M, half, vocab, 1, vocab, G, None, None, None, None, 2 * G, None, None)

for device in (0, 1, 5, 0):
    fake.fake_device(device)
    for form in ((128, 128, 2), (128, 64, 8), (64, 64, 4), (128, 128, 2000), (64, 64, 2000)):
        st = prefix(*form)
        assert st == tlq.TLQ_OK, (device, form, st, tlq.tl_last_error())
        assert fake.fake_launches() == (3 if form[2] == 2000 else 2), form
    for half, vocab in ((1, 1), (1, 131072), (0, 200000), (0, 1 << 20)):
        st = sample(half, vocab)
        assert st == tlq.TLQ_OK and fake.fake_launches() == 1, (device, half, vocab, st, tlq.tl_last_error())
fake.fake_device(3)  # a failure is not remembered
for call in (prefix, lambda: sample(1, 1000)):
    fake.fake_failures(1)
    assert call() == tlq.TLQ_ECUDA
    assert call() == tlq.TLQ_OK
print("done")
"""


def test_shared_memory_on_each_device(tmp_path):
    from test_devices import run_child

    run_child(DEVICES, tmp_path)


def test_what_the_calls_allocate_is_of_their_stream(monkeypatch):
    torch = pytest.importorskip("torch")
    import test_streams as ts
    import weight_only_int4_quant_gb300 as lib

    fake = ts.fake.__wrapped__ if hasattr(ts.fake, "__wrapped__") else None
    if fake is None:
        pytest.skip("the fixture cannot be called")
    made, launched = fake(monkeypatch)
    monkeypatch.setattr(torch, "zeros", lambda shape, dtype=None, device=None: torch.empty(shape, dtype, device))
    for name in ("tl_rope_table", "tl_qk_norm_rope", "tl_sample", "tl_kv4_attention_prefix"):
        monkeypatch.setattr(lib, name, lambda *a, **k: launched.append(a))
    monkeypatch.setattr(lib, "tl_kv4_attention_prefix_workspace_size", lambda *a: 64)

    class Cache(ts.Cache):
        prefix_workspace = lib.KV4Cache.prefix_workspace

    calls = [lambda s: lib.rope_table(9, ts.t(32), stream=s), lambda s: lib.qk_norm_rope(None, ts.t(3, 4, 64), ts.t(3, 2, 64), None, stream=s),
             lambda s: lib.sample(ts.t(3, 50), ts.t(3), stream=s),
             lambda s: lib.kv4_attention_prefix(Cache(), ts.t(3, 4, 64), ts.t(2), ts.t(1), ts.t(1, 4), ts.t(1), ts.t(5), 3, stream=s)]
    for call in calls:
        for stream, on in ((None, "caller's"), ("side", "side"), (77, "handle 77"), (0, "default")):
            made.clear(), launched.clear()
            out = call(stream)
            assert len(launched) == 1 and made and all(m.on == on for m in made)
            for x in out if isinstance(out, tuple) else (out,):
                assert x in made and x.kept_for == ([] if stream is None else ["caller's"])
