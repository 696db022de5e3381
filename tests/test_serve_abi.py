"""Host-side refusals of the serving operators: every bad argument is answered
before anything is launched (the addresses below are never read), and the
sizes the library reports follow from the documented layout."""
import ctypes
import os
import shutil

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

M = 1 << 20


@pytest.fixture(scope="module")
def tlq():
    import weight_only_int4_quant_gb300 as tlq

    tlq.build()
    tlq.load()
    return tlq


def cache(tlq, blocks=64 * M, num_pages=10, heads=4, head_dim=128, page_size=16, group=128):
    return tlq._KV4Cache(blocks, num_pages, heads, head_dim, page_size, group)


@pytest.mark.parametrize("page,d,g,ok", [(16, 128, 128, True), (64, 128, 64, True), (256, 64, 64, True),
                                         (8, 128, 128, False), (24, 128, 128, False), (512, 64, 64, False),
                                         (16, 96, 32, False), (16, 64, 128, False), (16, 128, 32, False),
                                         (0, 128, 128, False), (16, -64, 64, False)])
def test_block_bytes(tlq, page, d, g, ok):
    got = tlq.load().tl_kv4_block_bytes(page, d, g)
    assert got == (2 * page * (d // 2 + 4 * d // g) if ok else 0)
    assert ok or tlq.tl_last_error()


BAD_CACHES = [(dict(blocks=None), "null"), (dict(blocks=64 * M + 8), "aligned"), (dict(num_pages=0), "num_pages"),
              (dict(num_pages=1 << 31), "num_pages"), (dict(heads=0), "heads"), (dict(heads=5000), "heads"),
              (dict(head_dim=0), "head_dim"), (dict(page_size=17), "page_size"), (dict(group=0), "group"),
              (dict(head_dim=64, group=128), "multiple")]


def append(tlq, c, k=1 * M, ldk=512, v=2 * M, ldv=512, slots=3 * M, tokens=4):
    return tlq.load().tl_kv4_append(ctypes.byref(c) if c is not None else None, k, ldk, v, ldv, slots, tokens, None)


def read(tlq, c, slots=3 * M, tokens=4, k=1 * M, v=2 * M):
    return tlq.load().tl_kv4_read(ctypes.byref(c) if c is not None else None, slots, tokens, k, v, None)


def attention(tlq, c, q=1 * M, ldq=1024, hq=8, out=2 * M, ldo=1024, qs=3 * M, lens=4 * M, table=5 * M, ldt=4, b=2, t=6,
              max_q=3, scale=0.1, window=0, ws=256 * M, wsb=64 * M):
    return tlq.load().tl_kv4_attention(ctypes.byref(c) if c is not None else None, q, ldq, hq, out, ldo, qs, lens,
                                       table, ldt, b, t, max_q, scale, window, ws, wsb, None)


@pytest.mark.parametrize("bad,word", BAD_CACHES)
def test_cache_refusals(tlq, bad, word):
    for call in (append, read, attention):
        assert call(tlq, cache(tlq, **bad)) == tlq.TLQ_EINVAL
        assert word in tlq.tl_last_error()


def test_cache_unsupported_and_null(tlq):
    for call in (append, read, attention):
        assert call(tlq, None) == tlq.TLQ_EINVAL
        assert call(tlq, cache(tlq, head_dim=256, group=128)) == tlq.TLQ_EUNSUPPORTED
        assert call(tlq, cache(tlq, group=32)) == tlq.TLQ_EUNSUPPORTED


@pytest.mark.parametrize("bad,word", [(dict(tokens=-1), "tokens"), (dict(k=None), "null"), (dict(v=None), "null"),
                                      (dict(slots=None), "null"), (dict(ldk=504), "ldk"), (dict(ldv=516), "ldv"),
                                      (dict(k=1 * M + 8), "aligned"), (dict(slots=3 * M + 4), "aligned"),
                                      (dict(v=64 * M), "overlap"), (dict(slots=64 * M + 64), "overlap")])
def test_append_refusals(tlq, bad, word):
    assert append(tlq, cache(tlq), **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


@pytest.mark.parametrize("bad,word", [(dict(tokens=-1), "tokens"), (dict(k=None), "null"), (dict(slots=None), "null"),
                                      (dict(v=2 * M + 2), "aligned"), (dict(v=1 * M + 64), "overlap"),
                                      (dict(k=64 * M), "overlap"), (dict(v=3 * M), "overlap")])
def test_read_refusals(tlq, bad, word):
    assert read(tlq, cache(tlq), **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


@pytest.mark.parametrize("bad,word", [
    (dict(q=None), "null"), (dict(out=None), "null"), (dict(qs=None), "null"), (dict(lens=None), "null"),
    (dict(table=None), "null"), (dict(hq=0), "q_heads"), (dict(hq=6), "q_heads"), (dict(b=-1), "requests"),
    (dict(t=-1), "tokens"), (dict(max_q=-1), "max_q"), (dict(window=-1), "window"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(ldt=0), "ld_table"),
    (dict(ldq=1016), "ldq"), (dict(ldo=1028), "ldo"), (dict(q=1 * M + 8), "aligned"), (dict(out=2 * M + 4), "aligned"),
    (dict(ws=256 * M + 8), "aligned"), (dict(ws=None), "workspace"), (dict(wsb=64), "workspace"),
    (dict(out=1 * M + 64), "overlap"), (dict(out=64 * M), "overlap"), (dict(ws=1 * M), "overlap"),
    (dict(ws=64 * M - 1024), "overlap")])
def test_attention_refusals(tlq, bad, word):
    assert attention(tlq, cache(tlq), **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


def test_nothing_to_do_is_no_launch(tlq):
    """Empty batches return without touching the device (there may be none)."""
    assert append(tlq, cache(tlq), tokens=0) == tlq.TLQ_OK
    assert read(tlq, cache(tlq), tokens=0) == tlq.TLQ_OK
    for empty in (dict(b=0), dict(t=0), dict(max_q=0)):
        assert attention(tlq, cache(tlq), **empty) == tlq.TLQ_OK
        assert lora(tlq, **empty) == tlq.TLQ_OK


def test_workspace_size(tlq):
    assert tlq.tl_kv4_attention_workspace_size(8, 4, 128, 1) > 0
    # one workspace of the larger max_q serves every smaller step
    sizes = [tlq.tl_kv4_attention_workspace_size(8, 4, 128, m) for m in (1, 4, 5, 100, 4096)]
    assert sizes == sorted(sizes)
    for bad in ((0, 4, 128, 1), (8, 0, 128, 1), (7, 4, 128, 1), (8, 4, 96, 1), (8, 4, 128, -1)):
        assert tlq.tl_kv4_attention_workspace_size(*bad) == 0


def plan(tlq, cached=1 * M, added=2 * M, b=8, table=3 * M, ldt=16, free=4 * M, nfree=32, head=None, page=16,
         pages=100, qs=5 * M, lens=6 * M, req=7 * M, pos=8 * M, slots=9 * M, cap=64, counts=10 * M):
    return tlq.load().tl_kv_plan(cached, added, b, table, ldt, free, nfree, head, page, pages, qs, lens, req, pos,
                                 slots, cap, counts, None)


@pytest.mark.parametrize("bad,word", [
    (dict(b=-1), "requests"), (dict(cap=-1), "capacity"), (dict(nfree=-1), "num_free"), (dict(page=12), "page_size"),
    (dict(page=0), "page_size"), (dict(pages=0), "num_pages"), (dict(ldt=0), "ld_table"), (dict(cached=None), "null"),
    (dict(added=None), "null"), (dict(table=None), "null"), (dict(free=None), "null"), (dict(qs=None), "null"),
    (dict(lens=None), "null"), (dict(req=None), "null"), (dict(pos=None), "null"), (dict(slots=None), "null"),
    (dict(counts=None), "null"), (dict(slots=9 * M + 4), "aligned"), (dict(cached=1 * M + 2), "aligned"),
    (dict(lens=1 * M), "overlap"), (dict(head=10 * M + 8), "overlap"), (dict(req=8 * M + 16), "overlap"),
    (dict(table=4 * M + 64), "overlap"), (dict(qs=6 * M + 28), "overlap")])
def test_plan_refusals(tlq, bad, word):
    assert plan(tlq, **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


def lora(tlq, x=1 * M, ldx=256, A=2 * M, B=3 * M, scales=4 * M, qs=5 * M, ad=6 * M, b=3, t=10, max_q=4, K=256, N=512,
         rank=16, num=2, y=7 * M, ldy=512, out=8 * M, ldo=512):
    return tlq.load().tl_lora_add(x, ldx, A, B, scales, qs, ad, b, t, max_q, K, N, rank, num, y, ldy, out, ldo, None)


@pytest.mark.parametrize("bad,word", [
    (dict(b=-1), "requests"), (dict(t=-1), "tokens"), (dict(max_q=-1), "max_q"), (dict(K=12), "K="),
    (dict(K=0), "K="), (dict(N=20), "N="), (dict(rank=0), "rank"), (dict(rank=12), "rank"), (dict(num=-1), "num"),
    (dict(x=None), "null"), (dict(A=None), "null"), (dict(B=None), "null"), (dict(scales=None), "null"),
    (dict(qs=None), "null"), (dict(ad=None), "null"), (dict(y=None), "null"), (dict(out=None), "null"),
    (dict(ldx=248), "ldx"), (dict(ldy=510), "ldy"), (dict(ldo=504), "ldo"), (dict(x=1 * M + 2), "aligned"),
    (dict(B=3 * M + 8), "aligned"), (dict(out=7 * M + 16), "overlap"), (dict(out=7 * M, ldo=520), "overlap"),
    (dict(out=1 * M), "overlap"), (dict(out=3 * M), "overlap")])
def test_lora_refusals(tlq, bad, word):
    assert lora(tlq, **bad) == tlq.TLQ_EINVAL
    assert word in tlq.tl_last_error()


def test_lora_unsupported_rank(tlq):
    assert lora(tlq, rank=72) == tlq.TLQ_EUNSUPPORTED


@pytest.mark.parametrize("at", [3, 4, 5])
@pytest.mark.parametrize("name,size", [("out", 6 * 1024 * 2), ("ws", None)])
def test_attention_refuses_outputs_over_the_batch(tlq, at, name, size):
    """q_start, seq_lens and table lie at 3, 4 and 5 M; the buffer's first and its last bytes over their first."""
    size = size or tlq.tl_kv4_attention_workspace_size(8, 4, 128, 3)
    for address in (at * M, at * M - size + 16):
        if name == "ws" and address < 0:
            continue
        assert attention(tlq, cache(tlq), **{name: address}) == tlq.TLQ_EINVAL
        assert "overlaps" in tlq.tl_last_error()


@pytest.mark.parametrize("at", [4, 5, 6])
def test_lora_refuses_outputs_over_the_batch(tlq, at):
    """scales, q_start and adapters lie at 4, 5 and 6 M."""
    for address in (at * M, at * M - 10 * 512 * 2 + 16):
        assert lora(tlq, out=address) == tlq.TLQ_EINVAL
        assert "overlaps" in tlq.tl_last_error()
