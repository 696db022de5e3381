"""Rotations, shared prefix and sampling at the ends of their ranges: offsets past 32 bits, long prefixes, rows
behind the last request that hold anything."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from test_prefix_gpu import Batch  # noqa: E402
from test_rope_gpu import EPS, make_table, plain as rotated  # noqa: E402
from test_sample_gpu import plain as sampled  # noqa: E402


def test_rows_past_32_bits(lib):
    """Token strides of 65536 values: the last rows lie 2.6e9 values behind the first."""
    tokens, wide = 40000, 65536
    rows = torch.zeros(tokens, wide, dtype=torch.float16, device="cuda")
    g = torch.Generator("cuda").manual_seed(0)
    rows[:, -1024:] = torch.randn(tokens, 1024, device="cuda", generator=g).half()
    q = rows[:, -1024:-512].view(tokens, 4, 128)
    k = rows[:, -512:].view(tokens, 4, 128)
    w = (1 + 0.1 * torch.randn(128, device="cuda", generator=g)).half()
    pos = torch.randint(0, 900, (tokens,), dtype=torch.int32, device="cuda", generator=g)
    table = make_table(900, 64)
    some = torch.tensor([0, 1, 20000, 32767, 32768, 39998, 39999], device="cuda")
    want = [rotated(x[some], w, table, pos[None, some], [64], False).half() for x in (q, k)]
    rope = lib.Rope(table)
    cache = lib.KV4Cache(-(-tokens // 16), 4, 128)
    slots = torch.arange(tokens, device="cuda")
    out = torch.empty(tokens, 4, 128, dtype=torch.float16, device="cuda")
    lib.tl_kv4_append_rope(cache, rope, k, k, pos, slots, w, q, out, w, EPS)
    assert torch.equal(out[some], want[0])
    lib.tl_qk_norm_rope(rope, q, k, pos, q, k, w, w, EPS)  # in place
    assert torch.equal(q[some], want[0]) and torch.equal(k[some], want[1])
    # the cache has the rotated keys' codes
    two = lib.KV4Cache(1, 4, 128)
    two.blocks.zero_()
    lib.tl_kv4_append(two, want[1], want[1], torch.arange(len(some), device="cuda"))
    a, b, c, d = (torch.empty(len(some), 4, 128, dtype=torch.float16, device="cuda") for _ in range(4))
    lib.tl_kv4_read(cache, some, a, b)
    lib.tl_kv4_read(two, torch.arange(len(some), device="cuda"), c, d)
    assert torch.equal(a, c)


def test_a_table_past_32_bits(lib):
    """Positions whose table rows lie past 2^32 bytes."""
    f = torch.full((64,), 1e-6, dtype=torch.float64, device="cuda")
    n = 9_000_000  # 4.6 GB
    table = lib.rope_table(n, f)
    pos = torch.tensor([0, 1, 8_388_607, 8_388_608, n - 1], dtype=torch.int32, device="cuda")
    q = torch.randn(5, 2, 128, device="cuda").half()
    out = torch.empty_like(q)
    lib.tl_qk_norm_rope(lib.Rope(table), q, None, pos, out, None)
    angle = pos.double()[:, None, None] * 1e-6
    a, b = q.double()[..., :64], q.double()[..., 64:]
    want = torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1)
    big = torch.maximum(a.abs(), b.abs()).repeat(1, 1, 2)
    assert ((out.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -21 * big).all()


@pytest.mark.parametrize("hq,hkv,d,group,requests", [(1, 1, 64, 64, 3), (4, 1, 128, 128, 40), (2, 1, 128, 64, 5)])
def test_long_prefix(lib, hq, hkv, d, group, requests):
    Batch(lib, 131071, [9 + i for i in range(requests)], [1] * requests, hq, hkv, d, group, 64, seed=d).check()


@pytest.mark.parametrize("adds,pad", [([1, 1, 1], 5), ([1] * 60, 9), ([40, 1, 30], 100)])
def test_padded_batches(lib, adds, pad):
    """Rows behind the last request hold NaN, infinities and FP16's largest: the requests' rows do not show it, and
    the padding's output is left."""
    b = Batch(lib, 900, [a + 17 for a in adds], adds, 8, 2, 128, 128, 16)
    used = len(b.q)
    junk = torch.randn(pad, 8, 128, device="cuda").half()
    junk[0], junk[1], junk[2, ::2], junk[3:] = float("nan"), float("inf"), 65504.0, junk[3:] * 1000
    b.q = torch.cat((b.q, junk))
    out = torch.full_like(b.q, 3.0)
    b.run(out=out)
    want, tol = b.exact()
    assert (out[used:] == 3.0).all()
    assert ((out[:used].double() - want[:used]).abs() <= tol[:used] + 2.0 ** -24).all()


def test_logits_past_32_bits(lib):
    rows, vocab = 2100, 1 << 20
    x = torch.empty(rows, vocab, dtype=torch.float16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    x.mul_(3)
    u = torch.rand(rows, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    p = torch.full((rows,), 0.7, device="cuda")
    some = torch.tensor([0, 1, 2046, 2047, 2048, 2099], device="cuda")
    for f in (dict(), dict(p=p)):
        tokens, _ = lib.sample(x, u, top_p=f.get("p"))
        assert tokens[some].tolist() == sampled(x[some], u[some], p=None if not f else p[some])[0]
