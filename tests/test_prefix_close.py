"""Attention behind long prefixes within a bound that goes by each query's own terms, so that a part left out shows."""
import pytest

torch = pytest.importorskip("torch")

from attention_bound import attend, close, quantized  # noqa: E402
from test_prefix_gpu import Batch  # noqa: E402


@pytest.mark.parametrize("prefix,own,d,group", [(5000, 1, 128, 128), (1000, 50, 128, 64), (513, 33, 64, 64), (20000, 9, 64, 64)])
def test_the_bound_tells(prefix, own, d, group):
    """Weights rounded to FP16 and a rounded output are within it; zeros, the prefix left out, values in the wrong
    order and (of up to 5000 tokens) one page read from elsewhere are not."""
    g = torch.Generator().manual_seed(prefix)
    n, scale = prefix + own, d ** -0.5
    k = torch.randn(1, n, d, generator=g)
    k[..., ::29] *= 4
    v = torch.randn(1, n, d, generator=g) * torch.exp(torch.randn(1, n, 1, generator=g))
    key, value = quantized(k, group), quantized(v, group)
    q = torch.randn(1, 4, d, generator=g).half().double()
    see = torch.ones(4, n, dtype=torch.bool)
    o, tol, w = attend(q, key, value, see, scale)
    code, s, low = value
    got = torch.empty_like(o)
    for c in range(0, d, group):  # a group's weights p s, their largest at 2^10
        ps = w * s[:, None, :, c]
        up = 2.0 ** 10 / ps.amax(-1, keepdim=True)
        got[..., c:c + group] = (ps * up).half().double() @ (code - 8)[..., c:c + group] / up
    got = (got + w @ (low + 8 * s)).half().double()
    assert ((got - o).abs() <= tol).all()

    def share(x):  # of the elements outside
        return float(((x - o).abs() > tol).double().mean())

    cut = lambda z, at: tuple(x[:, at:] for x in z)  # noqa: E731
    assert share(torch.zeros_like(o)) > 0.4
    assert share(attend(q, cut(key, prefix), cut(value, prefix), see[:, prefix:], scale)[0]) > 0.9
    moved = tuple(x.clone() for x in value)
    for x in moved:
        x[:, :prefix] = x[:, :prefix].flip(1)
    assert share(attend(q, key, moved, see, scale)[0]) > 0.4
    if prefix > 5000:
        return  # 16 tokens are 2^-10 of the weights and less: not told from that many roundings of 2^-11
    page = [tuple(x.clone() for x in z) for z in (key, value)]
    for z in page:
        for x in z:
            x[:, 16:32] = x[:, 0:16]
    assert share(attend(q, *page, see, scale)[0]) > 0


SHAPES = [  # prefix, lens, adds, hq, hkv, d, group, page
    (777, [41, 7, 1, 130], [1] * 4, 16, 16, 128, 128, 16), (1000, [300, 2, 50], [1, 2, 1], 8, 2, 128, 64, 64),
    (2049, [17] * 40, [1] * 40, 32, 8, 128, 128, 16), (3000, [700, 90, 130], [300, 1, 130], 32, 8, 128, 128, 256),
    (5000, [1], [1], 7, 1, 128, 128, 32), (5000, [30, 9, 200], [30, 1, 120], 8, 2, 128, 64, 16),
    (4097, [3] * 65, [1] * 65, 1, 1, 128, 128, 16), (900, [20] * 500, [1] * 500, 4, 1, 64, 64, 16),
    (20000, [50, 9], [40, 9], 4, 2, 64, 64, 32), (131071, [9, 10, 11], [1] * 3, 1, 1, 64, 64, 64),
    (131071, [9 + i for i in range(40)], [1] * 40, 4, 1, 128, 128, 64), (131071, [9, 40, 11], [1, 2, 1], 2, 1, 128, 64, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("table", [0, 30000], ids=["table", "long_table"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%d-%dreq-%d-%d-%d" % (s[0], len(s[1]), sum(s[2]), s[5], s[6]))
def test_close(lib, monkeypatch, shape, table):
    monkeypatch.setattr(Batch, "spare", table)
    prefix, lens, adds, hq, hkv, d, group, page = shape
    b = Batch(lib, prefix, lens, adds, hq, hkv, d, group, page, seed=prefix + 1)
    close(b, b.run())


@pytest.mark.gpu
@pytest.mark.parametrize("adds", [[1, 1, 1], [1, 40, 3], [90, 130, 70]])
def test_one_table_of_both_parts(lib, adds):
    """A prefix that fills its pages, in front of each request's own table: tl_kv4_attention's output in the same bound."""
    b = Batch(lib, 4096, [a + 33 for a in adds], adds, 16, 4, 128, 128, 16, seed=2)
    table = torch.cat((b.prefix_table.expand(3, -1), b.table), 1).contiguous()
    close(b, b.run())
    close(b, lib.kv4_attention(b.cache, b.q, b.start, (b.lens + 4096).int(), table, b.max_q))


@pytest.mark.gpu
@pytest.mark.parametrize("table", [0, 30000], ids=["table", "long_table"])
def test_rows_of_no_request_are_left(lib, monkeypatch, table):
    """Rows in front of the first request, behind the last one, and those past max_q queries of a request."""
    monkeypatch.setattr(Batch, "spare", table)
    b = Batch(lib, 200, [100, 150, 50], [90, 30, 40], 8, 2, 128, 128, 16, seed=4)
    want = b.run()
    close(b, want)
    start = b.start.tolist()
    out = torch.full_like(b.q, 5.0)
    b.start[1] = 0  # the first request has no queries, the second one its rows too
    b.max_q = 120
    close(b, b.run(out=out))
    b.start[:] = torch.tensor(start, dtype=torch.int32)
    b.start[0], b.start[3] = 20, 140
    b.max_q = 25
    out.fill_(5.0)
    b.run(out=out)
    written = torch.zeros(len(b.q), dtype=torch.bool, device="cuda")
    for i in range(3):
        a, z = int(b.start[i]), int(b.start[i + 1])
        written[a:min(z, a + 25)] = True
    assert (out[~written] == 5.0).all() and (out[written] != 5.0).flatten(1).any(1).all()
    lib.tl_check_status()
