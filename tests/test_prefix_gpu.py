"""Attention behind a shared prefix against its definition in 64 bits.

Bound, as for the attention without a prefix (u = 2^-11): u |o| for the output, 3 u V for the weights' and
values' roundings, 2 dS V for the keys' with dS = scale * u * max sum |q||k|; V the largest |value| seen."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


@pytest.fixture(autouse=True, params=[0, 30000], ids=["table", "long_table"])
def spare(request, monkeypatch):
    """Which kernels run goes by the table's length: 65 rows and more behind a short one by one kernel, behind a long
    one by both."""
    monkeypatch.setattr(Batch, "spare", request.param)


def cached(blocks, ids, page, d, group, part):
    """Keys (0) or values (1) of pages in 64 bits: [heads, tokens, D]; a page outside the cache: None rows as NaN."""
    got = blocks[ids.clamp(0, blocks.shape[0] - 1)]
    half, par = page * d // 2, 4 * page * d // group
    code = got[..., part * half:(part + 1) * half].unflatten(-1, (page, d // 2))
    code = torch.stack((code & 15, code >> 4), -1).flatten(-2).double()
    at = 2 * half + part * par
    p = got[..., at:at + par].contiguous().view(torch.float16).unflatten(-1, (page, d // group, 2)).double()
    val = code * p[..., 0].repeat_interleave(group, -1) + p[..., 1].repeat_interleave(group, -1)
    return val.transpose(0, 1).flatten(1, 2)


class Batch:
    spare = 0  # entries behind the prefix's own in the table that the kernels get

    def __init__(self, lib, prefix, lens, adds, hq, hkv, d, group, page, seed=0, spread=1.0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.lib, self.page, self.d, self.group, self.hq, self.hkv = lib, page, d, group, hq, hkv
        shared, need = -(-prefix // page), [-(-n // page) for n in lens]
        pages = shared + sum(need) + 4
        self.cache = lib.KV4Cache(pages, hkv, d, page, group)
        order = torch.randperm(pages, device="cuda", generator=g)
        tokens = pages * page
        k = torch.randn(tokens, hkv, d, device="cuda", generator=g) * spread
        k[..., ::29] *= 4
        v = torch.randn(tokens, hkv, d, device="cuda", generator=g) * torch.exp(torch.randn(tokens, hkv, 1, device="cuda", generator=g))
        lib.tl_kv4_append(self.cache, k.half(), v.half(), torch.arange(tokens, device="cuda"))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.prefix_len, self.whole_table = torch.tensor([prefix], **i32), torch.full((shared + self.spare,), -1, **i32)
        self.prefix_table = self.whole_table[:shared]
        self.prefix_table[:] = order[:shared].int()
        self.table = torch.full((len(lens), max(need + [1]) + 1), -1, **i32)
        at = shared
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n].int()
            at += n
        self.lens, start = torch.tensor(lens, **i32), [0]
        for a in adds:
            start.append(start[-1] + a)
        self.start, self.max_q = torch.tensor(start, **i32), max(adds)
        self.q = torch.randn(start[-1], hq, d, device="cuda", generator=g).half()
        self.scale = d ** -0.5

    def run(self, out=None, **k):
        out = torch.full_like(self.q, float("nan")) if out is None else out
        args = dict(workspace=self.cache.prefix_workspace(self.hq, self.q.shape[0], self.max_q))
        args.update(k)
        self.lib.tl_kv4_attention_prefix(self.cache, self.q, out, self.start, self.lens, self.table, self.prefix_len,
                                         self.whole_table, self.max_q, self.scale, **args)
        return out

    def exact(self):
        """(output, bound) in 64 bits."""
        share, n = self.hq // self.hkv, min(max(int(self.prefix_len), 0), self.prefix_table.numel() * self.page)
        args = (self.page, self.d, self.group)
        out, tol = torch.zeros(self.q.shape, dtype=torch.double, device="cuda"), torch.zeros(self.q.shape, device="cuda").double()

        def side(ids, count, part):
            if count == 0:
                return torch.zeros(self.hkv, 0, self.d, device="cuda").double()
            return cached(self.cache.blocks, ids.long(), *args, part)[:, :count]

        def there(ids, count):  # tokens whose page is in the cache
            ok = (ids >= 0) & (ids < self.cache.num_pages)
            return ok.repeat_interleave(self.page)[:count]

        for i in range(len(self.lens)):
            a, b = int(self.start[i]), int(self.start[i + 1])
            m = min(int(self.lens[i]), self.table.shape[1] * self.page)
            if b == a:
                continue
            ids = self.table[i][:-(-m // self.page)]
            k = torch.cat((side(self.prefix_table, n, 0), side(ids, m, 0)), 1).repeat_interleave(share, 0)
            v = torch.cat((side(self.prefix_table, n, 1), side(ids, m, 1)), 1).repeat_interleave(share, 0)
            ok = torch.cat((there(self.prefix_table, n), there(ids, m)))
            q = self.q[a:b].double().transpose(0, 1)
            logit = q @ k.transpose(1, 2) * self.scale
            pos = int(self.lens[i]) - (b - a) + torch.arange(b - a, device="cuda")
            key = torch.arange(n + m, device="cuda") - n  # the prefix lies before the own tokens
            see = ((key[None] <= pos[:, None]) | (key < 0)[None]) & ok
            logit = logit.masked_fill(~see, float("-inf"))
            top = logit.amax(-1, keepdim=True).clamp_min(-1e300) if logit.shape[-1] else None
            if top is None:
                continue
            w = torch.exp(logit - top)
            total = w.sum(-1, keepdim=True)
            o = torch.where(total > 0, (w @ v.nan_to_num()) / total.clamp_min(1e-300), 0.0)
            big = torch.where(ok, v.abs().amax(-1), 0.0).amax(-1)[:, None, None] if v.shape[1] else 0.0
            ds = self.scale * U * (q.abs() @ k.abs().transpose(1, 2)).masked_fill(~see, 0).amax(-1, keepdim=True)
            out[a:b] = o.transpose(0, 1)
            tol[a:b] = (U * o.abs() + 3 * U * big + 2 * ds * big).transpose(0, 1)
        return out, tol

    def check(self, **k):
        got = self.run(**k)
        want, tol = self.exact()
        assert ((got.double() - want).abs() <= tol + 2.0 ** -24).all(), ((got.double() - want).abs() / (tol + 2.0 ** -24)).max()
        return got


SHAPES = [  # prefix, lens, adds, hq, hkv, d, group, page
    (1, [1], [1], 1, 1, 64, 64, 16), (15, [3], [1], 4, 4, 128, 128, 16), (16, [16, 1], [1, 1], 8, 2, 128, 128, 16),
    (777, [41, 7, 1, 130], [1] * 4, 16, 16, 128, 128, 16), (129, [5, 200, 64], [3, 2, 4], 14, 2, 64, 64, 32),
    (1000, [300, 2, 50], [1, 2, 1], 8, 2, 128, 64, 64), (2049, [17] * 40, [1] * 40, 32, 8, 128, 128, 16),
    (513, [60, 1, 33], [60, 1, 30], 12, 4, 128, 128, 128), (255, [400, 9, 90], [257, 1, 31], 8, 2, 64, 64, 16),
    (3000, [700, 90, 130], [300, 1, 130], 32, 8, 128, 128, 256), (5000, [1], [1], 7, 1, 128, 128, 32),
    (100, [150, 40], [100, 40], 4, 2, 128, 64, 16), (1, [2000], [1500], 4, 2, 128, 128, 16),
    (4097, [3] * 65, [1] * 65, 1, 1, 128, 128, 16), (900, [20] * 500, [1] * 500, 4, 1, 64, 64, 16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%d-%dreq-%d" % (s[0], len(s[1]), sum(s[2])))
def test_prefix(lib, shape):
    prefix, lens, adds, hq, hkv, d, group, page = shape
    Batch(lib, prefix, lens, adds, hq, hkv, d, group, page, seed=prefix).check()


@pytest.mark.parametrize("adds", [[1, 1, 1], [90, 1, 40]])
def test_empty_sides(lib, adds):
    """No prefix, no own tokens, neither; more queries than own tokens; a request without queries."""
    b = Batch(lib, 200, [100, 40, 50], adds, 8, 2, 128, 128, 16)
    b.prefix_len.zero_()
    b.check()
    b.prefix_len.fill_(-5)
    b.check()
    b.prefix_len.fill_(200)
    b.lens[1] = 0
    b.lens[2] = 0
    b.check()
    b.prefix_len.zero_()
    got = b.check()
    a = int(b.start[1])
    assert (got[a:] == 0).all()  # nothing to see
    b.prefix_len.fill_(10 ** 6)  # more than its table holds
    b.lens[:] = torch.tensor([100, 40, 50])
    b.check()
    # rows of no request are left
    b.start[1] = b.start[0]
    before = torch.full_like(b.q, 5.0)
    got = b.run(out=before.clone())
    assert (got[:0] == 5.0).all() and int(b.start[1]) == 0
    b.start[0] = b.start[1] = int(b.start[2]) - 1
    got = b.run(out=before.clone())
    assert (got[:int(b.start[1])] == 5.0).all() and got[int(b.start[1]):].isfinite().all()


@pytest.mark.parametrize("d,group,adds", [(128, 128, [1, 1]), (128, 128, [80, 70]), (64, 64, [2, 2]), (128, 64, [1, 3])])
def test_missing_pages_and_leftovers(lib, d, group, adds):
    """Pages outside the cache hold nothing, on either side; slots behind an end may hold anything."""
    b = Batch(lib, 250, [150, 77], adds, 8, 2, d, group, 16)
    par = b.cache.blocks[:, :, 16 * d:].view(torch.uint8).unflatten(-1, (2, 16, 4 * d // group))
    par[b.prefix_table[-1].long(), :, :, 250 % 16:] = 255  # NaN behind the prefix's last token
    par[b.table[1, 77 // 16].long(), :, :, 77 % 16:] = 255
    b.check()
    b.prefix_table[3] = -1
    b.prefix_table[7] = b.cache.num_pages
    b.table[0, 2] = 2 ** 31 - 1
    b.check()


def test_nan_shows_where_it_is_seen(lib):
    b = Batch(lib, 100, [40, 60], [1, 1], 8, 2, 128, 128, 16)
    par = b.cache.blocks[:, :, 16 * 128:].view(torch.uint8).unflatten(-1, (2, 16, 4))
    page = int(b.table[0, 1])
    par[page, 1, 1, 3] = 255  # a value of request 0's own, key head 1
    got = b.run()
    assert got[0, 4:].isnan().all() and not got[0, :4].isnan().any() and not got[1].isnan().any()
    par[int(b.prefix_table[2]), 0, 0, 5] = 255  # a key of the prefix, key head 0
    got = b.run()
    assert got[:, :4].isnan().all() and not got[1, 4:].isnan().any()


@pytest.mark.parametrize("adds", [[1, 1, 1], [100, 30, 1]])
def test_like_attention_over_one_table(lib, adds):
    """Where the prefix fills its pages, a table of both parts gives the same to the roundings."""
    b = Batch(lib, 320, [120, 47, 200], adds, 16, 4, 128, 128, 16)
    got = b.run()
    table = torch.cat((b.prefix_table.expand(3, -1), b.table), 1).contiguous()
    one = lib.kv4_attention(b.cache, b.q, b.start, (b.lens + 320).int(), table, b.max_q)
    _, tol = b.exact()
    assert ((got.double() - one.double()).abs() <= 2 * tol + 2.0 ** -23).all()


def test_repeatable_captured_and_on_other_streams(lib, monkeypatch):
    b = Batch(lib, 3000, [300, 40, 9, 150], [120, 1, 1, 70], 16, 4, 128, 128, 16)
    out = torch.empty_like(b.q)
    ws = b.cache.prefix_workspace(16, b.q.shape[0], b.max_q)
    first = b.run(out=out, workspace=ws).clone()
    assert torch.equal(first, b.run(out=out, workspace=ws))
    b.prefix_len.fill_(2001)
    want = b.run().clone()
    b.prefix_len.fill_(3000)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            b.run(out=out, workspace=ws)
    b.prefix_len.fill_(2001)  # lengths are read when the graph runs
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for way in (lib._short, lib._LongWay):
        monkeypatch.setattr(lib, "_short", way)
        out.zero_()
        torch.cuda.synchronize()
        b.run(out=out, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(lib.kv4_attention_prefix(b.cache, b.q, b.start, b.lens, b.table, b.prefix_len, b.prefix_table,
                                                b.max_q), want)
    lib.tl_check_status()


def test_strided_rows(lib):
    """Queries as columns of a fused projection's rows, outputs in a wider matrix."""
    b = Batch(lib, 500, [60, 10], [70, 1], 8, 2, 128, 128, 16)
    b.lens[0] = 70
    b.check()
    want = b.run()
    fused = torch.randn(71, 16, 128, device="cuda").half()
    fused[:, 3:11] = b.q
    b.q = fused[:, 3:11]
    wide = torch.full((71, 10, 128), 2.0, dtype=torch.float16, device="cuda")
    b.run(out=wide[:, 1:9])
    assert torch.equal(wide[:, 1:9], want) and (wide[:, 0] == 2).all() and (wide[:, 9] == 2).all()


def test_contradicting_lengths_write_within_their_rows(lib):
    """Requests whose queries overlap or run backwards: the numbers of such rows mean nothing, rows of sound
    requests are right (the work, and so the sums, may be split elsewhere), and the rows of no request are left."""
    b = Batch(lib, 700, [90, 120, 40, 30], [20, 60, 1, 1], 16, 4, 128, 128, 16)
    want, (exact, tol) = b.run(), b.exact()
    start = b.start.tolist()
    out = torch.full((len(b.q) + 8, 16, 128), 9.0, dtype=torch.float16, device="cuda")[:len(b.q)]
    for bad in ([0, 20, 10, 81, 82], [0, 50, 30, 81, 82], [5, 5, 80, 81, 82], [0, 90, 80, 81, 82], [-3, 20, 80, 81, 82],
                [2 ** 31 - 1, -2 ** 31, 80, 81, 82]):
        b.start[:] = torch.tensor(bad, dtype=torch.int32)
        out.fill_(9.0)
        b.run(out=out)
        torch.cuda.synchronize()
        assert ((out[81].double() - exact[81]).abs() <= tol[81] + 2.0 ** -24).all()  # the last request is sound in each
    lib.tl_check_status()
    b.start[:] = torch.tensor(start, dtype=torch.int32)
    assert torch.equal(b.run(), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("adds", [[1] * 33, [2, 47, 1], [200, 3]])
def test_both_ways(lib, d, adds, monkeypatch):
    """The same batch by one kernel and by both: within both bounds, and any prefix length behind either table."""
    lens = [a + 37 * i % 151 for i, a in enumerate(adds)]
    got = []
    for spare in (0, 30000):
        monkeypatch.setattr(Batch, "spare", spare)
        b = Batch(lib, 700, lens, adds, 8, 2, d, d, 16, seed=5)
        for n in (700, 1, 129, 0, 640):
            b.prefix_len.fill_(n)
            got.append(b.check().double())
        _, tol = b.exact()
    for one, two in zip(got[:5], got[5:]):
        assert ((one - two).abs() <= 4 * tol + 2.0 ** -22).all()
