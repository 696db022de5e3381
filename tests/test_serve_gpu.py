"""The serving operators on the GPU against their definitions in 64 bits.

Tolerances, from the formulas (u = 2^-11, half a step of FP16 relative to the
value):

* attention.  With weights p (summing to 1) and values |v| <= V over the keys a
  row sees: the output's rounding is u |o|.  Rounding the weights changes the
  mean by at most 2 u V; rounding each value to FP16 (prompt-sized rows may run
  on FP16 tiles) by u V; rounding each key to FP16 shifts a logit by at most
  dS = scale * u * max_t sum |q||k_t|, a weighted mean by at most 2 dS V.  FP32
  sums stay below all of these.  Bound: u |o| + 3 u V + 2 dS V.
* adapters.  u |out| for the output and n 2^-24 mag for the FP32 sums, with
  mag = scale |B| (|A| |x|) and n = K / 8 + rank + 16 roundings in a chain
  (the matrix instruction adds eight products at a time).
* cache and tables are exact.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -11


def quantize_rows(x, group):
    """Codes, scales, minima of FP16 rows [..., D] in binary32 steps."""
    x = np.asarray(x, np.float16).astype(np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    s = np.maximum(((hi - lo) / np.float32(15)).astype(np.float16), np.float16(2.0 ** -24)).astype(np.float32)
    b = lo.astype(np.float16).astype(np.float32)
    c = np.clip(np.rint((g - b) / s), 0, 15)
    return c.reshape(x.shape).astype(np.uint8), s[..., 0].astype(np.float16), b[..., 0].astype(np.float16)


def block_rows(blocks, page, d, group, slot, part):
    """(codes, parameters) of every head of one token, straight from the layout."""
    blk = blocks[slot // page].reshape(blocks.shape[1], -1)
    off, half, pw = slot % page, page * d // 2, 4 * (d // group)
    codes = blk[:, part * half + off * (d // 2):part * half + (off + 1) * (d // 2)]
    at = 2 * half + part * page * pw + off * pw
    par = np.ascontiguousarray(blk[:, at:at + pw]).view(np.float16).reshape(blk.shape[0], -1, 2)
    return np.stack([codes & 15, codes >> 4], -1).reshape(blk.shape[0], d), par


def kv_values(rng, t, h, d):
    x = rng.standard_normal((t, h, d)).astype(np.float32)
    x[..., ::29] *= 4
    x *= 10.0 ** rng.uniform(-2, 1, size=(t, h, 1))
    return x.astype(np.float16)


def odd_rows(x):
    """Rows whose range or spacing is a corner of the formula."""
    t = x.shape[0]
    x = x.copy()
    if t > 0:
        x[0] = 0
    if t > 1:
        x[1] = np.float16(-3.1416)
    if t > 2:
        x[2] = np.float16(6e-8) * (np.arange(x.shape[-1]) % 3)
    if t > 3:
        x[3, :, 0], x[3, :, 1:] = np.float16(65504), np.float16(-65504)
    if t > 4:
        x[4] = (np.arange(x.shape[-1]) % 31) * np.float16(0.5)  # exact halves between levels
    return x


@pytest.mark.parametrize("d,group,page,heads,t", [(128, 128, 16, 16, 5), (128, 64, 64, 3, 33), (64, 64, 16, 1, 1),
                                                  (64, 64, 256, 5, 257), (128, 128, 32, 8, 100)])
@pytest.mark.parametrize("fused", [False, True])
def test_append_and_read_exact(lib, d, group, page, heads, t, fused):
    rng = np.random.default_rng(d + page + t)
    k, v = odd_rows(kv_values(rng, t, heads, d)), odd_rows(kv_values(rng, t, heads, d))
    pages = -(-t // page) + 3
    cache = lib.KV4Cache(pages, heads, d, page, group)
    cache.blocks.fill_(0xA5)
    slots = rng.permutation(pages * page)[:t].astype(np.int64)
    passed = rng.random(t) < 0.2
    passed[:5] = False
    slots[passed] = np.where(rng.random(passed.sum()) < 0.5, -1, pages * page + 7)
    if fused:
        rows = torch.zeros((t, 3, heads, d), dtype=torch.float16, device="cuda")
        rows[:, 1], rows[:, 2] = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
        kt, vt = rows[:, 1], rows[:, 2]
    else:
        kt, vt = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    st = torch.from_numpy(slots).cuda()
    lib.tl_kv4_append(cache, kt, vt, st)
    ko, vo = (torch.full((t, heads, d), 7.0, dtype=torch.float16, device="cuda") for _ in "kv")
    lib.tl_kv4_read(cache, st, ko, vo)
    blocks = cache.blocks.cpu().numpy()
    for part, x, got in ((0, k, ko), (1, v, vo)):
        c, s, b = quantize_rows(x, group)
        val = (c.astype(np.float64).reshape(t, heads, -1, group) * s[..., None].astype(np.float64)
               + b[..., None].astype(np.float64)).astype(np.float32)
        with np.errstate(over="ignore"):  # the sixteenth level of the widest row lies past FP16's largest number
            val = val.astype(np.float16).reshape(t, heads, d)
        got = got.cpu().numpy()
        for i in range(t):
            if passed[i]:
                assert not got[i].any()
                continue
            codes, par = block_rows(blocks, page, d, group, int(slots[i]), part)
            assert np.array_equal(codes, c[i]), (part, i)
            assert np.array_equal(par[..., 0], s[i]) and np.array_equal(par[..., 1], b[i])
            assert np.array_equal(got[i], val[i])
    # nothing else was touched
    keep = np.ones((pages, page), bool)
    ok = slots[~passed]
    keep[ok // page, ok % page] = False
    for p, o in zip(*np.nonzero(keep)):
        for part in (0, 1):
            codes, par = block_rows(blocks, page, d, group, int(p) * page + int(o), part)
            assert (codes == np.tile([5, 10], d // 2)).all() and (par.view(np.uint16) == 0xA5A5).all()


def plan_reference(cached, added, table, free, head, page, num_pages, room):
    table = table.copy()
    req, pos, slot = (np.full(room, -1, np.int64) for _ in range(3))
    start, want, taken, t = [0], 0, 0, 0
    for b, (c, a) in enumerate(zip(np.maximum(cached, 0).tolist(), np.maximum(added, 0).tolist())):
        held, need = -(-c // page), -(-(c + a) // page) - (-(-c // page))
        want += need
        width = table.shape[1]
        for i in range(held, min(held + need, width)):
            at = head + taken_before(cached, added, page, width, b) + i - min(held, width)
            table[b, i] = free[at] if at < len(free) else -1
        taken += max(0, min(held + need, width) - min(held, width))
        for i in range(a):
            if t + i < room:
                p = c + i
                pg = table[b, p // page] if p // page < width else -1
                req[t + i], pos[t + i] = b, p
                slot[t + i] = pg * page + p % page if 0 <= pg < num_pages else -1
        t += a
        start.append(t)
    taken = min(taken, max(0, len(free) - head))
    return dict(table=table, q_start=np.array(start), seq_lens=np.maximum(cached, 0) + np.maximum(added, 0),
                token_req=req, token_pos=pos, slots=slot, counts=np.array([t, taken, head + taken, want - taken]))


def taken_before(cached, added, page, width, b):
    c, a = np.maximum(cached[:b], 0), np.maximum(added[:b], 0)
    return int((np.minimum(-(-(c + a) // page), width) - np.minimum(-(-c // page), width)).sum())


@pytest.mark.parametrize("n,page,top_c,top_a,short,narrow,room,head", [
    (1, 16, 0, 1, 0, 0, 0, None), (3, 16, 100, 1, 0, 0, 5, 0), (17, 64, 300, 90, 0, 0, -30, 3),
    (256, 16, 40, 3, 0, 0, 1, None), (257, 32, 100, 70, 0, 0, 0, 11), (700, 16, 200, 20, 0, 0, 333, 2),
    (40, 16, 64, 64, 25, 0, 0, 1), (40, 16, 64, 64, 0, 2, 0, None), (5, 16, 0, 0, 0, 0, 4, None), (0, 16, 0, 0, 0, 0, 3, 0)])
def test_plan_exact(lib, n, page, top_c, top_a, short, narrow, room, head):
    rng = np.random.default_rng(n + page + top_a)
    cached = rng.integers(-2 if n > 4 else 0, top_c + 1, n).astype(np.int32)
    added = rng.integers(-1 if n > 4 else 0, top_a + 1, n).astype(np.int32)
    if n == 1:
        cached[:], added[:] = 0, 1
    width = max(1, -(-(top_c + top_a) // page) - narrow)
    pages = n * (width + 1) + 20
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((n, width), -5, np.int32)
    at = 0
    for b in range(n):
        h = min(width, -(-max(cached[b], 0) // page))
        table[b, :h] = order[at:at + h]
        at += h
    if n > 20:
        table[3, 0] = pages + 3   # not a page of the cache
    h0 = head or 0
    need = taken_before(cached, added, page, width, n)
    free = np.concatenate([np.full(h0, -9, np.int32), order[at:at + max(0, need - short) + (0 if short else 7)]])
    room = int(np.maximum(added, 0).sum()) + room
    ref = plan_reference(cached, added, table, free, h0, page, pages, room)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    t = dev(table)
    out = {k: torch.full((m,), 99, dtype=torch.int64 if k == "slots" else torch.int32, device="cuda")
           for k, m in (("q_start", n + 1), ("seq_lens", n), ("token_req", room), ("token_pos", room),
                        ("slots", room), ("counts", 4))}
    hd = None if head is None else torch.tensor([head], dtype=torch.int32, device="cuda")
    for _ in range(2):  # a repeated call gives the same tables
        lib.tl_kv_plan(dev(cached), dev(added), t, dev(free), *out.values(), page_size=page, num_pages=pages,
                       free_head=hd)
    out["table"] = t
    for k, want in ref.items():
        assert np.array_equal(out[k].cpu().numpy(), want), k


class Case:
    """A filled cache, its values in 64 bits, and a batch over it."""

    def __init__(self, lib, lens, adds, hq, hkv, d, group, page, seed, spare=3, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.adds, self.hq, self.hkv, self.d, self.page = lens, adds, hq, hkv, d, page
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        self.cache = lib.KV4Cache(pages, hkv, d, page, group)
        self.cache.blocks.fill_(0xFF)  # NaN scales and minima wherever no token is
        order = rng.permutation(pages)
        width = max(need + [1]) + 1
        table = np.full((len(lens), width), -1, np.int32)
        self.k, self.v, slots, ks, vs = [], [], [], [], []
        at = 0
        for i, n in enumerate(lens):
            table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
            k, v = kv_values(rng, n, hkv, d), kv_values(rng, n, hkv, d)
            pos = np.arange(n)
            slots.append(table[i][pos // page].astype(np.int64) * page + pos % page)
            ks.append(k)
            vs.append(v)
            self.k.append(self.values(k, group))
            self.v.append(self.values(v, group))
        lib.tl_kv4_append(self.cache, *(torch.from_numpy(np.concatenate(x)).cuda() for x in (ks, vs, slots)))
        self.table = torch.from_numpy(table).cuda()
        self.start_host = np.concatenate([[0], np.cumsum(adds)]).astype(np.int32)
        self.start = torch.from_numpy(self.start_host).cuda()
        self.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = (rng.standard_normal((self.start_host[-1], hq, d)) * qscale).astype(np.float16)

    @staticmethod
    def values(x, group):
        c, s, b = quantize_rows(x, group)
        g = c.astype(np.float64).reshape(x.shape[:-1] + (x.shape[-1] // group, group))
        return (g * s[..., None].astype(np.float64) + b[..., None].astype(np.float64)).reshape(x.shape)

    def reference(self, scale, window=0, drop=()):
        """(output, bound); drop: (request, page index) pairs that hold no tokens."""
        out = np.zeros(self.q.shape)
        bound = np.zeros(self.q.shape)
        share = self.hq // self.hkv
        for i, (n, a) in enumerate(zip(self.lens, self.adds)):
            for t in range(a):
                p = n - a + t
                keys = np.arange(max(0, p - window + 1) if window else 0, max(0, p + 1))
                keys = keys[[(i, key // self.page) not in drop for key in keys]] if len(drop) else keys
                if len(keys) == 0:
                    continue
                row = self.start_host[i] + t
                q = self.q[row].astype(np.float64).reshape(self.hkv, share, self.d)
                k, v = self.k[i][keys].transpose(1, 0, 2), self.v[i][keys].transpose(1, 0, 2)
                s = scale * q @ k.transpose(0, 2, 1)
                w = np.exp(s - s.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o = w @ v
                vmax = np.abs(v).max(axis=(1, 2), keepdims=True)
                ds = abs(scale) * U * (np.abs(q) @ np.abs(k).transpose(0, 2, 1)).max(-1, keepdims=True)
                out[row] = o.reshape(self.hq, self.d)
                bound[row] = (U * np.abs(o) + 3 * U * vmax + 2 * ds * vmax).reshape(self.hq, self.d)
        return out, bound

    def run(self, lib, scale, window=0, q=None, **kw):
        q = torch.from_numpy(self.q).cuda() if q is None else q
        return lib.kv4_attention(self.cache, q, self.start, self.seq, self.table, max(self.adds + [0]), scale, window,
                                 **kw)


def check(got, ref, bound, what=""):
    got = got.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), what
    worst = np.abs(got - ref) - bound
    assert (worst <= 0).all(), "%s: off by %.3e where %.3e is allowed" % (
        what, np.abs(got - ref).flat[worst.argmax()], bound.flat[worst.argmax()])
    norm = np.linalg.norm(ref)
    if norm > 0:
        assert np.linalg.norm(got - ref) <= 2e-3 * norm, what


FORMS = [(128, 128), (128, 64), (64, 64)]


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (7, 1), (12, 1), (16, 1), (6, 3), (40, 2)])
def test_decode(lib, d, group, hq, hkv):
    lens = [1, 2, 15, 16, 17, 127, 128, 129, 300, 1000]
    c = Case(lib, lens, [1] * len(lens), hq, hkv, d, group, 16, seed=hq + d)
    check(c.run(lib, d ** -0.5), *c.reference(d ** -0.5))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,group", FORMS)
def test_pages(lib, page, d, group):
    lens = [page - 1, page, page + 1, 3 * page + 5, 2000]
    c = Case(lib, lens, [1, 2, 3, 1, 4], 4, 2, d, group, page, seed=page)
    check(c.run(lib, d ** -0.5), *c.reference(d ** -0.5))


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("window", [0, 1, 2, 16, 17, 100, 5000])
@pytest.mark.parametrize("hq,hkv,adds", [(4, 2, [1, 3, 5, 2]), (9, 3, [4, 1, 8, 33]), (8, 1, [17, 70, 40, 1])])
def test_window_and_several_queries(lib, d, group, window, hq, hkv, adds):
    lens = [130, 77, 400, 40]
    c = Case(lib, [max(n, a) for n, a in zip(lens, adds)], adds, hq, hkv, d, group, 32, seed=window + hq)
    check(c.run(lib, d ** -0.5, window), *c.reference(d ** -0.5, window))


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 1), (6, 2)])
@pytest.mark.parametrize("window", [0, 50])
def test_prompts(lib, d, group, hq, hkv, window):
    """Whole prompts and chunks behind cached tokens, beside decoding requests
    and a request without queries."""
    adds, lens = [300, 1, 0, 129, 257, 64, 1], [300, 50, 20, 500, 700, 64, 1]
    c = Case(lib, lens, adds, hq, hkv, d, group, 16, seed=hq + d + window)
    check(c.run(lib, d ** -0.5, window), *c.reference(d ** -0.5, window))


@pytest.mark.parametrize("adds", [[1, 3, 2, 4], [300, 3, 200, 140]])
def test_rows_that_see_nothing(lib, adds):
    """More queries than tokens: the first rows see no key and give zeros."""
    lens = [0, 1, 0, 3]
    for window in (0, 2):
        c = Case(lib, lens, adds, 4, 2, 128, 128, 16, seed=5)
        out = c.run(lib, 0.1, window)
        check(out, *c.reference(0.1, window))
        assert not out[:adds[0]].any()


def test_batches_of_nothing(lib):
    c = Case(lib, [5, 0, 9], [0, 0, 0], 4, 2, 64, 64, 16, seed=6)
    assert c.run(lib, 0.1).shape == (0, 4, 64)
    c = Case(lib, [5, 0, 9], [0, 0, 1], 4, 2, 64, 64, 16, seed=6)
    check(c.run(lib, 0.1), *c.reference(0.1))


@pytest.mark.parametrize("adds", [[1, 1, 1], [200, 260, 130]])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, 60])
def test_pages_outside_the_cache(lib, bad, adds):
    """Such a page holds no tokens; nothing is read through it."""
    c = Case(lib, [300, 290, 140], adds, 4, 2, 128, 64, 16, seed=7)
    assert c.cache.num_pages <= 60
    drop = [(0, 0), (0, 7), (0, 18), (1, 3), (2, 8)] + [(2, j) for j in range(8)]
    for i, j in drop:
        c.table[i, j] = bad
    ref = c.reference(0.1, drop=set(drop))
    check(c.run(lib, 0.1), *ref)
    assert not ref[0][c.start_host[2]:].any()  # the third request has no page left


def test_queries_outside_the_rows_count_as_none(lib):
    c = Case(lib, [50, 60, 70], [2, 1, 3], 4, 2, 64, 64, 16, seed=8)
    ref, bound = c.reference(0.1)
    q = torch.from_numpy(c.q).cuda()
    for start in ([0, 2, 3, 600], [-4, 2, 3, 3], [0, 2, 1, 1]):
        out = torch.full(q.shape, 5.0, dtype=torch.float16, device="cuda")
        lib.tl_kv4_attention(c.cache, q, out, torch.tensor(start, dtype=torch.int32, device="cuda"), c.seq, c.table,
                             3, 0.1, workspace=c.cache.attention_workspace(4, 3))
        torch.cuda.synchronize()
        good = [i for i in range(3) if start[i] >= 0 and start[i + 1] - start[i] == c.adds[i]
                and start[i + 1] <= 6 and start[i] == c.start_host[i]]
        rows = [r for i in good for r in range(c.start_host[i], c.start_host[i + 1])]
        check(out[rows], ref[rows], bound[rows])


@pytest.mark.parametrize("adds", [[1, 1], [150, 140]])
def test_hostile_scales(lib, adds):
    """Queries from the smallest to the largest FP16 numbers, values whose
    scales differ by 2^20 between tokens."""
    for qscale, scale in ((1e-7, 1e6), (2e-5, 1e3), (1.0, 0.1), (9000.0, 1e-5)):
        c = Case(lib, [200, 170], adds, 4, 2, 128, 128, 16, seed=9, qscale=qscale)
        check(c.run(lib, scale), *c.reference(scale), what="q %g" % qscale)


def test_constant_values_come_back(lib):
    """Value rows that are constant have the smallest scale: the mean of
    equal numbers is that number."""
    c = Case(lib, [100], [1], 2, 2, 128, 64, 16, seed=10)
    slots = (c.table[0, torch.arange(100, device="cuda") // 16].long() * 16 + torch.arange(100, device="cuda") % 16)
    k = torch.randn(100, 2, 128, device="cuda").half()
    lib.tl_kv4_append(c.cache, k, torch.full_like(k, -1.25), slots)
    assert (c.run(lib, 0.1) == -1.25).all()


def test_strided_rows_streams_and_graphs(lib):
    """Queries inside fused rows, outputs with a stride, work on another
    stream, and a captured step replayed after the requests have grown."""
    c = Case(lib, [90, 33, 300], [1, 1, 1], 8, 4, 128, 128, 16, seed=11)
    rows = torch.zeros((3, 8 + 8, 128), dtype=torch.float16, device="cuda")
    wide = torch.full((3, 10, 128), 3.0, dtype=torch.float16, device="cuda")
    rows[:, :8] = torch.from_numpy(c.q).cuda()
    ws = c.cache.attention_workspace(8, 1)
    ref, bound = c.reference(0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    lib.tl_kv4_attention(c.cache, rows[:, :8], wide[:, 1:9], c.start, c.seq, c.table, 1, 0.1, workspace=ws, stream=side)
    side.synchronize()
    check(wide[:, 1:9], ref, bound)
    assert (wide[:, 0] == 3).all() and (wide[:, 9] == 3).all()
    # a graph of the step: lengths live on the GPU
    seq = torch.tensor([40, 20, 100], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    out = torch.empty((3, 8, 128), dtype=torch.float16, device="cuda")
    q = torch.from_numpy(c.q).cuda()
    with torch.cuda.graph(graph):
        lib.tl_kv4_attention(c.cache, q, out, c.start, seq, c.table, 1, 0.1, workspace=ws)
    graph.replay()
    seq.copy_(c.seq)
    graph.replay()
    torch.cuda.synchronize()
    check(out, ref, bound)
    first = out.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


@pytest.mark.parametrize("adds", [[1] * 6, [130, 1, 1, 200, 3, 64]])
def test_same_bits_every_time(lib, adds):
    c = Case(lib, [1500, 20, 700, 300, 2500, 64], adds, 8, 2, 128, 128, 16, seed=12)
    first = c.run(lib, 0.1)
    for _ in range(3):
        assert torch.equal(first, c.run(lib, 0.1))
    check(first, *c.reference(0.1))


@pytest.mark.parametrize("adds", [[1, 3], [40, 129]])
def test_cache_beyond_32_bit_offsets(lib, adds):
    """Pages past 4 GB of the cache."""
    lens, d, page, hkv = [100, 200], 128, 16, 8
    pages = (5 << 30) // (hkv * 2176)
    c = Case(lib, lens, adds, 16, hkv, d, 128, page, seed=13)
    big = lib.KV4Cache(pages, hkv, d, page, 128)
    moved = pages - 1 - torch.arange(c.cache.num_pages, device="cuda")
    big.blocks[moved] = c.cache.blocks
    table = torch.where(c.table >= 0, (pages - 1 - c.table).int(), c.table)
    q = torch.from_numpy(c.q).cuda()
    out = lib.kv4_attention(big, q, c.start, c.seq, table, max(adds), 0.1)
    check(out, *c.reference(0.1))
    k = torch.randn(2, hkv, d, device="cuda").half()
    slots = torch.tensor([pages * page - 1, pages * page - 40], device="cuda")
    lib.tl_kv4_append(big, k, k, slots)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    lib.tl_kv4_read(big, slots, ko, vo)
    cq, s, b = quantize_rows(k.cpu().numpy(), 128)
    val = (cq.astype(np.float64) * s.astype(np.float64) + b.astype(np.float64)).astype(np.float32).astype(np.float16)
    assert np.array_equal(ko.cpu().numpy(), val) and np.array_equal(vo.cpu().numpy(), val)


@pytest.mark.parametrize("K,N,rank", [(64, 64, 8), (256, 512, 16), (2048, 6144, 16), (264, 328, 24), (512, 200, 64),
                                      (8, 8, 40), (1032, 96, 32)])
@pytest.mark.parametrize("adds,adapters", [([1, 1, 1, 1], [0, 2, -1, 1]), ([5, 0, 17, 100], [1, 1, 0, 7]),
                                           ([300], [2]), ([1], [0])])
@pytest.mark.parametrize("in_place", [False, True])
def test_lora(lib, K, N, rank, adds, adapters, in_place):
    rng = np.random.default_rng(K + N + rank + len(adds))
    T, num = sum(adds), 3
    x = rng.standard_normal((T, K)).astype(np.float16)
    y = rng.standard_normal((T, N)).astype(np.float16)
    A = (rng.standard_normal((num, rank, K)) / K ** 0.5).astype(np.float16)
    B = (rng.standard_normal((num, N, rank)) / rank ** 0.5).astype(np.float16)
    sc = rng.uniform(-2, 2, num).astype(np.float32)
    start = np.concatenate([[0], np.cumsum(adds)]).astype(np.int32)
    ref, bound = y.astype(np.float64), np.zeros((T, N))
    for i, w in enumerate(adapters):
        if 0 <= w < num:
            r = slice(start[i], start[i + 1])
            xd, Ad, Bd = x[r].astype(np.float64), A[w].astype(np.float64), B[w].astype(np.float64)
            ref[r] += float(sc[w]) * xd @ Ad.T @ Bd.T
            mag = abs(float(sc[w])) * (np.abs(xd) @ np.abs(Ad).T @ np.abs(Bd).T)
            bound[r] = U * np.abs(ref[r]) + (K / 8 + rank + 16) * 2.0 ** -24 * mag + 2.0 ** -25
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    yt = dev(y)
    out = yt if in_place else torch.full_like(yt, 9.0)
    lib.tl_lora_add(dev(x), dev(A), dev(B), dev(sc), dev(start), torch.tensor(adapters, dtype=torch.int32).cuda(),
                    max(adds), yt, out)
    got = out.cpu().numpy().astype(np.float64)
    assert (np.abs(got - ref) <= bound).all(), np.abs(got - ref).max()


def test_lora_large_sums_and_strides(lib):
    """A x beyond FP16's range; x, y and out as columns of wider rows; rows of
    no request are left alone."""
    T, K, N, rank = 6, 512, 256, 16
    g = torch.Generator().manual_seed(3)
    x = (torch.rand(T, K, generator=g) * 1000).half()
    A = torch.rand(1, rank, K, generator=g).half()          # A x is near 256000
    B = (torch.randn(1, N, rank, generator=g) * 1e-4).half()
    y = torch.randn(T, N, generator=g).half()
    xw, yw = torch.zeros(T, K + 64).half(), torch.zeros(T, 3 * N).half()
    xw[:, 64:], yw[:, N:2 * N] = x, y
    xw, yw = xw.cuda(), yw.cuda()
    start = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()  # rows 4 and 5 belong to nobody
    lib.tl_lora_add(xw[:, 64:], A.cuda(), B.cuda(), torch.tensor([0.5]).cuda(), start,
                    torch.tensor([0, 0], dtype=torch.int32).cuda(), 2, yw[:, N:2 * N], yw[:, N:2 * N])
    xd, Ad, Bd = x.double(), A[0].double(), B[0].double()
    ref = y.double()
    ref[:4] += 0.5 * (xd @ Ad.t() @ Bd.t())[:4]
    bound = U * ref.abs() + (K / 8 + rank + 16) * 2.0 ** -24 * 0.5 * (xd.abs() @ Ad.abs().t() @ Bd.abs().t())
    got = yw.cpu()
    assert ((got[:, N:2 * N].double() - ref).abs()[:4] <= bound[:4]).all()
    assert torch.equal(got[4:, N:2 * N], y[4:]) and not got[:, :N].any() and not got[:, 2 * N:].any()


def test_one_serving_step(lib):
    """Plan, adapters, append and attention together over several steps,
    against one pass over all tokens at the end."""
    rng = np.random.default_rng(21)
    hq, hkv, d, page, n = 4, 2, 64, 16, 3
    pages, width = 40, 10
    cache = lib.KV4Cache(pages, hkv, d, page, 64)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    free = torch.from_numpy(rng.permutation(pages).astype(np.int32)).cuda()
    counts = [torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2)]
    cached = torch.zeros(n, dtype=torch.int32, device="cuda")
    got, ks, vs, qs = [[] for _ in range(n)], [[] for _ in range(n)], [[] for _ in range(n)], [[] for _ in range(n)]
    for step, added in enumerate([[20, 1, 33], [1, 1, 1], [1, 0, 2], [17, 1, 1]]):
        t = sum(added)
        head = counts[step % 2][2:3]
        a = torch.tensor(added, dtype=torch.int32, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        q_start, seq, req, pos = (torch.empty(m, **i32) for m in (n + 1, n, t, t))
        slots = torch.empty(t, dtype=torch.int64, device="cuda")
        out_counts = counts[(step + 1) % 2]
        lib.tl_kv_plan(cached, a, table, free, q_start, seq, req, pos, slots, out_counts, page_size=page,
                       num_pages=pages, free_head=head)
        q, k, v = (torch.from_numpy(kv_values(rng, t, h, d)).cuda() for h in (hq, hkv, hkv))
        lib.tl_kv4_append(cache, k, v, slots)
        o = lib.kv4_attention(cache, q, q_start, seq, table, max(added))
        at = 0
        for i, m in enumerate(added):
            for lst, x in ((got, o), (ks, k), (vs, v), (qs, q)):
                lst[i].append(x[at:at + m].cpu())
            at += m
        cached = seq
        assert out_counts.cpu()[3] == 0
    for i in range(n):
        kd, vd = (torch.from_numpy(Case.values(torch.cat(x[i]).numpy(), 64)) for x in (ks, vs))
        q, o = torch.cat(qs[i]).double(), torch.cat(got[i]).double()
        m = q.shape[0]
        for h in range(hq):
            s = (q[:, h] @ kd[:, h // 2].t()) * d ** -0.5
            s = s.masked_fill(torch.arange(m)[None] > torch.arange(m)[:, None], float("-inf"))
            want = torch.softmax(s, -1) @ vd[:, h // 2]
            vmax = vd[:, h // 2].abs().max()
            ds = d ** -0.5 * U * (q[:, h].abs() @ kd[:, h // 2].abs().t()).max(-1, keepdim=True).values
            assert ((o[:, h] - want).abs() <= U * want.abs() + (3 * U + 2 * ds) * vmax).all()
