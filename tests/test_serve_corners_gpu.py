"""Corners of the serving attention: value scales that differ, lengths that do
not fit, and tokens that are not finite, against definitions in 64 bits.

Tolerances (U = 2^-11, half a step of FP16 relative to the value).  Keys and
value codes enter the products exactly; what is rounded is each weight p s'
once (the second product), the output once, and the logits in FP32.

* A weight's rounding moves o by at most U p_t |c_t - 8| s'_t with
  8 s' <= (8 / 15) (max - min) <= (16 / 15) V, V the largest value of the
  channel's group: 2 U V with what FP16 leaves out of the smallest weights
  (below 2^-31 of the largest: n 2^-28 V / 7.5 for n tokens, n <= 2^17).
* The output: U |o|, or half of FP16's smallest step, 2^-25.
* A logit is a sum of at most 128 products and two more terms, each rounded or
  cut to 2^-20 of the largest: dS = scale 2^-17 sum |q| (|b| + 15 s), and a
  weighted mean moves by at most 2 dS V.
* For independent tokens these add up as squares: the norm of the difference
  is held to 3 U of the norm, U for each of the three (and FP16's smallest half
  steps, 2^-25 each).
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -11
FORMS = [(128, 128), (128, 64), (64, 64)]


def value_gains(kind, t, h, d, gen):
    """Factors of the value rows [t, h, d]."""
    rand = lambda *s: torch.rand(*s, device="cuda", generator=gen)  # noqa: E731
    if kind == "zero rows":
        return (rand(t, h, 1) < 0.5).float()
    if kind == "zero half":
        return (torch.arange(d, device="cuda") >= 64).float().expand(t, h, d)
    if kind == "wide rows":  # scales over a factor of 2^22
        return 2.0 ** (22 * rand(t, h, 1) - 14)
    if kind == "wide halves":  # the scales of the two groups 2^21 apart
        return torch.where(torch.arange(d, device="cuda") >= 64, 2.0 ** 13, 2.0 ** -8).expand(t, h, d)
    return torch.ones(t, h, d, device="cuda")


class Batch:
    """A filled cache and queries whose logits have the given spread."""

    def __init__(self, lib, lens, adds, hq, hkv, d, group, page=16, spread=1.0, kind="", seed=1, width=None):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.lib, self.lens, self.adds, self.hq = lib, lens, adds, hq
        need = [-(-n // page) for n in lens]
        self.cache = lib.KV4Cache(sum(need) + 2, hkv, d, page, group)
        self.cache.blocks.fill_(0xFF)  # NaN scales and minima wherever no token is
        order = torch.randperm(sum(need) + 2, device="cuda", generator=gen).int()
        self.table = torch.full((len(lens), width or max(need + [1])), -1, dtype=torch.int32, device="cuda")
        at, self.slots = 0, []
        for i, n in enumerate(lens):
            self.table[i, :need[i]] = order[at:at + need[i]]
            at += need[i]
            pos = torch.arange(n, device="cuda")
            self.slots.append(self.table[i].long()[pos // page] * page + pos % page)
            for a in range(0, n, 1 << 15):
                part = self.slots[i][a:a + (1 << 15)]
                k = torch.randn(len(part), hkv, d, device="cuda", generator=gen)
                v = torch.randn(len(part), hkv, d, device="cuda", generator=gen)
                v = v * value_gains(kind, len(part), hkv, d, gen)
                lib.tl_kv4_append(self.cache, k.half(), v.half(), part.contiguous())
        self.start = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
        self.start[1:] = torch.tensor(adds, device="cuda").cumsum(0)
        self.q = (torch.randn(sum(adds), hq, d, device="cuda", generator=gen) * spread).half()
        self.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def tokens(self, i):
        """Keys and values (64 bits, [heads, n, d]) of a request's tokens and the keys' size |b| + 15 s."""
        c, n = self.cache, self.lens[i]
        d, p, g, h = c.head_dim, c.page_size, c.group, c.heads
        blk = c.blocks[self.table[i, :-(-n // p)].long()]
        half, par, got = p * d // 2, 4 * p * d // g, []
        for part in (0, 1):
            code = blk[:, :, part * half:(part + 1) * half].reshape(-1, h, p, d // 2)
            code = torch.stack((code & 15, code >> 4), -1).reshape(-1, h, p, d // g, g).double()
            at = 2 * half + part * par
            sb = blk[:, :, at:at + par].contiguous().view(torch.float16).reshape(-1, h, p, d // g, 2).double()
            s, b = sb[..., :1], sb[..., 1:]
            for x in (code * s + b, (b.abs() + 15 * s).expand_as(code)):
                got.append(x.permute(1, 0, 2, 3, 4).reshape(h, -1, d)[:, :n])
        return got[0], got[2], got[1]

    def run(self, max_q=None, window=0, seq=None, out=None, **kw):
        lib, scale = self.lib, self.cache.head_dim ** -0.5
        max_q = max(self.adds) if max_q is None else max_q
        out = torch.full_like(self.q, 7.0) if out is None else out
        lib.tl_kv4_attention(self.cache, self.q, out, self.start, self.seq if seq is None else seq, self.table, max_q,
                             scale, window, workspace=self.cache.attention_workspace(self.hq, max_q), **kw)
        torch.cuda.synchronize()
        lib.tl_check_status()
        return out

    def check(self, out, window=0, seq=None, max_q=None, norm=True):
        """out against the definition: query t of request i lies at position seq[i] - adds[i] + t and sees those of
        the request's tokens at its position or before it."""
        c, at = self.cache, 0
        d, hkv, share = c.head_dim, c.heads, self.hq // c.heads
        scale = d ** -0.5
        seq = (self.seq if seq is None else seq).tolist()
        for i, (n, a) in enumerate(zip(self.lens, self.adds)):
            m = a if max_q is None else min(a, max_q)
            if m > 0 and n > 0:
                k, v, size = self.tokens(i)
                q = self.q[at:at + m].double().reshape(m, hkv, share, d).permute(1, 2, 0, 3)
                s = scale * (q @ k[:, None].transpose(-1, -2))
                mag = scale * (q.abs() @ size[:, None].transpose(-1, -2))
                pos = torch.arange(seq[i] - a, seq[i] - a + m, device="cuda")[:, None]
                key = torch.arange(n, device="cuda")
                hide = (key > pos) | ((key <= pos - window) if window else torch.zeros_like(key, dtype=torch.bool))
                s.masked_fill_(hide, float("-inf"))
                ds = 2.0 ** -17 * mag.masked_fill_(hide, 0).amax(-1, keepdim=True)
                w = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e300))
                want = w @ v[:, None] / w.sum(-1, keepdim=True).clamp_min(1e-300)
                vmax = v.abs().unflatten(-1, (-1, c.group)).amax((1, 3), keepdim=True).expand(hkv, 1, d // c.group, c.group)
                vmax = vmax.reshape(hkv, 1, 1, d)
                bound = U * want.abs() + 2.0 ** -25 + 2 * U * vmax + 2 * ds * vmax
                got = out[at:at + m].double().reshape(m, hkv, share, d).permute(1, 2, 0, 3)
                assert torch.isfinite(got).all(), i
                off = (got - want).abs() - bound
                assert (off <= 0).all(), (i, n, a, off.max().item())
                if norm:  # group by group
                    diff, ref = (x.unflatten(-1, (-1, c.group)).square().sum((0, 1, 2, 4)).sqrt()
                                 for x in (got - want, want))
                    floor = 2.0 ** -25 * (want.numel() * c.group / d) ** 0.5
                    assert (diff <= 3 * U * ref + floor).all(), (i, (diff / ref).tolist())
            elif m > 0:
                assert not out[at:at + m].any()
            if m < a:
                assert (out[at + m:at + a] == 7).all()
            at += a


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("kind", ["", "zero rows", "wide rows", "zero half"])
@pytest.mark.parametrize("n,adds", [(300, 1), (300, 40), (8000, 1), (8000, 40), (131072, 1)])
@pytest.mark.parametrize("spread", [1.0, 3.0])
def test_value_scales_that_differ(lib, d, group, kind, n, adds, spread):
    """A token's share of the softmax does not depend on the scale of its value: zero and constant rows (scale
    2^-24) beside ordinary ones, scales over a factor of 2^22, a half of the channels at zero."""
    if kind == "zero half" and d == 64:
        kind = "zero rows"
    b = Batch(lib, [n, n // 2 + 3], [adds, adds], 4, 2, d, group, 16, spread, kind, seed=n + adds)
    b.check(b.run())


@pytest.mark.parametrize("n,adds", [(300, 1), (300, 40), (8000, 1), (8000, 40), (131072, 1)])
@pytest.mark.parametrize("spread", [1.0, 3.0])
@pytest.mark.parametrize("hq,hkv", [(4, 2), (12, 1)])
def test_groups_of_different_scales(lib, n, adds, spread, hq, hkv):
    """Two groups of a row whose scales are 2^21 apart: each is as exact as by itself."""
    b = Batch(lib, [n, n // 2 + 3], [adds, adds], hq, hkv, 128, 64, 16, spread, "wide halves", seed=n + adds)
    b.check(b.run())


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("window", [0, 1, 40, 300])
@pytest.mark.parametrize("adds,max_q", [([5, 2, 9], 3), ([5, 2, 9], 1), ([170, 40, 300], 100), ([170, 3, 300], 20)])
def test_max_q_below_a_requests_queries(lib, d, group, window, adds, max_q):
    """The queries that are left out are the last ones; the others keep their positions."""
    b = Batch(lib, [400, 90, 310], adds, 4, 2, d, group, 16, 1.0, seed=window + max_q)
    b.check(b.run(max_q, window), window, max_q=max_q, norm=False)


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("window", [0, 1, 30, 200, 320, 2000])
@pytest.mark.parametrize("adds", [[3, 1, 4], [130, 1, 290]])
def test_lengths_beyond_the_table(lib, d, group, window, adds):
    """Tokens behind the table's row are not in the cache (a step whose pages did not suffice counts them);
    positions are those of the full length."""
    b = Batch(lib, [320, 50, 320], adds, 4, 2, d, group, 16, 1.0, seed=window + adds[0])
    for more in (1, 17, 250):
        seq = b.seq + torch.tensor([more, 0, more + 3], dtype=torch.int32, device="cuda")
        b.check(b.run(window=window, seq=seq), window, seq, norm=False)


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["first", "last", "one each", "all", "with its opposite"])
def test_values_that_are_not_finite_show(lib, d, group, bad, where):
    """A group with one such value reads back as NaN; the groups beside it as they were."""
    gen = torch.Generator("cuda").manual_seed(5)
    t, h = 37, 3
    x = torch.randn(t, h, d, device="cuda", generator=gen).half()
    cache = lib.KV4Cache(3, h, d, 16, group)
    slots = torch.randperm(48, device="cuda", generator=gen)[:t].contiguous()

    def through(k):
        ko, vo = torch.empty_like(k), torch.empty_like(k)
        lib.tl_kv4_append(cache, k, x, slots)
        lib.tl_kv4_read(cache, slots, ko, vo)
        return ko, vo

    good, v = through(x)
    y = x.clone()
    rows = torch.arange(0, t, 2, device="cuda")
    at = {"first": [0], "last": [d - 1], "one each": list(range(5, d, group)), "all": list(range(group)),
          "with its opposite": [3, group - 2]}[where]
    for i, c in enumerate(at):
        y[rows, 1, c] = -bad if where == "with its opposite" and i else bad
    got, v2 = through(y)
    hit = torch.zeros(t, h, d // group, dtype=torch.bool, device="cuda")
    hit[rows[:, None], 1, torch.tensor(sorted({c // group for c in at}), device="cuda")] = True
    hit = hit.repeat_interleave(group, -1)
    assert got[hit].isnan().all()
    assert torch.equal(got[~hit], good[~hit]) and torch.equal(v, v2)
    at = 16 * d + (slots % 16) * (4 * d // group)  # the keys' scales and minima
    at = (at[:, None, None] + torch.arange(4 * d // group, device="cuda")).expand(t, h, -1)
    par = cache.blocks[slots // 16].gather(2, at)
    par = par.contiguous().view(torch.float16).reshape(t, h, -1, 2)
    assert torch.equal(par.isnan(), hit.unflatten(-1, (-1, group))[..., :2])


def with_bad_token(lib, b, i, at, what, part):
    """Token `at` of request i gets a NaN for scale, minimum or both, or a row with an infinity is written there."""
    c = b.cache
    slot = int(b.slots[i][at])
    d, p, g = c.head_dim, c.page_size, c.group
    if what == "written":
        rows = [torch.ones(1, c.heads, d, dtype=torch.float16, device="cuda") for _ in "kv"]
        rows[part][..., 1::64] = float("-inf")
        lib.tl_kv4_append(c, *rows, b.slots[i][at:at + 1])
        return
    blk = c.blocks[slot // p]
    width = 4 * d // g
    off = p * d + part * p * width + (slot % p) * width
    par = blk[:, off:off + width].contiguous().view(torch.float16).reshape(c.heads, -1, 2)
    if what != "minimum":
        par[..., 0] = float("nan")
    if what != "scale":
        par[..., 1] = float("nan")
    blk[:, off:off + width] = par.reshape(c.heads, -1).view(torch.uint8)


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("what", ["scale", "minimum", "both", "written"])
@pytest.mark.parametrize("part", [0, 1])
@pytest.mark.parametrize("adds,window", [(4, 0), (4, 20), (200, 0), (200, 70)])
def test_tokens_that_are_not_finite(lib, d, group, what, part, adds, window):
    """Rows that do not see such a token are what they were; rows that see it show it."""
    n = 330
    b = Batch(lib, [n, 100], [adds, 1], 4, 2, d, group, 16, 1.0, seed=adds + window)
    good = b.run(window=window)
    at = n - adds + (1 if adds < 10 else adds // 2)
    with_bad_token(lib, b, 0, at, what, part)
    got = b.run(window=window)
    pos = torch.arange(n - adds, n, device="cuda")
    sees = (pos >= at) & ((pos < at + window) if window else True)
    keep = torch.cat((~sees, torch.ones(1, dtype=torch.bool, device="cuda")))
    assert torch.equal(got[keep], good[keep])
    assert not torch.isfinite(got[:adds][sees].float()).any()


@pytest.mark.parametrize("d,group", [(128, 128), (64, 64)])
@pytest.mark.parametrize("adds", [[200, 260, 130], [40, 299, 33]])
@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, 60])
def test_pages_outside_the_cache_under_prompts(lib, d, group, adds, window, bad):
    """Such a page holds no tokens and nothing is read through it, in the tensor-core kernel too."""
    from test_serve_gpu import Case, check

    hq, hkv = 8, 2
    assert group == d and min(adds) * hq // hkv > 64  # every request has more rows than the few-rows kernel takes
    c = Case(lib, [300, 299, 140], adds, hq, hkv, d, group, 16, seed=7)
    assert c.cache.num_pages <= 60
    drop = [(0, 0), (0, 7), (0, 18), (1, 3)] + [(2, j) for j in range(9)]
    for i, j in drop:
        c.table[i, j] = bad
    ref = c.reference(0.1, window, drop=set(drop))
    check(c.run(lib, 0.1, window), *ref)
    assert not ref[0][c.start_host[2]:].any()  # the third request has no page left


@pytest.mark.parametrize("head", [-1, -2, -2 ** 31, 0, 2, 9, 10, 2 ** 31 - 1])
def test_free_list_heads(lib, head):
    """Whatever the head, the pages that a step hands out are those its counts say, and the next step's are others."""
    i32 = dict(dtype=torch.int32, device="cuda")
    free = torch.arange(100, 110, **i32)
    cached, added = torch.zeros(3, **i32), torch.tensor([17, 1, 30], **i32)  # 2, 1 and 2 pages
    first = torch.tensor([head], **i32)
    given = []
    for _ in range(2):
        table = torch.full((3, 2), -1, **i32)
        start, lens, counts = torch.empty(4, **i32), torch.empty(3, **i32), torch.empty(4, **i32)
        req, pos = torch.empty(48, **i32), torch.empty(48, **i32)
        slots = torch.empty(48, dtype=torch.int64, device="cuda")
        lib.tl_kv_plan(cached, added, table, free, start, lens, req, pos, slots, counts, page_size=16, num_pages=200,
                       free_head=first)
        pages = [p for p in table.flatten().tolist() if p >= 0]
        at = max(first.item(), 0)
        taken = min(5, max(0, 10 - at))
        assert pages == list(range(100 + at, 100 + at + taken))
        assert counts.tolist() == [48, taken, at + taken, 5 - taken]
        given += pages
        first = counts[2:3].clone()
    assert len(set(given)) == len(given)
