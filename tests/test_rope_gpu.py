"""Norms and rotary positions of heads, alone and on the way into the 4-bit cache.

The plain form below follows the header's order of operations in FP32, so equality is to the bit; a second
one in 64 bits bounds how far that order may be off: three roundings of the norm's factor and products, four
of the rotation and one to FP16."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

EPS = 1e-6


def fold(x):
    while x.shape[-1] > 1:
        x = x[..., :x.shape[-1] // 2] + x[..., x.shape[-1] // 2:]
    return x.squeeze(-1)


def plain(x, weight, table, pos, sections, interleaved, kind=torch.float32):
    """x [tokens, heads, D]; pos [axes, tokens].  kind FP32: the defined order; FP64: the formulas."""
    x = x.to(kind)
    d = x.shape[-1]
    if weight is not None:
        total = fold(fold((x * x).unflatten(-1, (d // 8, 8)))) if kind is torch.float32 else (x * x).sum(-1)
        x = (x * (1.0 / torch.sqrt(total * (1.0 / d) + EPS))[..., None]) * weight.to(kind)
    if table is None:
        return x
    half = table.shape[1]
    out = x.clone()
    pair = 0
    for axis, count in enumerate(sections):
        for _ in range(count):
            i, j = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + half)
            beyond = pos[axis] >= table.shape[0]
            row = table[pos[axis].long().clamp(0, table.shape[0] - 1), pair].to(kind)
            row = torch.where(beyond[:, None], float("nan"), row)
            c, s = row[:, :1], row[:, 1:]
            a, b = x[..., i], x[..., j]
            out[..., i], out[..., j] = a * c - b * s, b * c + a * s
            pair += 1
    return out


def make_table(positions, half, seed=0):
    f = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.stack((a.cos(), a.sin()), -1).float()


def inputs(tokens, hq, hk, d, seed, axes=1, top=500):
    g = torch.Generator("cuda").manual_seed(seed)
    rows = torch.randn(tokens, hq + 2 * hk, d, device="cuda", generator=g)
    rows[:, :, ::17] *= 6
    rows = rows.half()
    q, k, v = rows.split((hq, hk, hk), 1)
    pos = torch.randint(0, top, (axes, tokens), dtype=torch.int32, device="cuda", generator=g)
    w = [(1 + 0.3 * torch.randn(d, device="cuda", generator=g)).half() for _ in "qk"]
    return q, k, v, pos, w


def check(got, want32, want64):
    assert torch.equal(got, want32.half())
    # relative to the pair's size: 10 FP32 roundings and one to FP16 of the larger channel
    big = want64.abs().amax(-1, keepdim=True)
    assert ((got.double() - want64).abs() <= 2.0 ** -11 * want64.abs() + 10 * 2.0 ** -24 * big + 2.0 ** -25).all()


FORMS = [  # tokens, hq, hk, d, rot, sections, interleaved, normed
    (1, 1, 1, 64, 64, [32], False, True), (1, 32, 8, 128, 128, [64], False, True), (7, 5, 3, 128, 128, [64], True, True),
    (33, 4, 1, 128, 64, [32], False, True), (5, 3, 2, 128, 48, [24], False, True), (9, 2, 2, 256, 256, [128], False, True),
    (12, 3, 1, 256, 96, [48], False, True), (4, 2, 1, 256, 256, [128], True, False), (50, 12, 12, 64, 64, [16, 16], True, False),
    (31, 7, 1, 64, 16, [8], False, True), (19, 2, 1, 128, 128, [11, 30, 23], False, True), (2, 1, 1, 128, 128, [0, 64, 0], True, True),
    (3000, 32, 8, 128, 128, [16, 24, 24], False, True), (2049, 5, 3, 64, 32, [16], False, False), (1500, 9, 4, 256, 128, [64], True, True),
]


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f[:5])))
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope(lib, form, in_place):
    tokens, hq, hk, d, rot, sections, interleaved, normed = form
    q, k, _, pos, w = inputs(tokens, hq, hk, d, tokens + d, len(sections))
    table = make_table(500, rot // 2)
    qw, kw = w if normed else (None, None)
    rope = lib.Rope(table, interleaved, sections)
    want = [(plain(x, wt, table, pos, sections, interleaved), plain(x, wt, table, pos, sections, interleaved, torch.float64))
            for x, wt in ((q, qw), (k, kw))]
    if in_place:  # columns of the same fused rows
        q_out, k_out = q, k
    else:
        q_out, k_out = (torch.empty(tokens, h, d, dtype=torch.float16, device="cuda") for h in (hq, hk))
    lib.tl_qk_norm_rope(rope, q, k, pos, q_out, k_out, qw, kw, EPS)
    check(q_out, *want[0])
    check(k_out, *want[1])


def test_parts_alone(lib):
    q, k, _, pos, (qw, kw) = inputs(37, 6, 2, 128, 3)
    table = make_table(500, 64)
    rope = lib.Rope(table)
    qo, ko = torch.zeros(37, 6, 128, dtype=torch.float16, device="cuda"), torch.zeros(37, 2, 128, dtype=torch.float16, device="cuda")
    lib.tl_qk_norm_rope(rope, q, None, pos, qo, None, None, None, EPS)
    assert torch.equal(qo, plain(q, None, table, pos, [64], False).half())
    lib.tl_qk_norm_rope(rope, None, k, pos, None, ko, None, kw, EPS)
    assert torch.equal(ko, plain(k, kw, table, pos, [64], False).half())
    lib.tl_qk_norm_rope(None, q, k, None, qo, ko, qw, None, EPS)  # norms without rotation
    assert torch.equal(qo, plain(q, qw, None, None, None, False).half()) and torch.equal(ko, k)
    a, b = lib.qk_norm_rope(rope, q, k, pos, qw, kw, EPS)
    assert torch.equal(a, plain(q, qw, table, pos, [64], False).half())
    assert torch.equal(b, plain(k, kw, table, pos, [64], False).half())


def test_tokens_passed_over_and_beyond_the_table(lib):
    q, k, _, pos, (qw, kw) = inputs(40, 3, 2, 128, 5, axes=2, top=100)
    table = make_table(100, 64)
    pos[0, 3] = pos[1, 8] = pos[0, 39] = -1
    pos[1, 5] = 100
    pos[0, 6] = 2 ** 31 - 1
    rope = lib.Rope(table, sections=[40, 24])
    qo, ko = (torch.full((40, h, 128), 7.0, dtype=torch.float16, device="cuda") for h in (3, 2))
    lib.tl_qk_norm_rope(rope, q, k, pos, qo, ko, qw, kw, EPS)
    gone = (pos < 0).any(0)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        assert (got[gone] == 7.0).all()
        want = plain(x, w, table, pos, [40, 24], False).half()
        assert torch.equal(got[~gone].isnan(), want[~gone].isnan())
        assert torch.equal(got[~gone].nan_to_num(), want[~gone].nan_to_num())
    # the axis beyond gives NaN in its own pairs only
    assert qo[5, 0, 40:64].isnan().all() and qo[5, 0, 104:].isnan().all() and not qo[5, 0, :40].isnan().any()
    assert qo[6, 0, :40].isnan().all() and not qo[6, 0, 40:64].isnan().any()


def test_extremes(lib):
    """Zero rows, the largest and smallest FP16 numbers, infinities and NaN stay in their rows."""
    x = torch.zeros(8, 1, 64, dtype=torch.float16, device="cuda")
    x[1] = 65504
    x[2] = 2.0 ** -24
    x[3, 0, 5] = float("inf")
    x[4, 0, 6] = float("nan")
    x[5] = torch.randn(64, device="cuda").half()
    x[6, 0, 0] = 1.0
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    table = make_table(8, 32)
    pos = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    out = torch.empty_like(x)
    lib.tl_qk_norm_rope(lib.Rope(table), x, None, pos, out, None, w, None, EPS)
    want = plain(x, w, table, pos, [32], False).half()
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(), want.nan_to_num())
    assert (out[0] == 0).all() and out[[1, 2, 5, 6, 7]].isfinite().all()


@pytest.mark.parametrize("positions,half", [(1, 8), (1000, 64), (131072, 32)])
def test_table(lib, positions, half):
    f = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    got = lib.rope_table(positions, f, 1.25)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    want = torch.stack((a.cos(), a.sin()), -1) * 1.25
    # the angle's own rounding (2^-53 of up to 131072) and one of the result
    assert ((got.double() - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -35).all()


APPENDS = [  # tokens, hq, heads, d, group, page, rot, sections, interleaved, normed
    (1, 0, 1, 64, 64, 16, 64, [32], False, True), (16, 32, 8, 128, 128, 16, 128, [64], False, True),
    (67, 6, 3, 128, 64, 32, 128, [20, 22, 22], False, True), (45, 4, 2, 128, 64, 256, 64, [32], True, True),
    (33, 0, 5, 128, 128, 64, 48, [24], False, False), (1201, 14, 2, 64, 64, 128, 32, [16], False, True),
    (4001, 8, 8, 128, 64, 16, 128, [64], True, True),
]


@pytest.mark.parametrize("form", APPENDS, ids=lambda f: "-".join(map(str, f[:7])))
def test_append_rope_is_rope_then_append(lib, form):
    tokens, hq, heads, d, group, page, rot, sections, interleaved, normed = form
    q, k, v, pos, (qw, kw) = inputs(tokens, hq, heads, d, tokens, len(sections))
    if not normed:
        qw = kw = None
    rope = lib.Rope(make_table(500, rot // 2), interleaved, sections)
    pages = -(-tokens // page) + 3
    g = torch.Generator("cuda").manual_seed(1)
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:tokens].contiguous()
    if tokens > 30:
        slots[7] = -1
        slots[9] = pages * page
        pos[-1, 11] = -1
        pos[0, 12] = 500
    caches = []
    for _ in range(2):
        c = lib.KV4Cache(pages, heads, d, page, group)
        c.blocks.fill_(0xA5)
        caches.append(c)
    q_out = torch.full((tokens, hq, d), 3.0, dtype=torch.float16, device="cuda") if hq else None
    lib.tl_kv4_append_rope(caches[0], rope, k, v, pos, slots, kw, q if hq else None, q_out, qw if hq else None, EPS)
    q_two = torch.full((tokens, hq, d), 3.0, dtype=torch.float16, device="cuda") if hq else None
    k_two = torch.empty(tokens, heads, d, dtype=torch.float16, device="cuda")
    lib.tl_qk_norm_rope(rope, q if hq else None, k, pos, q_two, k_two, qw if hq else None, kw, EPS)
    passed = (pos < 0).any(0)
    kept = torch.where(passed, -1, slots)
    lib.tl_kv4_append(caches[1], k_two, v, kept)
    assert torch.equal(caches[0].blocks, caches[1].blocks)
    if hq:
        assert torch.equal(q_out.isnan(), q_two.isnan()) and torch.equal(q_out.nan_to_num(), q_two.nan_to_num())


def test_append_without_rope_is_append(lib):
    _, k, v, _, _ = inputs(100, 1, 4, 128, 9)
    slots = torch.arange(100, device="cuda")
    a, b = (lib.KV4Cache(10, 4, 128, 16, 128) for _ in range(2))
    for c in (a, b):
        c.blocks.zero_()
    lib.tl_kv4_append_rope(a, None, k, v, None, slots)
    lib.tl_kv4_append(b, k, v, slots)
    assert torch.equal(a.blocks, b.blocks)


def test_the_long_way_gives_the_same(lib, monkeypatch):
    q, k, v, pos, (qw, kw) = inputs(20, 4, 2, 128, 2)
    rope = lib.Rope(make_table(500, 64))
    slots = torch.arange(20, device="cuda")
    assert lib._short is not lib._LongWay
    got = []
    for way in (lib._short, lib._LongWay):
        monkeypatch.setattr(lib, "_short", way)
        c = lib.KV4Cache(4, 2, 128)
        c.blocks.zero_()
        qo, ko, q2 = (torch.empty(20, h, 128, dtype=torch.float16, device="cuda") for h in (4, 2, 4))
        lib.tl_qk_norm_rope(rope, q, k, pos, qo, ko, qw, kw)
        lib.tl_kv4_append_rope(c, rope, k, v, pos, slots, kw, q, q2, qw)
        got.append((c.blocks, qo, ko, q2))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_captured_and_on_another_stream(lib):
    q, k, v, pos, (qw, kw) = inputs(64, 8, 2, 128, 4)
    rope = lib.Rope(make_table(500, 64))
    slots = torch.arange(64, device="cuda")
    c = lib.KV4Cache(8, 2, 128)
    c.blocks.zero_()
    qo = torch.empty(64, 8, 128, dtype=torch.float16, device="cuda")
    call = lambda s=None: lib.tl_kv4_append_rope(c, rope, k, v, pos, slots, kw, q, qo, qw, EPS, stream=s)  # noqa: E731
    call()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    pos.copy_((pos + 17) % 500)
    q.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    blocks, out = c.blocks.clone(), qo.clone()
    c.blocks.zero_()
    with torch.cuda.stream(side):
        call(side)
    side.synchronize()
    assert torch.equal(blocks, c.blocks) and torch.equal(out, qo)
