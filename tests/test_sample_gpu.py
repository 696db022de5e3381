"""Sampling against its definition in 64 bits: tokens are equal, log-probabilities to FP32's own rounding."""
import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -40
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def plain(x, u, t=None, k=None, p=None, mp=None):
    """(tokens, log-probabilities, kept) row by row in 64 bits."""
    tokens, logs, sets = [], [], []
    for i in range(x.shape[0]):
        row = x[i].double()
        top = row.max()
        if not torch.isfinite(top):
            tokens.append(-1), logs.append(math.nan), sets.append(None)
            continue
        ti = 1.0 if t is None else float(t[i])
        order = torch.argsort(row, descending=True, stable=True)
        if not ti > 0:
            tokens.append(int(order[0])), logs.append(0.0), sets.append(None)
            continue
        w = torch.exp((row - top) / ti)
        w = torch.where(w < LEAST, 0.0, w)[order]
        n = row.numel()
        if k is not None and 0 < int(k[i]) < n:
            n = int(k[i])
        if p is not None and float(p[i]) < 1:
            upto = torch.cumsum(w[:n], 0)
            n = min(n, 1 + int((upto < float(p[i]) * upto[-1]).sum()))
        keep = torch.zeros_like(w)
        keep[:n] = w[:n]
        if mp is not None and float(mp[i]) > 0:
            keep = torch.where(w >= min(1.0, float(mp[i])), keep, 0.0)
        mass = torch.zeros_like(keep)
        mass[order] = keep
        run = torch.cumsum(mass, 0)
        token = int((run <= float(u[i]) * run[-1]).sum())
        token = min(token, int(torch.nonzero(mass)[-1]))
        tokens.append(token), logs.append(math.log(float(mass[token]) / float(run[-1]))), sets.append(mass > 0)
    return tokens, logs, sets


def compare(lib, x, u, **f):
    rows = x.shape[0]
    tokens = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    logs = torch.full((rows,), 9.0, device="cuda")
    lib.tl_sample(x, u, tokens, f.get("t"), f.get("k"), f.get("p"), f.get("mp"), logs)
    want, wlog, _ = plain(x, u, **f)
    assert tokens.tolist() == want
    for got, w in zip(logs.tolist(), wlog):
        # a difference of two logarithms, each rounded a few times in FP32, and 2^-24 of its size
        assert (math.isnan(got) and math.isnan(w)) or abs(got - w) <= 2.0 ** -20 + 2.0 ** -22 * abs(w), (got, w)


def logits(rows, vocab, seed, half=True, sigma=2.5):
    g = torch.Generator("cuda").manual_seed(seed)
    x = sigma * torch.randn(rows, vocab, device="cuda", generator=g)
    x.scatter_add_(1, torch.randint(0, vocab, (rows, 16), device="cuda", generator=g),
                   8 * torch.rand(rows, 16, device="cuda", generator=g))
    return (x.half() if half else x), torch.rand(rows, device="cuda", generator=g), g


def filters(rows, g, which):
    r = lambda: torch.rand(rows, device="cuda", generator=g)  # noqa: E731
    f = {}
    if "t" in which:
        f["t"] = torch.where(r() < 0.15, 0.0, 0.3 + 1.2 * r())
    if "k" in which:
        f["k"] = (r() * 120).int() - 10
    if "p" in which:
        f["p"] = r() * 1.1
    if "m" in which:
        f["mp"] = 0.2 * r() - 0.05
    return f


@pytest.mark.parametrize("vocab", [1, 2, 31, 500, 4096, 4097, 32000, 50021])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("which", ["", "t", "k", "p", "m", "tkpm"])
def test_sample(lib, vocab, half, which):
    x, u, g = logits(13, vocab, vocab + half, half)
    compare(lib, x, u, **filters(13, g, which))


@pytest.mark.parametrize("vocab,half", [(131072, True), (262147, False), (600000, False), (1 << 20, True), (1 << 20, False)])
def test_long_rows(lib, vocab, half):
    x, u, g = logits(5, vocab, 7, half)
    compare(lib, x, u, **filters(5, g, "tkp"))
    compare(lib, x, u)


def test_many_rows(lib):
    x, u, g = logits(700, 3001, 3, True)
    compare(lib, x, u, **filters(700, g, "tkpm"))


@pytest.mark.parametrize("vocab", [7, 1000, 70000, 1 << 20])
def test_equal_logits(lib, vocab):
    """Every weight the same: sums are whole numbers and borders are hit exactly; ties go by index."""
    rows = 24
    x = torch.full((rows, vocab), -3.25, dtype=torch.float16, device="cuda")
    u = torch.arange(rows, device="cuda") / rows
    compare(lib, x, u)
    compare(lib, x, u, k=torch.arange(rows, dtype=torch.int32, device="cuda"))
    compare(lib, x, u, p=torch.arange(rows, device="cuda") / 16.0)
    compare(lib, x, u, p=torch.full((rows,), 0.5, device="cuda"), k=torch.full((rows,), 4, dtype=torch.int32, device="cuda"))
    compare(lib, x, u, p=torch.full((rows,), 0.75, device="cuda"), k=torch.full((rows,), max(1, vocab * 2 // 3), dtype=torch.int32, device="cuda"))
    compare(lib, x, u, mp=torch.full((rows,), 1.0, device="cuda"))


@pytest.mark.parametrize("half", [True, False])
def test_ties_at_the_cut(lib, half):
    """Few distinct values, hundreds of each: the cut falls inside a run of equal ones."""
    g = torch.Generator("cuda").manual_seed(8)
    x = torch.randint(-6, 3, (40, 9001), device="cuda", generator=g).float() * 0.5
    x = x.half() if half else x
    u = torch.rand(40, device="cuda", generator=g)
    compare(lib, x, u, k=torch.randint(1, 9001, (40,), dtype=torch.int32, device="cuda", generator=g))
    compare(lib, x, u, p=torch.rand(40, device="cuda", generator=g))
    compare(lib, x, u, **filters(40, g, "tkpm"))


def test_masked_rows(lib):
    x, u, g = logits(9, 5000, 1, False)
    inf = float("inf")
    x[0] = -inf
    x[1, 17] = float("nan")
    x[2, 4999] = inf
    x[3] = -inf
    x[3, 4321] = -90.0
    x[4, ::2] = -inf
    x[5] = torch.finfo(torch.float32).min
    x[5, 77] = 1.0
    x[6] = torch.finfo(torch.float32).min  # alone in the row: as likely as each other
    x[7] = -inf
    x[7, [3, 800, 4999]] = torch.tensor([2.0, 2.0, -1.0], device="cuda")
    u[7] = 0.999999
    for f in ({}, filters(9, g, "tkpm"), dict(k=torch.full((9,), 2, dtype=torch.int32, device="cuda"))):
        y = x.clone()
        tokens = torch.empty(9, dtype=torch.int32, device="cuda")
        logs = torch.empty(9, device="cuda")
        lib.tl_sample(y, u, tokens, f.get("t"), f.get("k"), f.get("p"), f.get("mp"), logs)
        assert tokens[:3].tolist() == [-1, -1, -1] and logs[:3].isnan().all()
        assert torch.equal(y.nan_to_num(), x.nan_to_num())  # left as it was
        f = {n: v[3:] for n, v in f.items()}
        compare(lib, x[3:], u[3:].contiguous(), **{n: v.contiguous() for n, v in f.items()})


def test_ends_of_the_parameters(lib):
    inf, nan = float("inf"), float("nan")
    x, u, _ = logits(12, 3000, 5, True)
    u[:6] = torch.tensor([0.0, 1.0 - 2.0 ** -24, 2.0 ** -30, 0.5, 0.0, 0.25], device="cuda")
    v = lambda *a: torch.tensor(a, device="cuda")  # noqa: E731
    compare(lib, x, u, t=v(1e-6, 1e6, 1e-30, 1e30, 0.0, -1.0, 0.01, 100.0, 1.0, 1e-38, 3e38, 0.5))
    compare(lib, x, u, p=v(0.0, -1.0, 1.0, 2.0, 1e-30, 0.99999994, 2.0 ** -24, 0.5, 0.9, 0.1, 1e-10, 1.5))
    compare(lib, x, u, mp=v(0.0, -1.0, 1.0, 2.0, 1e-30, 0.99999994, 0.5, 0.1, 0.9, 1e-6, inf, 0.3))
    k = torch.tensor([0, -5, 1, 2, 2999, 3000, 3001, 2 ** 31 - 1, -2 ** 31, 10, 1, 3], dtype=torch.int32, device="cuda")
    compare(lib, x, u, k=k)
    compare(lib, x, u, k=k, p=v(*[0.7] * 12), mp=v(*[0.02] * 12))
    # out of range or not a number: taken to the nearest, and what leaves every token
    got, same = [torch.empty(12, dtype=torch.int32, device="cuda") for _ in range(2)]
    lib.tl_sample(x, v(-1.0, nan, 1.0, 2.0, inf, -inf, *[0.3] * 6), got, v(*[nan] * 3, *[inf] * 3, *[1.0] * 6), None,
                  v(*[nan] * 12), v(*[nan] * 12))
    lib.tl_sample(x, v(0.0, 0.0, *[1 - 2.0 ** -24] * 3, 0.0, *[0.3] * 6), same, v(*[0.0] * 3, *[3e38] * 3, *[1.0] * 6))
    assert torch.equal(got, same)


def test_frequencies(lib):
    """Numbers spread evenly over [0, 1) give each kept token its share, to one number."""
    n = 4096
    row = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -float("inf"), 1.5, 0.25], device="cuda")
    x = row.expand(n, 8).contiguous()
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tokens, logs = lib.sample(x, u, top_k=torch.full((n,), 5, dtype=torch.int32, device="cuda"))
    share = torch.softmax(torch.where(row >= 0.25, row, -math.inf), 0)  # five values
    count = torch.bincount(tokens.long(), minlength=8)
    assert ((count - n * share).abs() <= 1.0).all()
    assert ((logs.exp() - share[tokens.long()]).abs() < 1e-5).all()


def test_strided_rows_and_offsets(lib):
    """Rows of a wider matrix at odd offsets, without log-probabilities, twice the same."""
    x, u, g = logits(6, 10007, 2, True)
    wide = torch.full((6, 12001), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 3:10010] = x
    f = filters(6, g, "tkp")
    want = plain(x, u, **f)[0]
    for _ in range(2):
        tokens = torch.empty(6, dtype=torch.int32, device="cuda")
        lib.tl_sample(wide[:, 3:10010], u, tokens, f["t"], f["k"], f["p"])
        assert tokens.tolist() == want


def test_captured_on_other_streams_and_the_long_way(lib, monkeypatch):
    x, u, g = logits(8, 20000, 6, False)
    f = filters(8, g, "tkpm")
    tokens, logs = torch.empty(8, dtype=torch.int32, device="cuda"), torch.empty(8, device="cuda")
    call = lambda s=None: lib.tl_sample(x, u, tokens, f["t"], f["k"], f["p"], f["mp"], logs, stream=s)  # noqa: E731
    call()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
    u.copy_(1 - u)
    x.copy_(x.flip(1))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = tokens.tolist(), logs.tolist()
    assert got[0] == plain(x, u, **f)[0]
    for way in (lib._short, lib._LongWay):
        monkeypatch.setattr(lib, "_short", way)
        tokens.fill_(-3)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call(side)
        side.synchronize()
        assert (tokens.tolist(), logs.tolist()) == got


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("vocab", [3000, 150000])
def test_many_kept(lib, vocab, half):
    """top-k beyond a list's length, with and without top-p; cuts in a flat body, in a narrow peak and between two
    far groups of values."""
    g = torch.Generator("cuda").manual_seed(vocab)
    flat = torch.rand(4, vocab, device="cuda", generator=g) * 1e-3
    peak = torch.randn(4, vocab, device="cuda", generator=g) * 0.02
    peak[:, 7] = 30.0
    apart = torch.where(torch.rand(4, vocab, device="cuda", generator=g) < 0.01, 9.0, 0.0) + 0.3 * torch.randn(
        4, vocab, device="cuda", generator=g)
    x = torch.cat((flat, peak, apart))
    x = x.half() if half else x
    u = torch.rand(12, device="cuda", generator=g)
    k = (vocab * torch.rand(12, device="cuda", generator=g)).int().clamp_min(600)
    p = 0.05 + 0.94 * torch.rand(12, device="cuda", generator=g)
    t = 0.5 + torch.rand(12, device="cuda", generator=g)
    compare(lib, x, u, k=k)
    compare(lib, x, u, p=p, t=t)
    compare(lib, x, u, k=k, p=p, t=t)
    compare(lib, x, u, k=k, p=p, mp=torch.full((12,), 0.3, device="cuda"))


@pytest.mark.parametrize("vocab,rows", [(20000, 1), (20000, 40), (20000, 200), (5000, 90), (5000, 400), (65536, 30), (65536, 100)])
def test_the_same_by_any_number_of_blocks(lib, vocab, rows):
    """How many blocks take a row goes by the number of rows: the first rows are what they are alone."""
    x, u, g = logits(rows, vocab, 4, True)
    f = filters(rows, g, "tpm")
    tokens, logs = lib.sample(x, u, f["t"], None, f["p"], f["mp"])
    for i in (0, rows // 2, rows - 1):
        one = slice(i, i + 1)
        t, l = lib.sample(x[one], u[one], f["t"][one], None, f["p"][one], f["mp"][one])
        assert t[0] == tokens[i] and torch.equal(l[0].nan_to_num(), logs[i].nan_to_num())


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("kind", ["p", "tkpm"])
@pytest.mark.parametrize("vocab", [7, 4003, 70001, 200003])
def test_the_same_by_clusters_of_every_size(lib, vocab, kind, half):
    """17 to 152 rows go from clusters of eight blocks down to single blocks, by way of seven, six, five and three."""
    x, u, g = logits(152, vocab, 6, half)
    f = filters(152, g, kind)
    pick = lambda rows: [f[n][:rows] if f.get(n) is not None else None for n in ("t", "k", "p", "mp")]
    want_t, want_l = [torch.cat(parts) for parts in zip(*(
        lib.sample(x[i:i + 1], u[i:i + 1], *[None if f.get(n) is None else f[n][i:i + 1] for n in ("t", "k", "p", "mp")])
        for i in range(152)))]
    for rows in (17, 19, 21, 23, 26, 28, 33, 36, 40, 46, 50, 64, 76, 90, 100, 152):
        t, l = lib.sample(x[:rows], u[:rows], *pick(rows))
        assert torch.equal(t, want_t[:rows])
        assert torch.equal(l.nan_to_num(), want_l[:rows].nan_to_num())


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("vocab,t,k", [(5000, 0.02, 50), (60000, 0.03, 300), (5000, 0.3, 4000), (40000, 0.25, 39000),
                                       (3, 0.01, 2), (700, 0.001, 699)])
def test_fewer_with_weight_than_k(lib, vocab, t, k, half):
    """Cold rows: what is within 2^-40 of the greatest is less than top_k, from one value to more than a list holds."""
    x, u, g = logits(9, vocab, vocab + k, half)
    f = dict(t=torch.full((9,), t, device="cuda"), k=torch.full((9,), k, dtype=torch.int32, device="cuda"))
    weight = ((x.float() - x.float().amax(1, keepdim=True)) / t * math.log2(math.e) > -40).sum(1)
    assert (weight < k).any()
    compare(lib, x, u, **f)
    compare(lib, x, u, **f, p=torch.rand(9, device="cuda", generator=g))
    compare(lib, x, u, **f, p=torch.rand(9, device="cuda", generator=g), mp=0.1 * torch.rand(9, device="cuda", generator=g))


@pytest.mark.parametrize("vocab", [3000, 70000])
def test_kept_sets_of_every_size(lib, vocab):
    """top_p's cut behind 1 to some hundreds of values: by a ranked list, and around an estimate."""
    x, u, g = logits(96, vocab, 17, False)
    t = torch.full((96,), 0.9, device="cuda")
    ordered = torch.softmax(x.double() / 0.9, 1).sort(1, descending=True)[0].cumsum(1)
    behind = (1.09 ** torch.arange(96, device="cuda")).long().clamp(1, vocab - 1)  # 1 .. 3400
    behind = behind.clamp(max=vocab // 2)
    p = ordered.gather(1, behind[:, None])[:, 0].float()
    compare(lib, x, u, t=t, p=p)


FIRST = """
import torch, weight_only_int4_quant_gb300 as lib
lib.load()
g = torch.Generator("cuda").manual_seed(3)
x, u = torch.randn(40, 9000, device="cuda", generator=g), torch.rand(40, device="cuda", generator=g)
p, tokens = torch.full((40,), 0.9, device="cuda"), torch.zeros(40, dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    lib.tl_sample(x, u, tokens, top_p=p)
tokens.fill_(-7)
graph.replay()
assert torch.equal(tokens, lib.sample(x, u, top_p=p)[0])
print("same")
"""


def test_a_first_call_may_be_captured(lib):
    """What is asked of the device once may be asked while a stream is captured."""
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr
