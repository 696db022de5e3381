"""The attention over long contexts and large batches, and the serving example.

References are computed in 64 bits on the GPU by torch.  The bound per element
is that of the short cases: U |o| for the output, 3 U V for weights and values
rounded to FP16 and 2 dS V for keys (U = 2^-11, V the largest value a row's
head sees, dS = scale * U * max sum |q||k|).
"""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -11


def rows(gen, t, h, d, mean=0.0):
    x = torch.randn(t, h, d, device="cuda", generator=gen)
    x *= 10 ** (torch.rand(t, h, 1, device="cuda", generator=gen) - 0.5)
    return (x + mean).half()


def batch(lib, lens, adds, hq, hkv, d, group, page, seed, mean=0.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    cache = lib.KV4Cache(sum(need) + 2, hkv, d, page, group)
    cache.blocks.fill_(0xFF)  # NaN scales and minima wherever no token is
    order = torch.randperm(sum(need) + 2, device="cuda", generator=gen).int()
    table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32, device="cuda")
    at, slots = 0, []
    for i, n in enumerate(lens):
        table[i, :need[i]] = order[at:at + need[i]]
        at += need[i]
        pos = torch.arange(n, device="cuda")
        slots.append(table[i].long()[pos // page] * page + pos % page)
    slots = torch.cat(slots)
    for a in range(0, len(slots), 1 << 16):
        part = slots[a:a + (1 << 16)]
        k, v = rows(gen, len(part), hkv, d), rows(gen, len(part), hkv, d, mean)
        lib.tl_kv4_append(cache, k, v, part)
    start = torch.zeros(len(lens) + 1, dtype=torch.int32, device="cuda")
    start[1:] = torch.tensor(adds, device="cuda").cumsum(0)
    q = torch.randn(sum(adds), hq, d, device="cuda", generator=gen).half()
    return cache, q, start, torch.tensor(lens, dtype=torch.int32, device="cuda"), table


def request(cache, table, n):
    """Keys and values (64 bits, [heads, n, d]) of a request's tokens, from the layout of the blocks."""
    d, p, g, h = cache.head_dim, cache.page_size, cache.group, cache.heads
    blk = cache.blocks[table[:-(-n // p)].long()]
    half, par, got = p * d // 2, 4 * p * d // g, []
    for part in (0, 1):
        code = blk[:, :, part * half:(part + 1) * half].reshape(-1, h, p, d // 2)
        code = torch.stack((code & 15, code >> 4), -1).reshape(-1, h, p, d // g, g).double()
        at = 2 * half + part * par
        sb = blk[:, :, at:at + par].contiguous().view(torch.float16).reshape(-1, h, p, d // g, 2).double()
        val = (code * sb[..., :1] + sb[..., 1:]).permute(1, 0, 2, 3, 4).reshape(h, -1, d)
        got.append(val[:, :n])
    return got


def compare(lib, lens, adds, hq, hkv, d, group, page, window=0, seed=1, mean=0.0):
    cache, q, start, seq, table = batch(lib, lens, adds, hq, hkv, d, group, page, seed, mean)
    scale, at = d ** -0.5, 0
    out = lib.kv4_attention(cache, q, start, seq, table, max(adds), scale, window)
    torch.cuda.synchronize()
    lib.tl_check_status()
    assert torch.isfinite(out).all()
    for i, (n, a) in enumerate(zip(lens, adds)):
        if a == 0:
            continue
        k, v = request(cache, table[i], n)
        qq = q[at:at + a].double().reshape(a, hkv, -1, d).permute(1, 2, 0, 3)  # [hkv, share, a, d]
        s = scale * (qq @ k[:, None].transpose(-1, -2))
        mag = scale * (qq.abs() @ k[:, None].abs().transpose(-1, -2))
        pos, key = torch.arange(n - a, n, device="cuda")[:, None], torch.arange(n, device="cuda")
        hide = (key > pos) | ((key <= pos - window) if window else False)
        s.masked_fill_(hide, float("-inf"))
        ds = U * mag.masked_fill_(hide, 0).amax(-1, keepdim=True)
        want = torch.softmax(s, -1) @ v[:, None]
        want, ds = (z.permute(2, 0, 1, 3).reshape(a, hq, -1) for z in (want, ds))
        vmax = v.abs().amax((1, 2)).repeat_interleave(hq // hkv)[None, :, None]
        off = (out[at:at + a].double() - want).abs() - (U * want.abs() + (3 * U + 2 * ds) * vmax)
        assert (off <= 0).all(), (i, n, a, off.max().item())
        at += a


FORMS = [(128, 128), (128, 64), (64, 64)]


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (5, 1)])
@pytest.mark.parametrize("window", [0, 700])
def test_long_chunks(lib, d, group, hq, hkv, window):
    """Blocks that run through many stages and over the ends of several items."""
    compare(lib, [4700, 33, 2500, 1999], [700, 33, 1, 257], hq, hkv, d, group, 16, window)


@pytest.mark.parametrize("d,group", FORMS)
def test_long_contexts(lib, d, group):
    compare(lib, [40000, 17, 9999], [1, 1, 2], 4, 2, d, group, 64)


@pytest.mark.parametrize("d,group", FORMS)
@pytest.mark.parametrize("adds", [1, 40])
def test_values_far_from_zero(lib, d, group, adds):
    """Values with a common offset: nothing is lost where codes and minima are summed apart."""
    compare(lib, [6000, 3001], [adds, adds], 4, 1, d, group, 32, mean=3.0)


@pytest.mark.parametrize("count", [161, 385, 1100])
@pytest.mark.parametrize("d,group", FORMS)
def test_many_requests(lib, d, group, count):
    compare(lib, [1 + (i * 37) % 150 for i in range(count)], [1] * count, 2, 1, d, group, 16)


@pytest.mark.parametrize("count", [161, 500])
def test_many_requests_with_prompts(lib, count):
    adds = [(0, 1, 1, 3, 50, 1, 0)[i % 7] for i in range(count)]
    compare(lib, [a + (i * 53) % 300 for i, a in enumerate(adds)], adds, 4, 2, 128, 128, 16)


@pytest.mark.parametrize("heads,max_q", [((8, 8), 32), ((8, 8), 33), ((8, 1), 4), ((8, 1), 5), ((33, 1), 1),
                                         ((8, 8), 64), ((8, 8), 65), ((8, 1), 8), ((8, 1), 9), ((65, 1), 1)])
def test_either_side_of_the_row_rule(lib, heads, max_q):
    compare(lib, [900, 1800], [max_q, 1], *heads, 128, 128, 16)


def test_arguments_of_the_wrong_kind(lib):
    cache, q, start, seq, table = batch(lib, [20], [2], 4, 2, 64, 64, 16, 3)
    out = torch.full_like(q, 5.0)
    ws = cache.attention_workspace(4, 2)
    good = [cache, q, out, start, seq, table, 2, 0.1]

    def refused(at, value, **kw):
        args = list(good)
        args[at] = value
        with pytest.raises((ValueError, TypeError, lib.TLQError)):
            lib.tl_kv4_attention(*args, workspace=kw.get("workspace", ws))

    refused(1, q.float())
    refused(1, q.cpu())
    refused(1, q[0])
    refused(1, q.transpose(0, 1))
    refused(2, out[:1])
    refused(3, start[:1])
    refused(3, start.long())
    refused(4, seq.float())
    refused(5, table.long())
    refused(5, table[0])
    refused(6, -1)
    refused(7, float("nan"))
    refused(7, 0.1, workspace=ws[:16])
    refused(7, 0.1, workspace=None)
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    slots = torch.arange(3, device="cuda")
    for bad in ((k.float(), k, slots), (k, k[:2], slots), (k, k, slots.int()), (k[..., :32], k, slots)):
        with pytest.raises((ValueError, TypeError)):
            lib.tl_kv4_append(cache, *bad)
    with pytest.raises(ValueError):
        lib.KV4Cache(3, 2, 64, 16, 64, blocks=cache.blocks[:, :1])
    for page, d, g in ((24, 64, 64), (16, 96, 64), (16, 64, 128)):
        with pytest.raises(lib.TLQError):
            lib.KV4Cache(3, 2, d, page, g)
    torch.cuda.synchronize()
    assert (out == 5).all()
    lib.tl_kv4_attention(*good, workspace=ws)  # and the good ones still run
    torch.cuda.synchronize()
    assert not (out == 5).all()


def test_example(lib):
    """The layer of examples/serve_step.py.  Roundings to FP16 on the way, relative to the norms: rows of the
    fused projection and of the adapters' sum, the mix, the output twice, weights of the GEMM at most one each
    and the attention's two: nine half steps in all, each at most U; a key's rounding moves logits of size 1."""
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import serve_step
    finally:
        sys.path.pop(0)
    errors, _ = serve_step.serve(steps=3, width=256, q_heads=4, kv_heads=2, head_dim=64, prompts=(20, 1, 70), rank=8)
    assert len(errors) == 4 and max(errors) <= 9 * U
