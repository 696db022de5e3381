"""Attention over the 4-bit cache in 64 bits, with a bound of its error that a wrong answer does not meet.

With v = s (c - 8) + (b + 8 s), weights p and their sum L, u = 2^-11 (half a step of FP16), an output o is off by at most
    u |o|                              its own rounding,
    u sum p s |c - 8| / L              the weights' rounding to FP16 (they are entered as p s),
    N 2^-31 max(p s) |c - 8| / L       weights below FP16's normal numbers: 2^-25 each, the largest being 2^6 or more,
    T 2^-24 sum p (s |c - 8| + |b + 8 s|) / L   FP32 sums of T tokens a block, a cut of 2^-24 each,
    2 e sum p |v - o| / L              an error e of the logits, relative of the weights:
        e = scale (D + D / 8) 2^-24 sum |q| (15 s + |b|)   a cut for each product and instruction,
            + 2^-20 (1 + |logit|)                          the exponential and its argument
and sum p |v - o| / L <= sqrt(sum p v^2 / L - o^2).  All are weighted by what a query sees, so they shrink or grow with
the output's own terms and not with the largest value in the cache."""
import torch

U = 2.0 ** -11
RUN = 4096  # tokens that a block's sums run over, at most, and their joining


def parts(blocks, ids, page, d, group, part):
    """(code, scale, minimum) of keys (0) or values (1) of pages, in 64 bits: [heads, tokens, D] each."""
    got = blocks[ids]
    half, par = page * d // 2, 4 * page * d // group
    code = got[..., part * half:(part + 1) * half].unflatten(-1, (page, d // 2))
    code = torch.stack((code & 15, code >> 4), -1).flatten(-2).double()
    at = 2 * half + part * par
    pair = got[..., at:at + par].contiguous().view(torch.float16).unflatten(-1, (page, d // group, 2)).double()
    flat = lambda x: x.transpose(0, 1).flatten(1, 2)  # noqa: E731
    return tuple(flat(x) for x in (code, pair[..., 0].repeat_interleave(group, -1), pair[..., 1].repeat_interleave(group, -1)))


def quantized(x, group):
    """(code, scale, minimum) of x [heads, tokens, D] as the cache holds it."""
    y = x.half().float().unflatten(-1, (-1, group))
    low = y.amin(-1, keepdim=True)
    s = ((y.amax(-1, keepdim=True) - low) / 15).half().float().clamp_min(2.0 ** -24)
    code = ((y - low) / s).round().clamp(0, 15)
    return tuple(z.expand_as(y).flatten(-2).double() for z in (code, s, low))


def attend(q, key, value, see, scale, weights=lambda w: w):
    """(o, bound, p / L) of q [heads, queries, D] in 64 bits over key and value, each (code, scale, minimum)
    [heads, tokens, D]; see: [queries, tokens].  weights: what becomes of p s (to plant a rounding there)."""
    (ck, sk, bk), (cv, sv, bv) = key, value
    k, v = ck * sk + bk, cv * sv + bv
    n, d = k.shape[1], q.shape[-1]
    logit = (q @ k.transpose(1, 2) * scale).masked_fill(~see, float("-inf"))
    w = torch.softmax(logit, -1)
    o = w @ v
    centred = sv * (cv - 8).abs()
    e = scale * (d + d / 8) * 2.0 ** -24 * (q.abs() @ (15 * sk + bk.abs()).transpose(1, 2))
    e = (e + 2.0 ** -20 * (1 + logit.abs())).masked_fill(~see, 0).amax(-1, keepdim=True)
    spread = (w @ v.square() - o.square()).clamp_min(0).sqrt()
    rounded = w @ centred
    small = n * 2.0 ** -31 * 8 * (w * sv.amax(-1)[:, None]).amax(-1, keepdim=True)
    sums = RUN * 2.0 ** -24 * (rounded + w @ (bv + 8 * sv).abs())
    return o, U * o.abs() + U * rounded + small + sums + 2 * e * spread + 2.0 ** -24, w


def close(b, got, prefix=True):
    """Checks an output of a Batch of test_prefix_gpu, its prefix left out if it is not to be seen."""
    n = int(b.prefix_len) if prefix else 0
    share, args = b.hq // b.hkv, (b.page, b.d, b.group)
    starts, lens = b.start.tolist(), b.lens.tolist()
    for i, m in enumerate(lens):
        a, z = starts[i], starts[i + 1]
        if a == z:
            continue
        both = []
        for part in (0, 1):
            front = parts(b.cache.blocks, b.prefix_table.long(), *args, part)
            own = parts(b.cache.blocks, b.table[i][:-(-m // b.page)].long(), *args, part)
            both.append(tuple(torch.cat((f[:, :n], o[:, :m]), 1).repeat_interleave(share, 0) for f, o in zip(front, own)))
        at = torch.arange(n + m, device=got.device) - n
        see = at[None] <= (m - (z - a) + torch.arange(z - a, device=got.device))[:, None]
        want, tol, _ = attend(b.q[a:z].double().transpose(0, 1), *both, see, b.scale)
        off = (got[a:z].double().transpose(0, 1) - want).abs() / tol
        assert (off <= 1).all(), (i, float(off.max()))
