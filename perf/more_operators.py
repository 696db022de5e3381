"""Operators between a projection and the paged 4-bit cache, over it, and behind the last projection.

Four operators of a serving step beside those of perf/operators.py:

* rotate   per-head norms of queries and keys and their rotation by position, one pass
* append   the same on the way into the cache: keys normed, rotated and quantized with the
           values; the queries of the same tokens beside them
* prefix   attention of requests that share a long prefix of the cache
* sample   tokens from logits: temperature, top-k, top-p, min-p, one given number a row

Every function here works on plain values; the framework is imported only where ``own``
is true.

Norms and rotations are fixed to the bit, as the cache's codes are: FP32 with each
operation rounded, the squares of a head summed as a tree (``_fold``).  The cache's layout
is that of perf/operators.py.
"""
import math

import torch

own = False

F16_TINY = 2.0 ** -24   # the smallest FP16 scale
LEAST = 2.0 ** -40      # a token less likely than this, against the likeliest, is not drawn
EPS = 1e-6              # of the norms


def _cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a decode step of 16 requests: 32 query and 8 key heads, normed
        dict(name="rotate_decode", op="rotate", tokens=16, hq=32, hk=8, d=128, rot=128, sections="64", pairs="halves",
             norm=True, top=8192),
        # a long prompt, taken from the fused projection's rows
        dict(name="rotate_prompt", op="rotate", tokens=8192, hq=32, hk=8, d=128, rot=128, sections="64", pairs="halves",
             norm=True, top=8192),
        # an image's patches: positions of height and width, neighbouring pairs, no norm
        dict(name="rotate_image", op="rotate", tokens=4099, hq=12, hk=12, d=64, rot=64, sections="16,16",
             pairs="neighbours", norm=False, top=128),
        # a decode step of 64 requests into the cache, queries rotated beside the keys
        dict(name="append_decode", op="append", tokens=64, hq=32, hkv=8, d=128, group=128, page=16, rot=128,
             sections="64", pairs="halves", norm=True, top=32768),
        # a long prompt of text and pictures: three axes, two scales a row
        dict(name="append_prompt", op="append", tokens=16001, hq=32, hkv=8, d=128, group=64, page=32, rot=128,
             sections="16,24,24", pairs="halves", norm=True, top=16384),
        # keys and values alone, half of the channels rotated
        dict(name="append_partial", op="append", tokens=2500, hq=0, hkv=4, d=64, group=64, page=64, rot=32, sections="16",
             pairs="halves", norm=False, top=4096),
        # four requests behind a short common instruction, every head its own keys
        dict(name="prefix_small", op="prefix", hq=16, hkv=16, d=128, group=128, page=16, prefix=777, lens="41,7,1,130",
             adds="1"),
        # a full decode batch behind a long common prefix that ends inside a page
        dict(name="prefix_batch", op="prefix", hq=32, hkv=8, d=128, group=128, page=16, prefix=8190, lens="ragged:64:512",
             adds="1"),
        # new prompts of several requests over a common document, two requests decoding
        dict(name="prefix_chunks", op="prefix", hq=32, hkv=8, d=128, group=128, page=32, prefix=12001,
             lens="700,90,257,33,1500", adds="700,1,257,33,1"),
        # one conversation: temperature and top-p
        dict(name="sample_one", op="sample", rows=1, vocab=32000, half=True, filters="tp", banned=False),
        # a full batch with every filter, greedy rows and rows under a grammar's mask among them
        dict(name="sample_batch", op="sample", rows=64, vocab=131072, half=True, filters="tkpm", banned=True),
        # many FP32 rows of an odd length: temperature and top-p over the whole vocabulary
        dict(name="sample_wide", op="sample", rows=256, vocab=100003, half=False, filters="tp", banned=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotation(rng, d):
    rot = rng.choice([d, d, d, d // 2, 16])
    axes = rng.choice([1, 1, 2, 3])
    cuts = sorted(rng.sample(range(1, rot // 2), axes - 1))
    sections = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])]
    return dict(rot=rot, sections=",".join(map(str, sections)), pairs=rng.choice(["halves", "halves", "neighbours"]),
                norm=rng.random() < 0.6, top=_log_int(rng, 64, 32768))


def draw(rng):
    what = rng.choice(["rotate", "append", "prefix", "prefix", "sample", "sample"])
    if what == "rotate":
        d = rng.choice([64, 128, 128, 256])
        hk = rng.choice([1, 2, 3, 8, 16])
        hq = min(32, hk * rng.choice([1, 2, 4, 7]))
        return dict(op="rotate", tokens=_log_int(rng, 1, 8192 * 5120 // ((hq + hk) * d)) if rng.random() < 0.5 else
                    _log_int(rng, 1, 2048), hq=hq, hk=hk, d=d, **_draw_rotation(rng, d))
    if what == "append":
        d = rng.choice([64, 128])
        hkv = rng.choice([1, 2, 5, 8])
        return dict(op="append", tokens=_log_int(rng, 1, 16001), hq=rng.choice([0, hkv, 4 * hkv]), hkv=hkv, d=d,
                    group=rng.choice([64, d]), page=rng.choice([16, 32, 64, 128]), **_draw_rotation(rng, d))
    if what == "prefix":
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 4, 8, 8])
        hq = hkv * rng.choice([1, 2, 4, 4, 7])
        if hq > 32:
            hq = 28
            hkv = 4
        prefix = _log_int(rng, 1, 12001)
        if rng.random() < 0.6:
            count = _log_int(rng, 1, 96)
            lens = [_log_int(rng, 1, 512) for _ in range(count)]
            adds = [min(n, rng.choice([1, 1, 1, 2, 4])) for n in lens] if rng.random() < 0.4 else [1] * count
        else:
            count = rng.choice([1, 2, 3, 5])
            adds = [_log_int(rng, 1, 900 // count) for _ in range(count)]
            lens = [a + rng.choice([0, _log_int(rng, 1, 500)]) for a in adds]
        return dict(op="prefix", hq=hq, hkv=hkv, d=d, group=rng.choice([d, d, 64]) if sum(adds) < 64 else d,
                    page=rng.choice([16, 16, 32, 64, 128]), prefix=prefix, lens=",".join(map(str, lens)),
                    adds=",".join(map(str, adds)))
    vocab = _log_int(rng, 500, 200000)
    return dict(op="sample", rows=_log_int(rng, 1, min(512, max(1, 25000000 // vocab))), vocab=vocab,
                half=rng.random() < 0.5, filters=rng.choice(["t", "tk", "tp", "tpm", "tkpm", "kp", ""]),
                banned=rng.random() < 0.3)


def _requests(case):
    """Each request's own tokens behind the prefix (the step's among them) and the step's tokens."""
    if case["lens"].startswith("ragged"):
        _, count, top = case["lens"].split(":")
        count, top = int(count), int(top)
        lens = [max(1, top - (i * 7919 * 13) % (top - top // 16)) for i in range(count)]
    else:
        lens = [int(x) for x in case["lens"].split(",")]
    adds = [int(x) for x in case["adds"].split(",")]
    if len(adds) == 1:
        adds = adds * len(lens)
    return lens, [min(a, n) for a, n in zip(adds, lens)]


def work(case):
    op = case["op"]
    if op in ("rotate", "append"):
        axes = len(case["sections"].split(","))
        t, d = case["tokens"], case["d"]
        table = 8 * min(t, case["top"]) * case["rot"] // 2
        if op == "rotate":
            values = t * (case["hq"] + case["hk"]) * d
            return {"bytes": 4 * values + table + 4 * axes * t, "flops": 7 * values}
        queries, cached = t * case["hq"] * d, 2 * t * case["hkv"] * d
        codes = cached // 2 + 4 * cached // case["group"]
        # queries in and out; keys and values in, codes written, read again, values out
        return {"bytes": 4 * queries + 4 * cached + 2 * codes + table + (4 * axes + 8) * t,
                "flops": 7 * queries + 10 * cached}
    if op == "prefix":
        lens, adds = _requests(case)
        d, hq, hkv = case["d"], case["hq"], case["hkv"]
        pairs = sum(a * (case["prefix"] + n - a) + a * (a + 1) // 2 for n, a in zip(lens, adds))
        row = d // 2 + 4 * d // case["group"]
        keys = case["prefix"] + sum(lens)
        return {"bytes": keys * hkv * 2 * row + 4 * sum(adds) * hq * d + 8 * len(lens), "flops": pairs * hq * d * 4}
    values = case["rows"] * case["vocab"]
    return {"bytes": values * (2 if case["half"] else 4) + 32 * case["rows"], "flops": 10 * values}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _block_bytes(case):
    return case["page"] * case["d"] + 8 * case["page"] * case["d"] // case["group"]


def _codes_and_parameters(x, group):
    """4-bit codes, scales and minima of rows x [..., D] (32-bit floats): per group of
    channels minimum and scale are FP16, the scale no smaller than the smallest FP16
    number, and each value takes the nearest of the sixteen levels."""
    shape = x.shape
    x = x.reshape(shape[:-1] + (shape[-1] // group, group))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((high - low) / 15.0).half().float().clamp_min(F16_TINY)
    low = low.half().float()
    code = torch.round((x - low) / scale).clamp(0, 15)
    return code, scale, low


def _fill_cache(blocks, pages, case, gen):
    """Writes quantized keys and values into the given pages."""
    p, d, hkv, g = case["page"], case["d"], case["hkv"], case["group"]
    half = p * d // 2
    # keys have a few channels much wider than the others, values are even
    wide = torch.ones(hkv, 1, d, device="cuda")
    wide[:, :, ::29] = 4.0
    for part, gain in ((0, wide), (1, torch.ones_like(wide))):
        x = torch.randn(len(pages), hkv, p, d, device="cuda", generator=gen) * gain
        code, scale, low = _codes_and_parameters(x.half().float(), g)
        code = code.reshape(len(pages), hkv, p, d // 2, 2).to(torch.uint8)
        code = (code[..., 0] | (code[..., 1] << 4)).reshape(len(pages), hkv, half)
        par = torch.stack((scale.squeeze(-1), low.squeeze(-1)), -1).half().contiguous().view(torch.uint8)
        par = par.reshape(len(pages), hkv, -1)
        blocks[pages, :, part * half:(part + 1) * half] = code
        blocks[pages, :, 2 * half + part * par.shape[-1]:2 * half + (part + 1) * par.shape[-1]] = par


def _rope_inputs(case, st, gen):
    """Positions on each axis and the table of cosines and sines, in 64 bits and rounded once."""
    t, rot, top = case["tokens"], case["rot"], case["top"]
    sections = [int(s) for s in case["sections"].split(",")]
    st["sections"] = sections
    axis = torch.repeat_interleave(torch.arange(len(sections), device="cuda"),
                                   torch.tensor(sections, device="cuda"), output_size=rot // 2)
    st["axis"] = axis
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * freq
    st["table"] = torch.stack((angle.cos(), angle.sin()), -1).float()
    if t <= 256:  # a decode step: every request at a place of its own
        st["positions"] = torch.randint(0, top, (len(sections), t), dtype=torch.int32, device="cuda", generator=gen)
    else:  # runs of neighbouring tokens
        first = torch.randint(0, max(1, top - 16), (len(sections), _cdiv(t, 16), 1), device="cuda", generator=gen)
        step = torch.arange(16, device="cuda") * torch.randint(0, 2, first.shape, device="cuda", generator=gen)
        st["positions"] = (first + step).reshape(len(sections), -1)[:, :t].clamp_max(top - 1).int().contiguous()
    d = case["d"]
    for name in ("q_weight", "k_weight"):
        st[name] = (1 + 0.2 * torch.randn(d, device="cuda", generator=gen)).half() if case["norm"] else None
    if own:
        import weight_only_int4_quant_gb300 as tlq

        st["rope"] = tlq.Rope(st["table"], interleaved=case["pairs"] == "neighbours", sections=sections)


def prepare(case, seed):
    gen = _gen(seed)
    dev = "cuda"
    st = dict(case=case)
    op = case["op"]
    if op in ("rotate", "append"):
        t, d = case["tokens"], case["d"]
        hk = case["hk"] if op == "rotate" else case["hkv"]
        _rope_inputs(case, st, gen)
        # rows of the fused projection: queries, keys, values
        rows = torch.randn(t, case["hq"] + 2 * hk, d, device=dev, generator=gen)
        rows[:, case["hq"]:case["hq"] + hk, ::29] *= 4.0
        rows = rows.half()
        st["q"], st["k"], st["v"] = rows.split((case["hq"], hk, hk), 1)
        if op == "append":
            pages = _cdiv(t, case["page"]) + 5
            st["blocks"] = torch.randint(0, 256, (pages, hk, _block_bytes(case)), dtype=torch.uint8, device=dev,
                                         generator=gen)
            st["slots"] = torch.randperm(pages * case["page"], device=dev, generator=gen)[:t].contiguous()
        if own:
            st["q_out"] = torch.empty(t, case["hq"], d, dtype=torch.float16, device=dev)
            st["k_out"] = torch.empty(t, hk, d, dtype=torch.float16, device=dev)
            if op == "append":
                st["v_out"] = torch.empty_like(st["k_out"])
                st["cache"] = _kv_object(case, st["blocks"])
    elif op == "prefix":
        lens, adds = _requests(case)
        p, b = case["page"], len(lens)
        shared = _cdiv(case["prefix"], p)
        need = [_cdiv(n, p) for n in lens]
        pages = shared + sum(need) + 7
        # pages come from anywhere in the pool; slots behind an end hold what was there
        blocks = torch.randint(0, 256, (pages, case["hkv"], _block_bytes(case)), dtype=torch.uint8, device=dev,
                               generator=gen)
        order = torch.randperm(pages, device=dev, generator=gen)[:shared + sum(need)]
        _fill_cache(blocks, order, case, gen)
        held = torch.tensor(need, device=dev)
        index = torch.arange(max(need) + 2, device=dev)
        at = shared + torch.cumsum(held, 0) - held
        table = torch.where(index < held[:, None], order[(at[:, None] + index).clamp_max(len(order) - 1)], -1)
        st.update(blocks=blocks, table=table.int().contiguous(), prefix_table=order[:shared].int().contiguous(),
                  prefix_len=torch.tensor([case["prefix"]], dtype=torch.int32, device=dev))
        start = [0]
        for a in adds:
            start.append(start[-1] + a)
        st.update(lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                  start=torch.tensor(start, dtype=torch.int32, device=dev), max_q=max(adds), max_len=max(lens),
                  q=torch.randn(start[-1], case["hq"], case["d"], device=dev, generator=gen).half(),
                  scale=case["d"] ** -0.5)
        if own:
            st["out"] = torch.empty_like(st["q"])
            st["cache"] = _kv_object(case, blocks)
            st["workspace"] = st["cache"].prefix_workspace(case["hq"], start[-1], max(adds))
    else:
        r, v, f = case["rows"], case["vocab"], case["filters"]
        # a language model's logits: a wide body and some tokens far above it
        x = 2.2 * torch.randn(r, v, device=dev, generator=gen)
        high = torch.randint(0, v, (r, 48), device=dev, generator=gen)
        x.scatter_add_(1, high, 3.0 + 7.0 * torch.rand(r, 48, device=dev, generator=gen))
        if case["banned"]:  # every third row: a grammar leaves some hundred tokens; every 41st: none
            allowed = torch.rand(r, v, device=dev, generator=gen) < 200.0 / v
            row = torch.arange(r, device=dev)[:, None]
            allowed &= row % 41 != 40
            x = torch.where(allowed | (row % 3 != 2) & (row % 41 != 40), x, -math.inf)
        unit = torch.rand(r, 4, device=dev, generator=gen)
        st.update(logits=x.half() if case["half"] else x,
                  uniform=torch.rand(r, device=dev, generator=gen),
                  temperature=torch.where(unit[:, 0] < 0.1, 0.0, 0.5 + 0.8 * unit[:, 0]) if "t" in f else None,
                  top_k=torch.where(unit[:, 1] < 0.2, 0, (unit[:, 1] * 200).int()).int() if "k" in f else None,
                  top_p=torch.where(unit[:, 2] < 0.2, 1.0, 0.6 + 0.39 * unit[:, 2]) if "p" in f else None,
                  min_p=torch.where(unit[:, 3] < 0.4, 0.0, 0.1 * unit[:, 3]) if "m" in f else None)
        if own:
            st["tokens"] = torch.empty(r, dtype=torch.int32, device=dev)
            st["logprobs"] = torch.empty(r, dtype=torch.float32, device=dev)
    return st


def _kv_object(case, blocks):
    import weight_only_int4_quant_gb300 as tlq

    return tlq.KV4Cache(blocks.shape[0], case["hkv"], case["d"], page_size=case["page"], group=case["group"],
                        blocks=blocks)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rotate": _rotate, "append": _append, "prefix": _prefix, "sample": _sample}[op](state)


def _own(s, op):
    import weight_only_int4_quant_gb300 as tlq

    if op == "rotate":
        tlq.tl_qk_norm_rope(s["rope"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"], s["q_weight"],
                            s["k_weight"], EPS)
        return s["q_out"], s["k_out"]
    if op == "append":
        queries = s["case"]["hq"] > 0
        tlq.tl_kv4_append_rope(s["cache"], s["rope"], s["k"], s["v"], s["positions"], s["slots"], s["k_weight"],
                               s["q"] if queries else None, s["q_out"] if queries else None,
                               s["q_weight"] if queries else None, EPS)
        tlq.tl_kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return (s["q_out"], s["k_out"], s["v_out"]) if queries else (s["k_out"], s["v_out"])
    if op == "prefix":
        tlq.tl_kv4_attention_prefix(s["cache"], s["q"], s["out"], s["start"], s["lens"], s["table"], s["prefix_len"],
                                    s["prefix_table"], s["max_q"], s["scale"], workspace=s["workspace"])
        return s["out"]
    tlq.tl_sample(s["logits"], s["uniform"], s["tokens"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                  s["logprobs"])
    return s["tokens"], s["logprobs"]


def _fold(x):
    """Sums over the last axis, a power of two long: halves onto each other."""
    while x.shape[-1] > 1:
        x = x[..., :x.shape[-1] // 2] + x[..., x.shape[-1] // 2:]
    return x.squeeze(-1)


def _norm_rotate(s, x, weight):
    """Rows x [tokens, heads, D] normed and rotated, FP16.  The sum of squares: chunks of
    8 channels by halves, then the chunks by halves (squares of FP16 are exact in FP32)."""
    case = s["case"]
    d, half = case["d"], case["rot"] // 2
    x = x.float()
    if weight is not None:
        total = _fold(_fold((x * x).unflatten(-1, (d // 8, 8))))
        r = 1.0 / torch.sqrt(total * (1.0 / d) + EPS)
        x = (x * r[..., None]) * weight.float()
    at = s["positions"].long()[s["axis"]].t()  # [tokens, pairs]
    turn = s["table"][at, torch.arange(half, device=at.device)][:, None]
    c, n = turn[..., 0], turn[..., 1]
    if case["pairs"] == "halves":
        a, b = x[..., :half], x[..., half:2 * half]
        both = torch.cat((a * c - b * n, b * c + a * n), -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        both = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    return torch.cat((both, x[..., 2 * half:]), -1).half()


def _rotate(s):
    return _norm_rotate(s, s["q"], s["q_weight"]), _norm_rotate(s, s["k"], s["k_weight"])


def _append(s):
    case = s["case"]
    p, d, hkv, g = case["page"], case["d"], case["hkv"], case["group"]
    half = p * d // 2
    page, off = s["slots"] // p, s["slots"] % p
    n = len(page)

    def put(part, x):
        code, scale, low = _codes_and_parameters(x.float(), g)
        pair = code.reshape(n, hkv, d // 2, 2).to(torch.uint8)
        rows = s["blocks"][:, :, part * half:(part + 1) * half].unflatten(2, (p, d // 2))
        rows[page, :, off] = pair[..., 0] | (pair[..., 1] << 4)
        par = torch.cat((scale, low), -1).half().view(torch.uint8).reshape(n, hkv, -1)
        at = 2 * half + part * p * par.shape[-1]
        rows = s["blocks"][:, :, at:at + p * par.shape[-1]].unflatten(2, (p, par.shape[-1]))
        rows[page, :, off] = par
        return (code * scale + low).reshape(n, hkv, d).half()

    k, v = put(0, _norm_rotate(s, s["k"], s["k_weight"])), put(1, s["v"])
    return (_norm_rotate(s, s["q"], s["q_weight"]), k, v) if case["hq"] else (k, v)


def _pages_values(blocks, ids, case, part):
    """Keys (part 0) or values (part 1) of the given pages as floats: [..., hkv, page, D]."""
    p, d, g = case["page"], case["d"], case["group"]
    half, par = p * d // 2, 4 * p * d // g
    got = blocks[ids]
    code = got[..., part * half:(part + 1) * half].unflatten(-1, (p, d // 2))
    code = torch.stack((code & 15, code >> 4), -1).flatten(-2).unflatten(-1, (d // g, g)).float()
    at = 2 * half + part * par
    par = got[..., at:at + par].contiguous().view(torch.float16).unflatten(-1, (p, d // g, 2)).float()
    return (code * par[..., :1] + par[..., 1:]).flatten(-2)


def _prefix(s):
    case = s["case"]
    hq, hkv, d, n, dev = case["hq"], case["hkv"], case["d"], case["prefix"], s["q"].device
    g, t = hq // hkv, s["q"].shape[0]
    start, lens = s["start"].long(), s["lens"].long()
    b, most, width = len(lens), s["max_q"], s["max_len"]
    req = torch.repeat_interleave(torch.arange(b, device=dev), start[1:] - start[:-1], output_size=t)
    at = torch.arange(t, device=dev) - start[req]
    q = (s["q"].float() * s["scale"]).unflatten(1, (hkv, g))

    def tokens(ids, part):  # [pages, hkv, page, D] -> [hkv, tokens, D] behind any leading axes
        x = _pages_values(s["blocks"], ids, case, part)
        return x.transpose(-4, -3).flatten(-3, -2)

    # scores on the prefix [hkv, g * t, n], on the own tokens of each request [b, hkv, g * most, width]
    shared = q.permute(1, 2, 0, 3).reshape(hkv, g * t, d) @ tokens(s["prefix_table"].long(), 0)[:, :n].transpose(1, 2)
    ids = s["table"].long()[:, :_cdiv(width, case["page"])].clamp_min(0)
    padded = torch.zeros(b, most, hkv, g, d, device=dev)
    padded[req, at] = q
    alone = padded.permute(0, 2, 3, 1, 4).reshape(b, hkv, g * most, d) @ tokens(ids, 0)[:, :, :width].transpose(2, 3)
    pos = (lens - (start[1:] - start[:-1]))[:, None] + torch.arange(most, device=dev)
    key = torch.arange(width, device=dev)
    hide = (key > pos[..., None]) | (key >= lens[:, None, None])
    alone = alone.unflatten(2, (g, most)).masked_fill_(hide[:, None, None], -math.inf).flatten(2, 3)
    # padding rows may see nothing; their numbers are not taken
    top = alone.amax(-1, keepdim=True).clamp_min(-1e30)
    alone = torch.exp(alone - top)
    first = shared.amax(-1, keepdim=True)
    shared = torch.exp(shared.sub_(first))
    o1, l1 = shared @ tokens(s["prefix_table"].long(), 1)[:, :n], shared.sum(-1, keepdim=True)
    values = torch.where((key < lens[:, None])[:, None, :, None], tokens(ids, 1)[:, :, :width], 0.0)
    o2, l2 = alone @ values, alone.sum(-1, keepdim=True)

    def own_rows(x):  # to [hkv, g, t, ...]
        return x.unflatten(2, (g, most)).permute(0, 3, 1, 2, 4)[req, at].permute(1, 2, 0, 3)

    o2, l2, top = own_rows(o2), own_rows(l2), own_rows(top)
    o1, l1, first = (x.unflatten(1, (g, t)) for x in (o1, l1, first))
    m = torch.maximum(first, top)
    w1, w2 = torch.exp(first - m), torch.exp(top - m)
    out = (o1 * w1 + o2 * w2) / (l1 * w1 + l2 * w2)
    return out.permute(2, 0, 1, 3).reshape(t, hq, d).half()


def _sample(s):
    """In 64 bits: which token a number falls on depends on the last bits of long sums."""
    x = s["logits"].double()
    r, v = x.shape
    dev = x.device
    index = torch.arange(v, device=dev)
    top = x.amax(-1, keepdim=True)
    fine = torch.isfinite(top)  # a row that is masked throughout has no token
    t = s["temperature"].double()[:, None] if s["temperature"] is not None else torch.ones(r, 1, device=dev).double()
    greedy = t <= 0
    w = torch.exp((x - torch.where(fine, top, 0.0)) / torch.where(greedy, 1.0, t))
    w = torch.where(w < LEAST, 0.0, w)
    down, order = torch.sort(x, dim=-1, descending=True, stable=True)
    ws = w.gather(1, order)
    keep = torch.ones(r, v, dtype=torch.bool, device=dev)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (index < k) | (k <= 0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        upto = torch.cumsum(ws * keep, -1)
        before = torch.cat((torch.zeros(r, 1, device=dev).double(), upto[:, :-1]), -1)
        keep &= (before < p * upto[:, -1:]) | (p >= 1)
    if s["min_p"] is not None:
        keep &= ws >= s["min_p"].double().clamp(0, 1)[:, None]
    keep[:, 0] = True
    w = torch.zeros_like(w).scatter_(1, order, ws * keep)
    upto = torch.cumsum(w, -1)
    total = upto[:, -1:]
    token = (upto <= s["uniform"].double()[:, None] * total).sum(-1, keepdim=True)
    token = torch.minimum(token, torch.where(w > 0, index, 0).amax(-1, keepdim=True))
    log = torch.log(w.gather(1, token) / total)
    token = torch.where(greedy, order[:, :1], token)
    log = torch.where(greedy, 0.0, log)
    return (torch.where(fine, token, -1).squeeze(1).int(), torch.where(fine, log, math.nan).squeeze(1).float())


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rows(s, x, weight):
    case = s["case"]
    x = x.double()
    d, rot = case["d"], case["rot"]
    if weight is not None:
        x = x * weight.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    first, second = (list(range(rot // 2)), list(range(rot // 2, rot))) if case["pairs"] == "halves" else \
        (list(range(0, rot, 2)), list(range(1, rot, 2)))
    out = x.clone()
    pair = 0
    for axis, count in enumerate(s["sections"]):
        for _ in range(count):
            row = s["table"][s["positions"][axis].long(), pair].double()
            z = torch.complex(x[..., first[pair]], x[..., second[pair]]) * torch.complex(row[:, 0], row[:, 1])[:, None]
            out[..., first[pair]], out[..., second[pair]] = z.real, z.imag
            pair += 1
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rows(s, s["q"], s["q_weight"]), _exact_rows(s, s["k"], s["k_weight"])
    if case["op"] == "append":
        res = [_exact_rows(s, s["q"], s["q_weight"])] if case["hq"] else []
        # the cache takes FP16 keys; its scales and minima are FP16 by definition
        for x in (_exact_rows(s, s["k"], s["k_weight"]).half().double(), s["v"].double()):
            t = x.unflatten(-1, (-1, case["group"]))
            top, bot = t.max(-1).values, t.min(-1).values
            step = ((top - bot) / 15).half().double().clamp_min(F16_TINY)[..., None]
            level = ((t - bot[..., None]) / step).round().clamp(0, 15)
            res.append((bot[..., None] + level * step).flatten(-2))
        return tuple(res)
    if case["op"] == "prefix":
        return _exact_prefix(case, s)
    return _exact_sample(case, s)


def _exact_prefix(case, s):
    d, g, page, n = case["d"], case["group"], case["page"], case["prefix"]
    share = case["hq"] // case["hkv"]
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    begin, lens, front = s["start"].tolist(), s["lens"].tolist(), s["prefix_table"].tolist()

    def cached(spots, ids, h, part):
        """Keys or values [tokens, D] in 64 bits from the block's bytes."""
        block = s["blocks"][torch.tensor(ids, device="cuda")[spots // page], h]
        at = part * page * d // 2 + (spots % page) * (d // 2)
        words = torch.gather(block, 1, at[:, None] + torch.arange(d // 2, device="cuda"))
        nib = ((words.contiguous().view(torch.int32)[:, :, None] >> shift) & 15).reshape(-1, d).double()
        width = 4 * d // g
        at = page * d + part * page * width + (spots % page) * width
        par = torch.gather(block, 1, at[:, None] + torch.arange(width, device="cuda")).contiguous()
        par = par.view(torch.float16).double().reshape(-1, d // g, 2).repeat_interleave(g, 1)
        return nib * par[:, :, 0] + par[:, :, 1]

    res = torch.zeros(s["q"].shape, dtype=torch.double, device="cuda")
    for h in range(case["hkv"]):
        spots = torch.arange(n, device="cuda")
        k0, v0 = cached(spots, front, h, 0), cached(spots, front, h, 1)
        for i, m in enumerate(lens):
            ids = s["table"][i].tolist()[:_cdiv(m, page)]
            spots = torch.arange(m, device="cuda")
            k = torch.cat((k0, cached(spots, ids, h, 0)))
            v = torch.cat((v0, cached(spots, ids, h, 1)))
            a = begin[i + 1] - begin[i]
            qq = s["q"][begin[i]:begin[i + 1], h * share:(h + 1) * share].double()
            logit = torch.einsum("mgd,nd->mgn", qq, k) / math.sqrt(d)
            last = n + m - a + torch.arange(a, device="cuda")[:, None, None]
            logit = torch.where(torch.arange(n + m, device="cuda") <= last, logit, -math.inf)
            res[begin[i]:begin[i + 1], h * share:(h + 1) * share] = torch.softmax(logit, -1) @ v
    return res


def _exact_sample(case, s):
    """The tokens' log-probabilities, row by row (tokens are whole numbers)."""
    log = []
    for i in range(case["rows"]):
        x = s["logits"][i].double()
        t = float(s["temperature"][i]) if s["temperature"] is not None else 1.0
        if not torch.isfinite(x.max()) or t <= 0:
            log.append(0.0 if torch.isfinite(x.max()) else math.nan)
            continue
        z = (x - x.max()) / t
        z = torch.where(z < math.log(LEAST), -math.inf, z)
        rank = torch.argsort(torch.argsort(-x, stable=True), stable=True)
        allowed = torch.ones_like(x, dtype=torch.bool)
        if s["top_k"] is not None and int(s["top_k"][i]) > 0:
            allowed = rank < int(s["top_k"][i])
        if s["top_p"] is not None and float(s["top_p"][i]) < 1:
            p = torch.softmax(torch.where(allowed, z, -math.inf), -1)
            by_rank = torch.zeros_like(p).index_copy_(0, rank, p)
            above = torch.cumsum(by_rank, 0)[rank] - p  # of the likelier tokens
            allowed &= (above < float(s["top_p"][i])) | (rank == 0)
        if s["min_p"] is not None and float(s["min_p"][i]) > 0:
            allowed &= (z >= math.log(min(1.0, float(s["min_p"][i])))) | (rank == 0)
        p = torch.softmax(torch.where(allowed, z, -math.inf), -1)
        hit = torch.nonzero(torch.cumsum(p, 0) > float(s["uniform"][i]))
        token = hit[0, 0] if len(hit) else torch.nonzero(p)[-1, 0]
        log.append(float(torch.log(p[token])))
    return None, torch.tensor(log, dtype=torch.double)
