"""The operators of a multi-request serving step, as a user's program meets them.

Five operators stand beside the quantized projections when many requests share
one step:

* plan       block tables, slots and positions of the step's tokens, from request lengths
* append     the step's keys and values quantized into a paged 4-bit cache, read back as
             the values that the cache now stands for
* attention  the step's queries over that cache: single tokens, short drafts, prompt chunks
* lora       low-rank adapters of many requests beside a shared projection

Every function here works on plain values; the framework is imported only where
``own`` is true.

The cache: ``blocks`` is uint8 [pages][kv heads][block bytes]; the block of one page
and head holds, one after another, the key codes [page][D/2], the value codes
[page][D/2], the key parameters [page][D/group][2] and the value parameters (FP16
scale and minimum).  Byte j of a code row holds channel 2j in its low and channel
2j + 1 in its high four bits; a value is scale * code + minimum.
"""
import math

import torch

own = False

F16_TINY = 2.0 ** -24  # the smallest FP16 scale


def _cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request decoding on a short context: 16 heads of 128, the shape of a 2048-wide block
        dict(name="attn_decode_one", op="attention", hq=16, hkv=16, d=128, group=128, page=16, window=0, pool=1.2,
             lens="500", adds="1"),
        # a full decode batch, ragged contexts, four query heads per key head
        dict(name="attn_decode_batch", op="attention", hq=32, hkv=8, d=128, group=128, page=16, window=0, pool=1.1,
             lens="ragged:64:8192", adds="1"),
        # few requests on very long contexts, larger pages, two scales per row
        dict(name="attn_decode_long", op="attention", hq=32, hkv=8, d=128, group=64, page=64, window=0, pool=1.02,
             lens="ragged:4:131072", adds="1"),
        # drafts of three tokens to verify, an odd group of heads, narrow heads, a sliding window
        dict(name="attn_verify_window", op="attention", hq=14, hkv=2, d=64, group=64, page=16, window=1024, pool=1.3,
             lens="ragged:33:4000", adds="3"),
        # a prompt of 2048 tokens in one pass, every head its own keys
        dict(name="attn_prompt", op="attention", hq=16, hkv=16, d=128, group=128, page=16, window=0, pool=1.1,
             lens="2048", adds="2048"),
        # prompt chunks on long cached contexts beside requests that decode
        dict(name="attn_chunks_mixed", op="attention", hq=32, hkv=8, d=128, group=128, page=16, window=0, pool=1.1,
             lens="16384,9001,2047,700,12345,31", adds="2048,1001,1,1,1,31"),
        # a small decode step: each request one token
        dict(name="plan_decode", op="plan", requests=16, page=16, max_added=1, max_cached=4096, pad=0),
        # a large mixed step: prompts beside decoding requests, outputs with room to spare
        dict(name="plan_mixed", op="plan", requests=1000, page=16, max_added=256, max_cached=8192, pad=321),
        # keys and values of a decode step, taken from the fused projection's rows
        dict(name="append_decode", op="append", tokens=16, hkv=16, d=128, group=128, page=16, fused=True),
        # keys and values of a long prompt
        dict(name="append_prompt", op="append", tokens=16001, hkv=16, d=128, group=64, page=32, fused=True),
        # a decode step of 32 requests over 8 adapters beside the fused qkv projection
        dict(name="lora_decode", op="lora", k=2048, n=6144, rank=16, adapters=8, requests=32, max_added=1),
        # prompts of several requests beside the up projection
        dict(name="lora_prompts", op="lora", k=2048, n=8192, rank=32, adapters=6, requests=9, max_added=900),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    what = rng.choice(["decode", "decode", "decode", "verify", "prompt", "prompt", "plan", "append", "append", "lora",
                       "lora"])
    if what in ("decode", "verify", "prompt"):
        d = rng.choice([64, 128, 128])
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        hq = hkv * rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8])
        group = rng.choice([64, d])
        page = rng.choice([16, 16, 32, 64, 128])
        window = rng.choice([0, 0, 0, _log_int(rng, 1, 4096)])
        if what == "prompt":
            hkv, hq = min(hkv, 8), min(hq, 32)
            hq -= hq % hkv
            count = rng.choice([1, 1, 2, 3, 5])
            adds = [_log_int(rng, 1, 2048 // count + 1) if rng.random() < 0.8 else 1 for _ in range(count)]
            adds[0] = _log_int(rng, 60, 2048)
            lens = [a + rng.choice([0, _log_int(rng, 1, 12000)]) for a in adds]
        else:
            count = _log_int(rng, 1, 128)
            most = min(131072, max(16, 4000000 // (count * hkv)))
            lens = [_log_int(rng, 1, most) for _ in range(count)]
            adds = [1] * count if what == "decode" else [min(n, rng.choice([1, 2, 3, 4, 5, 8])) for n in lens]
        return dict(op="attention", hq=hq, hkv=hkv, d=d, group=group, page=page, window=window, pool=1.1,
                    lens=",".join(map(str, lens)), adds=",".join(map(str, adds)))
    if what == "plan":
        return dict(op="plan", requests=_log_int(rng, 1, 2000), page=rng.choice([16, 32, 64, 128]),
                    max_added=rng.choice([1, 1, _log_int(rng, 2, 256)]), max_cached=_log_int(rng, 16, 8192),
                    pad=rng.choice([0, 0, rng.randint(1, 500)]))
    if what == "append":
        d = rng.choice([64, 128])
        return dict(op="append", tokens=_log_int(rng, 1, 16001), hkv=rng.choice([1, 2, 5, 8, 16]), d=d,
                    group=rng.choice([64, d]), page=rng.choice([16, 32, 64, 128]), fused=rng.random() < 0.5)
    return dict(op="lora", k=rng.choice([512, 1024, 2048, 2048, 2056, 8192]),
                n=rng.choice([512, 2048, 2056, 6144, 8192]), rank=rng.choice([8, 16, 16, 24, 32, 64]),
                adapters=_log_int(rng, 1, 32), requests=_log_int(rng, 1, 48),
                max_added=rng.choice([1, 1, _log_int(rng, 2, 100)]))


def _requests(case):
    """Request lengths (cached tokens with the step's own) and the step's tokens of each."""
    if case["lens"].startswith("ragged"):
        _, count, top = case["lens"].split(":")
        count, top = int(count), int(top)
        # spread between an eighth and the whole of the longest, odd ones among them
        lens = [max(1, top - (i * 7919 * 13) % (top - top // 8)) for i in range(count)]
    else:
        lens = [int(x) for x in case["lens"].split(",")]
    adds = [int(x) for x in case["adds"].split(",")]
    if len(adds) == 1:
        adds = adds * len(lens)
    return lens, [min(a, n) for a, n in zip(adds, lens)]


def _visible(length, added, window):
    """Keys that the step's queries of one request see: (all pairs, distinct keys)."""
    pairs = 0
    first = length
    for p in (range(length - added, length) if window else ()):
        pairs += min(p + 1, window)
    if window:
        first = max(0, length - added - window + 1)
        return pairs, length - first
    return added * (length - added) + added * (added + 1) // 2, length


def work(case):
    if case["op"] == "attention":
        lens, adds = _requests(case)
        d, hq, hkv = case["d"], case["hq"], case["hkv"]
        pairs = keys = 0
        for n, a in zip(lens, adds):
            p, s = _visible(n, a, case["window"])
            pairs, keys = pairs + p, keys + s
        row = d // 2 + 4 * d // case["group"]
        pages = sum(_cdiv(n, case["page"]) for n in lens)
        return {"bytes": keys * hkv * 2 * row + 2 * sum(adds) * hq * d * 2 + 4 * pages + 8 * len(lens),
                "flops": pairs * hq * d * 4}
    if case["op"] == "plan":
        b = case["requests"]
        cached, added = _plan_lengths(case, 0)
        tokens = sum(added)
        fresh = sum(_cdiv(c + a, case["page"]) - _cdiv(c, case["page"]) for c, a in zip(cached, added))
        return {"bytes": 8 * b + 4 * b + 8 * fresh + 8 * b + 16 * (tokens + case["pad"]) + 16, "flops": 8 * tokens}
    if case["op"] == "append":
        values = 2 * case["tokens"] * case["hkv"] * case["d"]
        codes = values // 2 + 4 * values // case["group"]
        # in, codes written, codes read, out
        return {"bytes": 2 * values + 2 * codes + 2 * values + 8 * case["tokens"], "flops": 6 * values}
    added, adapter = _lora_requests(case, 0)
    tokens = sum(a for a, _ in zip(added, adapter))
    used = len({x for a, x in zip(added, adapter) if x >= 0 and a})
    active = sum(a for a, x in zip(added, adapter) if x >= 0)
    return {"bytes": 2 * active * case["k"] + 4 * tokens * case["n"] + 2 * used * case["rank"] * (case["k"] + case["n"]),
            "flops": 2 * active * case["rank"] * (case["k"] + case["n"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lcg(seed, count, low, high):
    """Whole numbers low..high from the seed alone (the host's lengths)."""
    x = (seed * 2654435761 + 12345) & 0xFFFFFFFF
    out = []
    for _ in range(count):
        x = (x * 1664525 + 1013904223) & 0xFFFFFFFF
        out.append(low + (x >> 8) % (high - low + 1))
    return out


def _plan_lengths(case, seed):
    """Lengths are the case's (a seed changes tables and pages, not the work)."""
    b = case["requests"]
    cached = _lcg(7 + b, b, 0, case["max_cached"])
    kind = _lcg(11 + b, b, 0, 9)
    size = _lcg(13 + b, b, 0, case["max_added"])
    added = [1 if k < 6 else s for k, s in zip(kind, size)]
    return cached, added


def _lora_requests(case, seed):
    b = case["requests"]
    if case["max_added"] == 1:
        added = [1] * b
    else:
        added = _lcg(17 + b, b, 1, case["max_added"])
    adapter = [x - 1 if x == 0 and b > 3 else x % case["adapters"] for x in _lcg(19 + b, b, 0, case["adapters"])]
    return added, adapter


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
    step = max(1, (1 << 25) // (p * d * hkv))
    # keys have a few channels much wider than the others, values are even
    wide = torch.ones(hkv, 1, d, device="cuda")
    wide[:, :, ::29] = 4.0
    for at in range(0, len(pages), step):
        ids = pages[at:at + step]
        for part, gain in ((0, wide), (1, torch.ones_like(wide))):
            x = torch.randn(len(ids), hkv, p, d, device="cuda", generator=gen) * gain
            code, scale, low = _codes_and_parameters(x.half().float(), g)
            code = code.reshape(len(ids), hkv, p, d // 2, 2).to(torch.uint8)
            code = (code[..., 0] | (code[..., 1] << 4)).reshape(len(ids), hkv, p * d // 2)
            par = torch.stack((scale.squeeze(-1), low.squeeze(-1)), -1).half().contiguous().view(torch.uint8)
            par = par.reshape(len(ids), hkv, -1)
            half = p * d // 2
            blocks[ids, :, part * half:(part + 1) * half] = code
            blocks[ids, :, 2 * half + part * par.shape[-1]:2 * half + (part + 1) * par.shape[-1]] = par


def _kv_object(case, blocks):
    import weight_only_int4_quant_gb300 as tlq

    return tlq.KV4Cache(blocks.shape[0], case["hkv"], case["d"], page_size=case["page"], group=case["group"],
                        blocks=blocks)


def prepare(case, seed):
    gen = _gen(seed)
    dev = "cuda"
    st = dict(case=case)
    if case["op"] == "attention":
        lens, adds = _requests(case)
        need = [_cdiv(n, case["page"]) for n in lens]
        pages = int(sum(need) * case["pool"]) + 3
        # pages come from anywhere in the pool; slots behind a request's end hold what was there
        blocks = torch.randint(0, 256, (pages, case["hkv"], _block_bytes(case)), dtype=torch.uint8, device=dev,
                               generator=gen)
        order = torch.randperm(pages, device=dev, generator=gen)[:sum(need)]
        _fill_cache(blocks, order, case, gen)
        table = torch.full((len(lens), max(need) + 2), -1, dtype=torch.int32, device=dev)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n].int()
            at += n
        # what lies behind a request's last token in its last page is left over from others
        row = 2 * case["d"] // case["group"] * 2
        par = blocks[:, :, case["page"] * case["d"]:].view(pages, case["hkv"], 2, case["page"], row)
        for i, (n, k) in enumerate(zip(lens, need)):
            if n % case["page"]:
                par[table[i, k - 1].long(), :, :, n % case["page"]:] = 255
        start = [0]
        for a in adds:
            start.append(start[-1] + a)
        st.update(blocks=blocks, table=table, host_lens=lens, host_adds=adds,
                  lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                  start=torch.tensor(start, dtype=torch.int32, device=dev),
                  q=torch.randn(start[-1], case["hq"], case["d"], device=dev, generator=gen).half(),
                  scale=case["d"] ** -0.5, max_q=max(adds))
        if own:
            st["out"] = torch.empty_like(st["q"])
            st["cache"] = _kv_object(case, blocks)
            st["workspace"] = st["cache"].attention_workspace(case["hq"], max(adds))
    elif case["op"] == "plan":
        cached, added = _plan_lengths(case, seed)
        b, p = case["requests"], case["page"]
        width = _cdiv(case["max_cached"] + case["max_added"], p) + 1
        held = torch.tensor([_cdiv(c, p) for c in cached], device=dev)
        fresh = sum(_cdiv(c + a, p) - _cdiv(c, p) for c, a in zip(cached, added))
        pages = int(held.sum().item()) + fresh + 64
        order = torch.randperm(pages, device=dev, generator=gen).int()
        index = torch.arange(width, device=dev)
        at = torch.cumsum(held, 0) - held
        mine = index < held[:, None]
        table = torch.where(mine, order[(at[:, None] + index).clamp_max(pages - 1)], -1).int().contiguous()
        free = order[int(held.sum().item()):].contiguous()
        st.update(cached=torch.tensor(cached, dtype=torch.int32, device=dev),
                  added=torch.tensor(added, dtype=torch.int32, device=dev), table=table, free=free, pages=pages,
                  tokens=sum(added), room=sum(added) + case["pad"])
        if own:
            room = st["room"]
            st.update(start=torch.empty(b + 1, dtype=torch.int32, device=dev),
                      lens=torch.empty(b, dtype=torch.int32, device=dev),
                      token_req=torch.empty(room, dtype=torch.int32, device=dev),
                      token_pos=torch.empty(room, dtype=torch.int32, device=dev),
                      slots=torch.empty(room, dtype=torch.int64, device=dev),
                      counts=torch.empty(4, dtype=torch.int32, device=dev))
    elif case["op"] == "append":
        t, hkv, d = case["tokens"], case["hkv"], case["d"]
        pages = _cdiv(t, case["page"]) + 5
        blocks = torch.randint(0, 256, (pages, hkv, _block_bytes(case)), dtype=torch.uint8, device=dev, generator=gen)
        slots = torch.randperm(pages * case["page"], device=dev, generator=gen)[:t].contiguous()
        wide = torch.ones(d, device=dev)
        wide[::29] = 4.0
        if case["fused"]:  # columns of one projection's rows: queries, keys, values
            rows = torch.randn(t, 3, hkv, d, device=dev, generator=gen).half()
            rows[:, 1] *= wide.half()
            k, v = rows[:, 1], rows[:, 2]
        else:
            k = (torch.randn(t, hkv, d, device=dev, generator=gen) * wide).half()
            v = torch.randn(t, hkv, d, device=dev, generator=gen).half()
        st.update(blocks=blocks, slots=slots, k=k, v=v)
        if own:
            st["cache"] = _kv_object(case, blocks)
            st["k_out"], st["v_out"] = (torch.empty(t, hkv, d, dtype=torch.float16, device=dev) for _ in "kv")
    else:
        added, adapter = _lora_requests(case, seed)
        start = [0]
        for a in added:
            start.append(start[-1] + a)
        t, k, n, r = start[-1], case["k"], case["n"], case["rank"]
        st.update(x=torch.randn(t, k, device=dev, generator=gen).half(),
                  y=torch.randn(t, n, device=dev, generator=gen).half(),
                  a=(torch.randn(case["adapters"], r, k, device=dev, generator=gen) * k ** -0.5).half(),
                  b=(torch.randn(case["adapters"], n, r, device=dev, generator=gen) * 0.5 * r ** -0.5).half(),
                  scales=0.5 + torch.rand(case["adapters"], device=dev, generator=gen),
                  start=torch.tensor(start, dtype=torch.int32, device=dev),
                  adapter=torch.tensor(adapter, dtype=torch.int32, device=dev),
                  host_start=start, host_adapter=adapter, max_q=max(added))
        if own:
            st["out"] = torch.empty_like(st["y"])
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"attention": _attention, "plan": _plan, "append": _append, "lora": _lora}[op](state)


def _own(state, op):
    import weight_only_int4_quant_gb300 as tlq

    s = state
    if op == "attention":
        tlq.tl_kv4_attention(s["cache"], s["q"], s["out"], s["start"], s["lens"], s["table"], s["max_q"], s["scale"],
                             window=s["case"]["window"], workspace=s["workspace"])
        return s["out"]
    if op == "plan":
        tlq.tl_kv_plan(s["cached"], s["added"], s["table"], s["free"], s["start"], s["lens"], s["token_req"],
                       s["token_pos"], s["slots"], s["counts"], page_size=s["case"]["page"], num_pages=s["pages"])
        return {k: s[k] for k in ("table", "start", "lens", "token_req", "token_pos", "slots", "counts")}
    if op == "append":
        tlq.tl_kv4_append(s["cache"], s["k"], s["v"], s["slots"])
        tlq.tl_kv4_read(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    tlq.tl_lora_add(s["x"], s["a"], s["b"], s["scales"], s["start"], s["adapter"], s["max_q"], s["y"], s["out"])
    return s["out"]


def _pages_values(blocks, ids, case, part):
    """Keys (part 0) or values (part 1) of the given pages as floats: [hkv, tokens, D]."""
    p, d, hkv, g = case["page"], case["d"], case["hkv"], case["group"]
    half, par = p * d // 2, 4 * p * d // g
    got = blocks[ids]
    code = got[:, :, part * half:(part + 1) * half].reshape(-1, hkv, p, d // 2)
    code = torch.stack((code & 15, code >> 4), -1).reshape(-1, hkv, p, d // g, g).float()
    at = 2 * half + part * par
    par = got[:, :, at:at + par].contiguous().view(torch.float16).reshape(-1, hkv, p, d // g, 2).float()
    val = code * par[..., :1] + par[..., 1:]
    return val.permute(1, 0, 2, 3, 4).reshape(hkv, -1, d)


def _attention(s):
    case = s["case"]
    hq, hkv, d, window = case["hq"], case["hkv"], case["d"], case["window"]
    out = torch.empty_like(s["q"])
    at = 0
    for i, (n, a) in enumerate(zip(s["host_lens"], s["host_adds"])):
        ids = s["table"][i, :_cdiv(n, case["page"])].long()
        keys = _pages_values(s["blocks"], ids, case, 0)[:, :n]
        vals = _pages_values(s["blocks"], ids, case, 1)[:, :n]
        rows = max(1, (1 << 28) // (hq * n))
        for r in range(0, a, rows):
            m = min(rows, a - r)
            q = s["q"][at + r:at + r + m].float() * s["scale"]
            q = q.reshape(m, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
            score = (q @ keys.transpose(1, 2)).reshape(hkv, hq // hkv, m, n)
            pos = (n - a + r + torch.arange(m, device=score.device))[:, None]
            key = torch.arange(n, device=score.device)
            hide = key > pos
            if window:
                hide = hide | (key <= pos - window)
            score.masked_fill_(hide, -math.inf)
            score = torch.exp(score - score.amax(-1, keepdim=True))
            total = score.sum(-1, keepdim=True)
            mix = (score.reshape(hkv, -1, n) @ vals).reshape(hkv, hq // hkv, m, d) / total
            out[at + r:at + r + m] = mix.permute(2, 0, 1, 3).reshape(m, hq, d).half()
        at += a
    return out


def _plan(s):
    p, room = s["case"]["page"], s["room"]
    cached, added, free = s["cached"].long(), s["added"].long(), s["free"]
    b, width = s["table"].shape
    zero = torch.zeros(1, dtype=torch.long, device=free.device)
    start = torch.cat((zero, torch.cumsum(added, 0)))
    held, total = (cached + p - 1) // p, (cached + added + p - 1) // p
    need = total - held
    at = torch.cumsum(need, 0) - need
    index = torch.arange(width, device=free.device)
    fresh = (index >= held[:, None]) & (index < total[:, None])
    src = (at[:, None] + index - held[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[src], s["table"])
    req = torch.repeat_interleave(torch.arange(b, device=free.device), added, output_size=s["tokens"])
    pos = cached[req] + torch.arange(s["tokens"], device=free.device) - start[req]
    slot = table[req, pos // p].long() * p + pos % p
    out = {"table": table, "start": start.int(), "lens": (cached + added).int()}
    for name, val, kind in (("token_req", req, torch.int32), ("token_pos", pos, torch.int32),
                            ("slots", slot, torch.int64)):
        full = torch.full((room,), -1, dtype=kind, device=free.device)
        full[:s["tokens"]] = val.to(kind)
        out[name] = full
    taken = need.sum()
    out["counts"] = torch.stack((start[-1], taken, taken, torch.zeros_like(taken))).int()
    return out


def _append(s):
    case = s["case"]
    p, d, hkv, g = case["page"], case["d"], case["hkv"], case["group"]
    half = p * d // 2
    page, off = s["slots"] // p, s["slots"] % p
    n = len(page)
    got = []
    for part, x in ((0, s["k"]), (1, s["v"])):
        code, scale, low = _codes_and_parameters(x.float(), g)
        pair = code.reshape(n, hkv, d // 2, 2).to(torch.uint8)
        rows = s["blocks"][:, :, part * half:(part + 1) * half].unflatten(2, (p, d // 2))
        rows[page, :, off] = pair[..., 0] | (pair[..., 1] << 4)
        par = torch.cat((scale, low), -1).half().view(torch.uint8).reshape(n, hkv, -1)
        at = 2 * half + part * p * par.shape[-1]
        rows = s["blocks"][:, :, at:at + p * par.shape[-1]].unflatten(2, (p, par.shape[-1]))
        rows[page, :, off] = par
        got.append((code * scale + low).reshape(n, hkv, d).half())
    return tuple(got)


def _lora(s):
    out = s["y"].clone()
    start = s["host_start"]
    for i, w in enumerate(s["host_adapter"]):
        if w < 0:
            continue
        rows = slice(start[i], start[i + 1])
        low = s["x"][rows].float() @ s["a"][w].float().t()
        delta = (low @ s["b"][w].float().t()) * s["scales"][w]
        out[rows] = (s["y"][rows].float() + delta).half()
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":  # whole numbers, the same however they are computed
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        g = case["group"]
        res = []
        for x in (s["k"], s["v"]):
            t = x.double().unflatten(-1, (-1, g))
            top, bot = t.max(-1).values, t.min(-1).values
            # FP16 roundings of exact values: the range of two FP16 numbers fits 64 bits
            step = torch.maximum(((top - bot) / 15).half().double(), torch.tensor(F16_TINY, dtype=torch.double,
                                                                                device=t.device))[..., None]
            level = ((t - bot[..., None]) / step).round().clamp(0, 15)
            res.append((bot[..., None] + level * step).flatten(-2))
        return tuple(res)
    if case["op"] == "lora":
        low = torch.zeros_like(s["y"], dtype=torch.double)
        owner = torch.repeat_interleave(s["adapter"].long(), (s["start"][1:] - s["start"][:-1]).long())
        for w in range(case["adapters"]):
            mine = (owner == w).nonzero().squeeze(1)
            if len(mine):
                both = s["b"][w].double() @ (s["a"][w].double() @ s["x"][mine].double().t())
                low[mine] = s["scales"][w].double() * both.t()
        return low + s["y"].double()
    if work(case)["flops"] > 4e12:
        return None
    d, g, page = case["d"], case["group"], case["page"]
    share = case["hq"] // case["hkv"]
    res = torch.zeros(s["q"].shape, dtype=torch.double, device="cuda")
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    begin = s["start"].tolist()
    for i, n in enumerate(s["lens"].tolist()):
        ids = s["table"][i].tolist()[:(n + page - 1) // page]
        spots = torch.arange(n, device="cuda")
        where = torch.tensor(ids, device="cuda")[spots // page]
        queries = s["q"][begin[i]:begin[i + 1]].double()
        a = queries.shape[0]
        for h in range(case["hkv"]):
            block = s["blocks"][where, h]
            rows = []
            for part in range(2):
                at = part * page * d // 2 + (spots % page) * (d // 2)
                words = torch.gather(block, 1, at[:, None] + torch.arange(d // 2, device="cuda"))
                words = words.contiguous().view(torch.int32)
                nib = ((words[:, :, None] >> shift) & 15).reshape(n, d).double()
                width = 4 * d // g
                at = page * d + part * page * width + (spots % page) * width
                par = torch.gather(block, 1, at[:, None] + torch.arange(width, device="cuda"))
                par = par.contiguous().view(torch.float16).double().reshape(n, d // g, 2)
                par = par.repeat_interleave(g, 1)
                rows.append(nib * par[:, :, 0] + par[:, :, 1])
            at = 0
            while at < a:
                m = min(a - at, max(1, (1 << 26) // (share * n)))
                qq = queries[at:at + m, h * share:(h + 1) * share]
                logit = torch.einsum("mgd,nd->mgn", qq, rows[0]) / math.sqrt(d)
                last = n - a + at + torch.arange(m, device="cuda")[:, None, None]
                seen = spots[None, None] <= last
                if case["window"]:
                    seen &= spots[None, None] > last - case["window"]
                prob = torch.softmax(torch.where(seen, logit, -math.inf), -1)
                res[begin[i] + at:begin[i] + at + m, h * share:(h + 1) * share] = torch.einsum("mgn,nd->mgd", prob,
                                                                                              rows[1])
                at += m
    return res
