"""Requests that share a prompt's beginning generate tokens through one attention layer with INT4 weights.

    python examples/generate.py [--steps N]

The common beginning goes into the cache once.  A step of all requests is then
seven calls and no host copy of a length or a token:

    tl_kv_plan               tables, slots and positions of the requests' own tokens
    tl_quant_gemm_ws         the fused projection: queries, keys, values
    tl_kv4_append_rope       keys normed, rotated and quantized into the cache with the values,
                             the queries normed and rotated in place
    tl_kv4_attention_prefix  the queries over the beginning and their requests' own tokens
    tl_quant_gemm_ws         the output projection
    tl_quant_gemm_ws         the logits
    tl_sample                a token for each request, from a uniform number each

Weights are random; the figures printed are step times and the distance of the
layer's output from the same in 64 bits over the cached values.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import weight_only_int4_quant_gb300 as tlq

BITS, GROUP, EPS = 4, 128, 1e-6


class Model:
    def __init__(self, width, q_heads, kv_heads, head_dim, vocab, requests, pages, page_size, rows, positions, seed=0):
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.nq = q_heads, kv_heads, head_dim, q_heads * head_dim
        self.embed = torch.randn(vocab, width, device="cuda", generator=self.gen).half()
        self.qkv = self.weights(self.nq + 2 * kv_heads * head_dim, width)
        self.o, self.head = self.weights(width, self.nq), self.weights(vocab, width)
        near_one = lambda: (1 + 0.1 * torch.randn(head_dim, device="cuda", generator=self.gen)).half()  # noqa: E731
        self.q_weight, self.k_weight = near_one(), near_one()
        freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        self.turns = tlq.rope_table(positions, freq)
        self.cache = tlq.KV4Cache(pages, kv_heads, head_dim, page_size, group=head_dim)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, pages), -1, **i32)
        order = torch.randperm(pages, device="cuda", generator=self.gen).int()
        self.order, self.cached = order, torch.zeros(requests, **i32)
        self.counts, self.turn = [torch.zeros(4, **i32) for _ in range(2)], 0
        self.seq_lens = [torch.zeros(requests, **i32) for _ in range(2)]
        self.q_start = torch.empty(requests + 1, **i32)
        self.token_req, self.token_pos = torch.empty(rows, **i32), torch.empty(rows, **i32)
        self.slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        f16 = dict(dtype=torch.float16, device="cuda")
        self.rows = torch.empty(rows, self.nq + 2 * kv_heads * head_dim, **f16)
        self.mixed, self.out = torch.empty(rows, q_heads, head_dim, **f16), torch.empty(rows, width, **f16)
        self.logits = torch.empty(requests, vocab, **f16)
        self.tokens, self.logprobs = torch.empty(requests, **i32), torch.empty(requests, device="cuda")
        self.workspace = self.cache.prefix_workspace(q_heads, rows, rows)

    def weights(self, n, k):
        codes = torch.randint(0, 16, (n, k), dtype=torch.uint8, device="cuda", generator=self.gen)
        scales = ((0.005 + 0.015 * torch.rand(n, k // GROUP, device="cuda", generator=self.gen)) * 8 / k ** 0.5).half()
        zeros = (6 + 3 * torch.rand(n, k // GROUP, device="cuda", generator=self.gen)).half()
        return tlq.pack_weights(codes, BITS), scales, zeros

    def project(self, x, w, out):
        ws = tlq.gemm_workspace(x.shape[0], out.shape[1], x.shape[1], BITS, GROUP)
        tlq.tl_quant_gemm_ws(x, w[0], w[1], w[2], out, BITS, GROUP, workspace=ws)

    def heads(self, x):
        rows = self.rows[:x.shape[0]]
        self.project(x, self.qkv, rows)
        return rows.view(len(rows), -1, self.head_dim).split((self.q_heads, self.kv_heads, self.kv_heads), 1)

    def begin(self, ids):
        """The common beginning into pages of its own, in pieces of the buffers' rows."""
        n, p = len(ids), self.cache.page_size
        self.prefix_len = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.prefix_table = self.order[:-(-n // p)].contiguous()
        self.free_pages = self.order[-(-n // p):].contiguous()
        # own tokens lie behind the common ones: their positions count from a later row of the table, and what the
        # plan marks as no token stays marked
        rope, self.rope = tlq.Rope(self.turns), tlq.Rope(self.turns[n:])
        for at in range(0, n, len(self.rows)):
            pos = torch.arange(at, min(n, at + len(self.rows)), dtype=torch.int32, device="cuda")
            slots = self.prefix_table.long()[pos // p] * p + pos % p
            _, k, v = self.heads(self.embed[ids[at:at + len(pos)]])
            tlq.tl_kv4_append_rope(self.cache, rope, k, v, pos, slots, self.k_weight, eps=EPS)

    def step(self, ids, added, max_q, last, uniform, temperature, top_k, top_p):
        """Each request's next token, after its tokens of this step (ids, laid out request after request; last: the
        row of each request's last one)."""
        t, was = ids.shape[0], self.turn
        self.turn = now = 1 - was
        seq = self.seq_lens[now]
        tlq.tl_kv_plan(self.cached, added, self.table, self.free_pages, self.q_start, seq, self.token_req,
                       self.token_pos, self.slots, self.counts[now], self.cache.page_size, self.cache.num_pages,
                       free_head=self.counts[was][2:3])
        self.cached = seq
        q, k, v = self.heads(self.embed[ids])
        tlq.tl_kv4_append_rope(self.cache, self.rope, k, v, self.token_pos[:t], self.slots[:t], self.k_weight, q, q,
                               self.q_weight, EPS)
        self.queries, mixed, out = q, self.mixed[:t], self.out[:t]
        tlq.tl_kv4_attention_prefix(self.cache, q, mixed, self.q_start, seq, self.table, self.prefix_len,
                                    self.prefix_table, max_q, self.head_dim ** -0.5, workspace=self.workspace)
        self.project(mixed.view(t, self.nq), self.o, out)
        self.project(out[last], self.head, self.logits)
        tlq.tl_sample(self.logits, uniform, self.tokens, temperature, top_k, top_p, logprobs=self.logprobs)
        return self.tokens

    def reference(self, added):
        """The mixed rows of the last step in 64 bits, from its queries and the cached values."""
        p, at = self.cache.page_size, 0
        q = self.queries.double()
        want = torch.empty_like(q)

        def read(table, n):
            pos = torch.arange(n, device="cuda")
            k, v = (torch.empty(n, self.kv_heads, self.head_dim, dtype=torch.float16, device="cuda") for _ in "kv")
            tlq.tl_kv4_read(self.cache, table.long()[pos // p] * p + pos % p, k, v)
            return k, v

        n = int(self.prefix_len)
        front = read(self.prefix_table, n)
        for i, (m, a) in enumerate(zip(self.cached.tolist(), added)):
            k, v = (torch.cat(z).double().repeat_interleave(self.q_heads // self.kv_heads, 1)
                    for z in zip(front, read(self.table[i], m)))
            s = torch.einsum("qhd,khd->hqk", q[at:at + a], k) * self.head_dim ** -0.5
            key = torch.arange(n + m, device="cuda")
            s.masked_fill_(key > (n + m - a + torch.arange(a, device="cuda"))[:, None], float("-inf"))
            want[at:at + a] = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v)
            at += a
        return want


def generate(steps=8, width=2048, q_heads=16, kv_heads=4, head_dim=128, vocab=32000, common=1000, prompts=(9, 1, 40, 3),
             check=True, seed=0):
    """(tokens of each step, relative errors, ms of each step); tokens are a list a step."""
    n, page = len(prompts), 16
    rows = max(sum(prompts), 64)
    pages = -(-common // page) + sum(-(-(p + steps) // page) for p in prompts)
    m = Model(width, q_heads, kv_heads, head_dim, vocab, n, pages, page, rows, common + max(prompts) + steps + 1, seed)
    draw = lambda count: torch.randint(0, vocab, (count,), device="cuda", generator=m.gen)  # noqa: E731
    m.begin(draw(common))
    ids = draw(sum(prompts))
    temperature = torch.linspace(0.0, 1.2, n, device="cuda")  # the first request is greedy
    top_k = torch.tensor([0, 50, 0, 8] * n, dtype=torch.int32, device="cuda")[:n].contiguous()
    top_p = torch.full((n,), 0.9, device="cuda")
    tokens, errors, times = [], [], []
    for step in range(steps + 1):
        added = list(prompts) if step == 0 else [1] * n
        added_dev = torch.tensor(added, dtype=torch.int32, device="cuda")
        last = torch.cumsum(added_dev, 0) - 1
        uniform = torch.rand(n, device="cuda", generator=m.gen)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in "be")
        begin.record()
        got = m.step(ids, added_dev, max(added), last, uniform, temperature, top_k, top_p)
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
        tlq.tl_check_status()
        assert m.counts[m.turn].tolist()[3] == 0, "the cache is full"
        tokens.append((got.tolist(), m.logits.clone(), uniform, temperature, top_k, top_p))
        ids = got.long()
        if check:
            mixed, want = m.mixed[:sum(added)].double(), m.reference(added)
            errors.append(((mixed - want).norm() / want.norm()).item())
    return tokens, errors, times


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    tokens, errors, times = generate(ap.parse_args().steps)
    for (ids, *_), err, ms in zip(tokens, errors, times):
        print("%.3f ms, relative error %.1e, tokens %s" % (ms, err, ids))
