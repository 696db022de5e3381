"""Several requests through one attention layer with INT4 weights, adapters and a
4-bit paged cache: prompts first, then single tokens, all in one batch a step.

    python examples/serve_step.py [--steps N]

A step is seven calls and no host copy of a length:

    tl_kv_plan        block tables, slots and positions from the requests' lengths
    tl_quant_gemm_ws  the fused projection: queries, keys, values of every token
    tl_lora_add       each request's adapter on it, in place
    tl_kv4_append     keys and values into the cache, read from the projection's columns
    tl_kv4_attention  the queries over everything their requests have cached
    tl_quant_gemm_ws  the output projection
    tl_lora_add       its adapter, in place

Weights, adapters and activations are random; the figures printed are the step
times and the distance from the same layer in 64 bits over the cached values.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import weight_only_int4_quant_gb300 as tlq

BITS, GROUP = 4, 128


class Layer:
    """Projections, adapters and cache, with the buffers of steps of up to `rows` tokens."""

    def __init__(self, width, q_heads, kv_heads, head_dim, requests, pages, page_size, rows, rank, adapters, seed=0):
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.requests = q_heads, kv_heads, head_dim, requests
        self.nq, self.nk = q_heads * head_dim, kv_heads * head_dim
        self.qkv = self.weights(self.nq + 2 * self.nk, width)
        self.o = self.weights(width, self.nq)
        self.qkv_lora = self.adapter(self.nq + 2 * self.nk, width, rank, adapters)
        self.o_lora = self.adapter(width, self.nq, rank, adapters)
        self.lora_scales = 0.5 + torch.rand(adapters, device="cuda", generator=self.gen)
        self.cache = tlq.KV4Cache(pages, kv_heads, head_dim, page_size, group=min(128, head_dim))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((requests, pages), -1, **i32)
        self.free_pages = torch.randperm(pages, device="cuda", generator=self.gen).int()
        self.cached = torch.zeros(requests, **i32)
        # two in turn: a step reads the free list's head where the step before left it
        self.counts = [torch.zeros(4, **i32) for _ in range(2)]
        self.seq_lens = [torch.zeros(requests, **i32) for _ in range(2)]
        self.q_start = torch.empty(requests + 1, **i32)
        self.token_req, self.token_pos = torch.empty(rows, **i32), torch.empty(rows, **i32)
        self.slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        f16 = dict(dtype=torch.float16, device="cuda")
        self.rows = torch.empty(rows, self.nq + 2 * self.nk, **f16)
        self.mixed = torch.empty(rows, q_heads, head_dim, **f16)
        self.out = torch.empty(rows, width, **f16)
        self.turn = 0

    def rand(self, *shape):
        return torch.rand(shape, device="cuda", generator=self.gen)

    def weights(self, n, k):
        codes = torch.randint(0, 16, (n, k), dtype=torch.uint8, device="cuda", generator=self.gen)
        scales = ((0.005 + 0.015 * self.rand(n, k // GROUP)) * 8 / k ** 0.5).half()
        zeros = (6 + 3 * self.rand(n, k // GROUP)).half()
        dense = (codes.view(n, -1, GROUP).double() - zeros[..., None].double()) * scales[..., None].double()
        return tlq.pack_weights(codes, BITS), scales, zeros, dense.view(n, k)

    def adapter(self, n, k, rank, count):
        randn = lambda *s: torch.randn(s, device="cuda", generator=self.gen)  # noqa: E731
        return (randn(count, rank, k) * k ** -0.5).half(), (randn(count, n, rank) * 0.2 * rank ** -0.5).half()

    def step(self, x, added, adapters, max_q):
        """Output rows of the step's tokens x [tokens, width]; added, adapters: int32 per request."""
        t, was = x.shape[0], self.turn
        self.turn = now = 1 - was
        seq = self.seq_lens[now]
        tlq.tl_kv_plan(self.cached, added, self.table, self.free_pages, self.q_start, seq, self.token_req,
                       self.token_pos, self.slots, self.counts[now], self.cache.page_size, self.cache.num_pages,
                       free_head=self.counts[was][2:3])
        self.cached = seq
        rows, mixed, out = self.rows[:t], self.mixed[:t], self.out[:t]
        self.project(x, self.qkv, rows)
        tlq.tl_lora_add(x, *self.qkv_lora, self.lora_scales, self.q_start, adapters, max_q, rows, rows)
        heads = rows.view(t, -1, self.head_dim)
        q, k, v = heads.split((self.q_heads, self.kv_heads, self.kv_heads), 1)
        tlq.tl_kv4_append(self.cache, k, v, self.slots[:t])
        tlq.tl_kv4_attention(self.cache, q, mixed, self.q_start, seq, self.table, max_q, self.head_dim ** -0.5,
                             workspace=self.workspace(max_q))
        flat = mixed.view(t, self.nq)
        self.project(flat, self.o, out)
        tlq.tl_lora_add(flat, *self.o_lora, self.lora_scales, self.q_start, adapters, max_q, out, out)
        return out

    def workspace(self, max_q):
        need = tlq.tl_kv4_attention_workspace_size(self.q_heads, self.kv_heads, self.head_dim, max_q)
        if getattr(self, "_ws", None) is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        return self._ws

    def project(self, x, w, out):
        ws = tlq.gemm_workspace(x.shape[0], out.shape[1], x.shape[1], BITS, GROUP)
        tlq.tl_quant_gemm_ws(x, w[0], w[1], w[2], out, BITS, GROUP, workspace=ws)

    def reference(self, x, added, adapters):
        """The step once more in 64 bits, from the cached values (after step())."""
        x = x.double()
        rows = x @ self.qkv[3].t()
        owner = [i for i, a in enumerate(added) for _ in range(a)]
        low = lambda x, pair: torch.stack([  # noqa: E731
            self.lora_scales[adapters[i]].double() * (pair[1][adapters[i]].double() @ (pair[0][adapters[i]].double() @ r))
            if adapters[i] >= 0 else torch.zeros(pair[1].shape[1], dtype=torch.double, device="cuda")
            for i, r in zip(owner, x)])
        q = (rows + low(x, self.qkv_lora))[:, :self.nq].view(-1, self.q_heads, self.head_dim)
        mixed, at, p = torch.empty_like(q), 0, self.cache.page_size
        for i, (n, a) in enumerate(zip(self.cached.tolist(), added)):
            pos = torch.arange(n, device="cuda")
            slots = self.table[i].long()[pos // p] * p + pos % p
            k, v = (torch.empty(n, self.kv_heads, self.head_dim, dtype=torch.float16, device="cuda") for _ in "kv")
            tlq.tl_kv4_read(self.cache, slots, k, v)
            k, v = (z.double().repeat_interleave(self.q_heads // self.kv_heads, 1) for z in (k, v))
            s = torch.einsum("qhd,khd->hqk", q[at:at + a], k) * self.head_dim ** -0.5
            s.masked_fill_(pos > pos[n - a:, None], float("-inf"))
            mixed[at:at + a] = torch.einsum("hqk,khd->qhd", torch.softmax(s, -1), v)
            at += a
        mixed = mixed.view(-1, self.nq)
        return mixed @ self.o[3].t() + low(mixed, self.o_lora)


def serve(steps=8, width=2048, q_heads=16, kv_heads=16, head_dim=128, prompts=(40, 1, 200, 7), rank=16, adapters=3,
          check=True):
    """Runs the prompts and `steps` single-token steps; returns (relative errors, ms of each step)."""
    n, page = len(prompts), 16
    pages = sum(-(-(p + steps) // page) for p in prompts)
    layer = Layer(width, q_heads, kv_heads, head_dim, n, pages, page, sum(prompts), rank, adapters)
    which = [i % (adapters + 1) - 1 for i in range(n)]  # the first request has no adapter
    errors, times = [], []
    which_dev = torch.tensor(which, dtype=torch.int32, device="cuda")
    for step in range(steps + 1):
        added = list(prompts) if step == 0 else [1] * n
        added_dev = torch.tensor(added, dtype=torch.int32, device="cuda")
        x = torch.randn(sum(added), width, device="cuda", generator=layer.gen).half()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in "be")
        begin.record()
        out = layer.step(x, added_dev, which_dev, max(added))
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
        tlq.tl_check_status()
        short = layer.counts[layer.turn].tolist()[3]
        assert short == 0, "%d pages short" % short
        if check:
            want = layer.reference(x, added, which)
            errors.append(((out.double() - want).norm() / want.norm()).item())
    return errors, times


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    errors, times = serve(ap.parse_args().steps)
    print("prompts: %.3f ms, relative error %.1e" % (times[0], errors[0]))
    for ms, err in zip(times[1:], errors[1:]):
        print("step:    %.3f ms, relative error %.1e" % (ms, err))
