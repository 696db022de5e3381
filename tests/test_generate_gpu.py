"""Rotations, cache, shared prefix and sampling together, as a serving loop uses them."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("common,prompts", [(130, (9, 1, 40, 3)), (16, (1, 1)), (77, (100, 30, 1))])
def test_generate(lib, common, prompts):
    """The attention's rows against 64 bits: queries and cached values are taken as they are, so what is left is
    the output's rounding (2^-11 of each value) and the weights' (2^-11 of the values, twice): 3 * 2^-11 of the
    norm where values are spread evenly, and half as much again for the values' own spread."""
    from generate import generate
    from test_sample_gpu import plain

    tokens, errors, _ = generate(steps=4, width=256, q_heads=4, kv_heads=2, head_dim=64, vocab=1000, common=common,
                                 prompts=prompts)
    assert len(errors) == 5 and max(errors) <= 4.5 * 2.0 ** -11
    for got, logits, uniform, temperature, top_k, top_p in tokens:
        assert got == plain(logits, uniform, temperature, top_k, top_p)[0]


def test_a_step_is_captured(lib):
    """A decode step replayed as a graph goes on like the same step called."""
    from generate import Model

    def model():
        m = Model(256, 4, 2, 64, 504, 3, 60, 16, 64, 400, seed=3)
        m.begin(torch.arange(100, device="cuda"))
        return m

    one = torch.ones(3, dtype=torch.int32, device="cuda")
    last, u = torch.arange(3, device="cuda"), torch.tensor([0.2, 0.5, 0.9], device="cuda")
    t, k, p = torch.tensor([0.0, 0.7, 1.1], device="cuda"), torch.tensor([0, 0, 40], dtype=torch.int32, device="cuda"), \
        torch.full((3,), 0.95, device="cuda")
    eager, want = model(), []
    ids = torch.tensor([1, 2, 3], device="cuda")
    for _ in range(6):
        ids = eager.step(ids, one, 1, last, u, t, k, p).long()
        want.append((ids.tolist(), eager.mixed[:3].clone(), eager.logits.clone()))
    m = model()
    ids = torch.tensor([1, 2, 3], device="cuda")
    got = []
    for _ in range(2):  # two steps called: the plan's buffers go in turn
        ids.copy_(m.step(ids, one, 1, last, u, t, k, p))
        got.append((ids.tolist(), m.mixed[:3].clone(), m.logits.clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # and two captured
        for _ in range(2):
            ids.copy_(m.step(ids, one, 1, last, u, t, k, p))
    for i in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert ids.tolist() == want[3 + 2 * i][0]
        assert torch.equal(m.mixed[:3], want[3 + 2 * i][1]) and torch.equal(m.logits, want[3 + 2 * i][2])
    for a, b in zip(got, want):
        assert a[0] == b[0] and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    lib.tl_check_status()
