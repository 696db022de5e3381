"""Blocks of a cluster look at each other's shared memory only once all of them have begun."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_quant_gb300", "csrc")
PEER = r"map_shared_rank\s*\(|\bmapa\."  # an address in another block's shared memory
BARRIER = r"cluster\.sync\s*\(|\bcluster_sync\s*\(|\bcluster_wait\s*\(|barrier\.cluster\.wait"


def functions(text):
    """(name, is a kernel, body) of the functions of a source, without comments."""
    text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))
    for m in re.finditer(r"(__global__|__device__)[^;{}=]*?(\w+)\((?:[^(){};]|\([^()]*\))*\)\s*\{", text):
        if m.group(2) in ("__launch_bounds__", "__align__"):
            continue
        at, depth = m.end(), 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(2), m.group(1) == "__global__", text[m.end():at]


def first(pattern, body):
    m = re.search(pattern, body)
    return m.start() if m else None


def kernels_of_peers():
    found = []
    for name in sorted(os.listdir(CSRC)):
        every = list(functions(open(os.path.join(CSRC, name)).read()))
        helpers = [f for f, kernel, body in every if not kernel and re.search(PEER, body)]
        peer = "|".join([PEER] + [r"\b%s\s*\(" % f for f in helpers])
        found += [(name, f, first(peer, body), first(BARRIER, body)) for f, kernel, body in every
                  if kernel and re.search(peer, body)]
    return found


def test_all_blocks_have_begun_before_one_looks_at_another():
    found = kernels_of_peers()
    assert {f for _, f, _, _ in found} >= {"sample_kernel", "lora_kernel"}
    for source, kernel, peer, barrier in found:
        assert barrier is not None and barrier < peer, (source, kernel)


@pytest.mark.gpu
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("vocab", [2, 3, 5, 8, 9, 17, 100])
def test_blocks_with_next_to_nothing_to_load(lib, vocab, half):
    """Rows of few values over several blocks, one call straight after another: a block is there to be looked at
    however short the others' loading is."""
    torch = pytest.importorskip("torch")
    from test_sample_gpu import compare, logits, plain

    x, u, g = logits(3, vocab, vocab, half)
    p = torch.full((3,), 0.8, device="cuda")
    compare(lib, x, u, p=p)
    want = plain(x, u, p=p)[0]
    out = [torch.full((3,), -7, dtype=torch.int32, device="cuda") for _ in range(200)]
    for tokens in out:
        lib.tl_sample(x, u, tokens, top_p=p)
    assert all(tokens.tolist() == want for tokens in out)
