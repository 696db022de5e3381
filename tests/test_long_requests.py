"""How the prompt kernel counts the work of requests of many rows: each count has one writer, long requests in any
number and order."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_quant_gb300", "csrc")


def test_counts_have_one_writer_between_barriers():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "kv_prefill.cu")).read())
    stores = [len(re.findall(r"request_units\[\w+\]\s*=[^=]", part)) for part in re.split(r"__syncthreads\s*\(\s*\)", text)]
    assert sum(stores) > 0 and max(stores) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("adds", [
    [300] * 40,                          # more long ones than warps, side by side
    ([260] + [1] * 11) * 8 + [700, 90],  # long ones as far apart as there are warps
    [1] * 31 + [1500] + [40] * 33 + [257, 256, 255],
    [300] * 3 + [2] * 380,               # 384 with the prefix's own
])
def test_long_and_short_requests(lib, adds, prefix):
    torch = pytest.importorskip("torch")
    from attention_bound import close
    from test_prefix_gpu import Batch

    b = Batch(lib, prefix, [a + 13 * i % 40 for i, a in enumerate(adds)], adds, 4, 1, 128, 128, 16, seed=len(adds))
    own = lib.kv4_attention(b.cache, b.q, b.start, b.lens, b.table, b.max_q)
    close(b, own, prefix=False)
    close(b, b.run())
    torch.cuda.synchronize()
    lib.tl_check_status()
