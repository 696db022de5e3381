"""A step with rows behind its last token, as one captured for the largest batch has them."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_rows_behind_the_last_token_are_passed_over(lib):
    """The plan gives them position -1, behind a common beginning too: their queries stay as the projection left
    them, the cache and the requests' rows do not show them."""
    from generate import Model

    m = Model(256, 4, 2, 64, 504, 3, 60, 16, 64, 400, seed=3)
    m.begin(torch.arange(100, device="cuda"))
    added, pad = [4, 1, 2], 5
    ids = torch.randint(0, 504, (sum(added) + pad,), device="cuda", generator=m.gen)
    raw = m.heads(m.embed[ids])[0].clone()
    added_dev = torch.tensor(added, dtype=torch.int32, device="cuda")
    v = lambda *a: torch.tensor(a, device="cuda")  # noqa: E731
    m.step(ids, added_dev, 4, torch.cumsum(added_dev, 0) - 1, v(0.2, 0.5, 0.9), v(0.0, 0.7, 1.1), v(0, 0, 40).int(),
           v(0.95, 0.95, 0.95))
    used = sum(added)
    assert torch.equal(m.queries[used:], raw[used:])
    assert (m.queries[:used] != raw[:used]).flatten(1).any(1).all()
    want = m.reference(added)[:used]
    assert ((m.mixed[:used].double() - want).norm() / want.norm()).item() <= 4.5 * 2.0 ** -11
    lib.tl_check_status()
