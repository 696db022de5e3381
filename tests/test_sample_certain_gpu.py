"""Rows that keep one token: its log-probability is 0, not a little less.  Equal ones: ln of their number."""
import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def rows(vocab, half):
    g = torch.Generator("cuda").manual_seed(vocab)
    x = torch.randn(7, vocab, device="cuda", generator=g)
    return x.half() if half else x, torch.rand(7, device="cuda", generator=g)


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 900, 40001, 300007])
def test_one_kept_token_is_certain(lib, vocab, half):
    x, u = rows(vocab, half)
    x[:, vocab // 2] = 9.0  # alone at the top
    f = lambda v, kind=torch.float32: torch.full((7,), v, dtype=kind, device="cuda")  # noqa: E731
    cold = x.clone()
    cold[:, :vocab // 2] = cold[:, vocab // 2 + 1:] = -float("inf")
    t = torch.tensor([0.0, 1e-3, 1.0, 2.0, 0.5, 1.0, 0.01], device="cuda")
    for got in (lib.sample(x, u, top_k=f(1, torch.int32)), lib.sample(x, u, top_p=f(0.0)), lib.sample(x, u, min_p=f(1.0)),
                lib.sample(cold, u, t), lib.sample(cold, u, t, top_p=f(0.9)), lib.sample(x, u, f(1e-3)),
                lib.sample(x, u, t, f(1, torch.int32), f(0.3), f(0.1))):
        assert got[0].tolist() == [vocab // 2] * 7
        assert got[1].tolist() == [0.0] * 7


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("vocab", [2, 3, 700, 65536])
def test_equal_tokens_share(lib, vocab, half):
    """-ln n: the sum is a whole number of the largest weight, so what is left are the logarithm's own roundings
    (the argument's half step moves it by 2^-24, the function by two steps of its size)."""
    x, u = rows(vocab, half)
    x[:] = -1.5
    _, logs = lib.sample(x, u, torch.full((7,), 0.7, device="cuda"))
    want = -math.log(vocab)
    assert ((logs.double() - want).abs() <= 2.0 ** -24 + 2.0 ** -22 * abs(want)).all()
