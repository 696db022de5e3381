"""qk_norm_rope takes queries or keys alone, as tl_qk_norm_rope does."""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_quant_gb300 as tlq  # noqa: E402
from test_streams import fake, t  # noqa: E402,F401


@pytest.mark.parametrize("stream,on", [(None, "caller's"), ("side", "side")])
@pytest.mark.parametrize("side", [0, 1])
def test_one_side_is_enough(fake, monkeypatch, side, stream, on):  # noqa: F811
    made, launched = fake
    monkeypatch.setattr(torch, "zeros", lambda shape, dtype=None, device=None: torch.empty(shape, dtype, device))
    monkeypatch.setattr(tlq, "tl_qk_norm_rope", lambda *a: launched.append(a))
    heads = [None, None]
    heads[side] = t(3, 4, 64)
    got = tlq.qk_norm_rope(None, *heads, None, stream=stream)
    assert len(made) == len(launched) == 1 and made[0].on == on and made[0].shape == (3, 4, 64)
    assert got[side] is made[0] and got[1 - side] is None and launched[0][4 + side] is made[0]
    assert made[0].kept_for == ([] if stream is None else ["caller's"])


@pytest.mark.gpu
def test_alone_as_together(lib):
    g = torch.Generator("cuda").manual_seed(1)
    q, k = (torch.randn(5, h, 128, device="cuda", generator=g).half() for h in (4, 2))
    w = torch.randn(128, device="cuda", generator=g).half()
    f = 10000.0 ** (-torch.arange(0, 128, 2, device="cuda", dtype=torch.float64) / 128)
    rope, pos = lib.Rope(lib.rope_table(50, f)), torch.tensor([0, 3, -1, 49, 7], dtype=torch.int32, device="cuda")
    both = lib.qk_norm_rope(rope, q, k, pos, w, w)
    one, none = lib.qk_norm_rope(rope, q, None, pos, w)
    assert none is None and torch.equal(one, both[0]) and not one[2].any()
    none, one = lib.qk_norm_rope(rope, None, k, pos, k_weight=w, stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    assert none is None and torch.equal(one, both[1])
    with pytest.raises(ValueError, match="both None"):
        lib.qk_norm_rope(rope, None, None, pos)
