"""What is not finite in a channel that no rotation turns stays in its channel: the definition joins only the
channels of a pair."""
import pytest
import torch

from test_norm_rope import args, make, plan

pytestmark = pytest.mark.gpu

CASES = [  # B, T, Hq, Hk, d, rot, style, io, out, packed
    (1, 9, 5, 2, 64, 32, "halves", "f32", "f32", False),
    (1, 9, 5, 2, 64, 32, "pairs", "f32", "f32", False),
    (2, 7, 3, 2, 128, 96, "halves", "bf16", "bf16", True),
    (2, 7, 3, 2, 128, 64, "pairs", "bf16", "bf16", True),
    (1, 5, 2, 2, 96, 0, "halves", "f32", "bf16", False),
]
AT = {64: 40, 128: 100, 96: 13}  # a channel that is not rotated


def others(d):
    return [c for c in range(d) if c != AT[d]]


@pytest.mark.parametrize("case", CASES)
def test_an_infinite_value(case):
    """r = 0 in its row: every other channel of the row is x 0 w = 0, its own is no number."""
    d = case[4]
    x = make(*case, seed=61)
    p = plan(case)
    good, _ = p.forward(*args(x))
    x["q"][0, 3, 1, AT[d]] = float("inf")
    y, _ = p.forward(*args(x))
    assert y[0, 3, 1, AT[d]].isnan() and (y[0, 3, 1, others(d)] == 0).all()
    y[0, 3, 1] = good[0, 3, 1]
    assert torch.equal(y, good)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_weight(case, bad):
    d = case[4]
    x = make(*case, seed=62)
    p = plan(case)
    good, gk = p.forward(*args(x))
    grad = p.backward(*args(x), x["dyq"], x["dyk"])
    x["wq"][AT[d]] = bad
    y, yk = p.forward(*args(x))
    assert not y[..., AT[d]].isfinite().any()
    assert torch.equal(y[..., others(d)], good[..., others(d)]) and torch.equal(yk, gk)
    g = p.backward(*args(x), x["dyq"], x["dyk"])  # dw does not know the weight
    assert torch.equal(g["dwq"], grad["dwq"]) and torch.equal(g["dwk"], grad["dwk"])


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_an_incoming_gradient(case, bad):
    d = case[4]
    x = make(*case, seed=63)
    p = plan(case)
    good = p.backward(*args(x), x["dyq"], x["dyk"])
    x["dyq"][0, 2, 0, AT[d]] = bad
    g = p.backward(*args(x), x["dyq"], x["dyk"])
    assert not g["dwq"][AT[d]].isfinite()
    assert torch.equal(g["dwq"][others(d)], good["dwq"][others(d)])
    g["dq"][0, 2, 0] = good["dq"][0, 2, 0]
    assert torch.equal(g["dq"], good["dq"]) and torch.equal(g["dk"], good["dk"])
