"""Causal attention where the scores are unusual: scales below and at zero, scores that are not finite."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from test_prompt_attn import Case

pytestmark = pytest.mark.gpu


def scaled(case, io, scale, seed):
    c = Case(case, io, seed=seed)
    _, _, Hq, H, d, window, _ = case
    c.scale = scale
    c.plan = binding.PromptAttention(c.lay.B, c.lay.T, Hq, H, d, seqs=c.lay.seqs, io=io, scale=scale, window=window)
    return c


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [-0.11, 0.0, 1e-6])
@pytest.mark.parametrize("case", [([300, 70, 0, 1], True, 4, 2, 64, 0, False), ([300], False, 2, 1, 128, 37, True)])
def test_scales(case, scale, io):
    c = scaled(case, io, scale, seed=51)
    o, lse = c.forward()
    c.check(dict(o=o, lse=lse, **c.backward(o, lse)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_key_of_minus_infinity(sign, io):
    """The row that sees this key alone is NaN with lse -inf; to the others it is no key."""
    c = scaled(([300], False, 1, 1, 64, 0, False), io, sign * 0.125, seed=52)
    c.q.fill_(1.0)
    c.k[:, 0] = -sign * float("inf")
    o, lse = c.forward()
    assert torch.isnan(o[0, 0]).all() and lse[0, 0, 0] == -float("inf")
    rest = binding.PromptAttention(1, 299, 1, 1, 64, io=io, scale=sign * 0.125)
    want, wlse = rest.forward(*(t[:, 1:].contiguous() for t in (c.q, c.k, c.v)), want_lse=True)
    # The same weights and sums in another place of the tiles: fp32 sums of up to 299 weights and products, each side off
    # by 2^-16 (2^-17 the powers, 300 2^-24 the sums) of sums of sizes below the largest value; bf16: the weights'
    # operands 2^-8 each side, and the rounding of o, 2^-8 each side.
    top = float(c.v.float().abs().max())
    assert float((lse[:, 1:] - wlse).abs().max()) <= 2 * 2.0 ** -16 * (1 + float(wlse.abs().max()))
    assert float((o[:, 1:].float() - want.float()).abs().max()) <= top * (2.0 ** -15 if io == "f32" else 4 * 2.0 ** -8 + 2.0 ** -15)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 60])
def test_a_key_that_is_no_number_reaches_the_rows_that_see_it(window, bad, io):
    case = ([300], False, 2, 1, 64, window, False)
    c, clean = Case(case, io, seed=53), Case(case, io, seed=53)
    c.q.abs_(), clean.q.abs_()  # so that an infinite key makes infinite scores
    c.k[:, 140] = bad
    o, lse = c.forward()
    want, wlse = clean.forward()
    last = 140 + window if window else 300
    assert torch.isnan(o[:, 140:last]).all()
    for a, b in ((0, 140), (last, 300)):
        assert torch.equal(o[:, a:b], want[:, a:b]) and torch.equal(lse[:, a:b], wlse[:, a:b])
    assert c.plan.status() == binding.DR_OK
