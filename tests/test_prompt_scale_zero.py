"""Causal attention with a scale of zero, or near it, and products of queries and keys near the largest numbers."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from test_prompt_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("scale,size", [(0.0, 1e18), (1e-38, 1e18), (-1e-38, 1e18), (1e-37, 3e17)])
def test_large_products(scale, size, io):
    """A scale of zero makes all scores zero, whatever the products are (up to 1e38 here); small ones are taken as they
    are.  Forward only, with the bounds of test_prompt_attn.py."""
    case = ([300, 70], True, 2, 1, 64, 0, False)
    c = Case(case, io, seed=61)
    c.q *= size
    c.k *= size
    c.scale = scale
    c.plan = binding.PromptAttention(1, c.lay.T, 2, 1, 64, seqs=2, io=io, scale=scale)
    o, lse = c.forward()
    c.check(dict(o=o, lse=lse))
