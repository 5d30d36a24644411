"""Linear attention over dense batches whose sequences are split into segments, forward and gradient, against the fp64
restatement; the bounds are those of mixers.py."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from test_linear_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("case", [  # as in test_linear_attn.py
    ([2000, 2000], False, 2, 64, 64, True, False),    # 16 chunks a sequence, the last of 80 tokens
    ([2000, 2000], False, 2, 128, 64, True, True),
    ([2000, 2000], False, 2, 64, 128, True, False),
    ([1537], False, 2, 128, 128, True, False),        # the last segment is one token
    ([1601, 1601, 1601], False, 1, 128, 64, False, True),  # one of 65, no states
])
def test_dense_sequences_in_segments(case, io):
    c = Case(case, io, seed=31)
    assert c.plan._ws_bytes > 16  # room for segments' states: the sequences are split
    c.check(c.run())
    assert c.plan.status() == binding.DR_OK


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_decays_across_segments(io):
    """Heads that keep everything, that forget within a chunk, and that keep nothing."""
    g = torch.tensor([0.0, -0.3, -float("inf")])
    c = Case(([1700, 1700], False, 3, 64, 64, True, False), io, seed=32, g=g)
    assert c.plan._ws_bytes > 16
    c.check(c.run())
