"""A bounded wait that ran out in any layer of a stack shows in the stack's status.  Here the host writes what such a wait
would leave in the status words."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding, hybrid

pytestmark = pytest.mark.gpu


@pytest.fixture
def plans(monkeypatch):
    """All plans of the token mixers that the test's stacks make, in order."""
    made = []
    for name in ("LinearAttention", "PromptAttention"):
        class Kept(getattr(binding, name)):
            def __init__(self, *args, **kw):
                super().__init__(*args, **kw)
                made.append(self)
        monkeypatch.setattr(binding, name, Kept)
    return made


def assert_all_show(stack, plans):
    assert plans and stack.status() == binding.DR_OK
    for p in plans:
        p.word[0] = 1
        assert stack.status() == binding.DR_ERR_TIMEOUT
        p.word[0] = 0
        assert stack.status() == binding.DR_OK


def test_serving_stack(plans):
    """Prompts of two lengths and steps, whose plans come and go."""
    stack = hybrid.HybridStack(2, linear="decay")
    x = torch.randn(2, 60, 256, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    stack(x[:, :30]), stack(x[:, 30:50]), stack(x[:, 50:51])
    torch.cuda.synchronize()
    assert_all_show(stack, plans)


def test_training_stack(plans):
    stack = hybrid.TrainingStack(50, 2)
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(50, 256, generator=gen).bfloat16().cuda() for _ in range(2))
    stack.forward(x, torch.tensor([0, 20, 50], dtype=torch.int32).cuda())
    stack.backward(dy)
    torch.cuda.synchronize()
    assert len(plans) == 4
    assert_all_show(stack, plans)
