"""What a serving program holds does not grow with the number of prompt lengths it has met."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import hybrid

pytestmark = pytest.mark.gpu


def test_prompts_of_many_lengths():
    gen = torch.Generator().manual_seed(0)
    layer = hybrid.AttentionLayer(256, 4, 2, 64, 2, 1024, gen, "cuda")
    x = torch.randn(2, 60, 256, generator=gen).bfloat16().cuda()

    def prompt(T):
        layer.lens.zero_()
        layer(x[:, :T])
        torch.cuda.synchronize()
        return torch.cuda.memory_allocated()

    for T in (1, 20, 50):
        before = prompt(T)
    for T in range(2, 60):
        after = prompt(T)
    assert after - before < 1 << 20
