"""The hybrid stack as a serving program runs it: a prompt at once, then token by token."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding, hybrid

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("attention", [dict(), dict(code="e4m3", page=16, rot=32), dict(window=40, page=32)])
def test_prompt_and_steps_agree_with_the_whole(attention):
    B, T, steps, hidden = 2, 150, 5, 256
    x = torch.randn(B, T + steps, hidden, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    whole = hybrid.HybridStack(B, **attention)(x)
    stack = hybrid.HybridStack(B, **attention)
    parts = [stack(x[:, :T])] + [stack(x[:, T + i:T + i + 1]) for i in range(steps)]
    got = torch.cat(parts, 1)
    assert stack.status() == binding.DR_OK and got.isfinite().all()
    # the prompt is the same computation up to the pages' scales (a started page of the prompt grows
    # later), the steps another order of it: bf16 activations through four layers, 2^-8 a rounding,
    # and the attention's codes of 2^-7 (int8) or 2^-4 (e4m3) of the largest value, averaged over many
    rel = lambda a, b: float((a - b).float().norm() / b.float().norm())  # noqa: E731
    assert rel(got[:, :T], whole[:, :T]) < 2e-2
    assert rel(got[:, T:], whole[:, T:]) < 4e-2


def test_the_command_runs(capsys):
    hybrid.main()
    assert "status 0" in capsys.readouterr().out


def test_steps_in_a_captured_graph():
    """A step is capture-safe: replays of one graph advance lengths, cache and states."""
    B, hidden = 2, 256
    xs = torch.randn(6, B, 1, hidden, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    plain, graphed = hybrid.HybridStack(B), hybrid.HybridStack(B)
    prompt = torch.randn(B, 70, hidden, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    plain(prompt), graphed(prompt)
    x = xs[0].clone()
    plain(xs[0]), graphed(x)  # a step before the capture: plans and attributes are in place
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = graphed(x)
    for i in range(1, 6):
        ref = plain(xs[i])
        x.copy_(xs[i])
        g.replay()
        assert torch.equal(y, ref)
    assert graphed.status() == binding.DR_OK
