"""A plan's status word is made on one stream and used on others."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding

pytestmark = pytest.mark.gpu


def busy(stream_work=60):
    """Some 20 ms of work on the current stream."""
    x = torch.empty(1 << 31, dtype=torch.uint8, device="cuda")
    for _ in range(stream_work):
        x.fill_(1)


def make(kind, **kw):
    return binding.LinearAttention(1, 40, 2, 64, 64, **kw) if kind == "linear" else binding.PromptAttention(1, 40, 2, 2, 64, **kw)


def call(kind, plan, x, g):
    if kind == "linear":
        return plan.forward(x, x, x, g)
    return plan.forward(x, x, x, want_lse=True)


@pytest.mark.parametrize("kind", ["prompt", "linear"])
def test_a_new_plan_on_another_stream(kind):
    """The zeros of the word wait behind other work when the plan is first used elsewhere; its memory held a code before."""
    x, g, side = torch.randn(1, 40, 2, 64).bfloat16().cuda(), torch.zeros(2).cuda(), torch.cuda.Stream()
    make(kind)  # whatever is loaded at first
    for first in ("status", "call"):
        torch.cuda.synchronize()
        old = [torch.full((4,), 1, dtype=torch.int32, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        del old
        busy()
        plan = make(kind)
        with torch.cuda.stream(side):
            if first == "call":
                call(kind, plan, x, g)
            assert plan.status() == binding.DR_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["prompt", "linear"])
def test_a_new_plan_is_captured_at_once(kind):
    """A plan that no call was made of before goes into a graph, also one that is made while the graph is captured."""
    x, g = torch.randn(1, 40, 2, 64).bfloat16().cuda(), torch.zeros(2).cuda()
    want = call(kind, make(kind), x, g)
    before = make(kind)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(kind, before, x, g)
        inside = make(kind)
        more = call(kind, inside, x, g)
    graph.replay()
    torch.cuda.synchronize()
    after = call(kind, inside, x, g)
    assert all(torch.equal(a, b) for r in (got, more, after) for a, b in zip(r, want))
    assert before.status() == inside.status() == binding.DR_OK
