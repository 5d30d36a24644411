"""Plans of PromptAttention and LinearAttention on several streams and threads: every result is that of a call alone."""
import threading

import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from test_linear_attn import Case as Linear
from test_prompt_attn import Case as Prompt

pytestmark = pytest.mark.gpu


def prompt_call(plan, c):
    o, lse = plan.forward(c.q, c.k, c.v, cu=c.lay.cu, want_lse=True)
    return [o, lse, *plan.backward(c.q, c.k, c.v, o, lse, c.dO, cu=c.lay.cu).values()]


def linear_call(plan, c):
    o, hT = plan.forward(c.q, c.k, c.v, c.g, h0=c.h0, cu=c.lay.cu)
    return [o, hT, *plan.backward(c.q, c.k, c.v, c.g, c.dO, h0=c.h0, dhT=c.dhT, cu=c.lay.cu).values()]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("make,call,case", [
    (Prompt, prompt_call, ([700, 200, 31], True, 4, 2, 64, 0, True)),
    (Linear, linear_call, ([2400, 200, 31], True, 2, 64, 128, True, True)),  # the first one in segments
])
def test_two_threads_on_streams_of_their_own_and_on_one(make, call, case, io):
    cs = [make(case, io, seed=s, rest=0) for s in (41, 42)]
    plan = cs[0].plan
    alone = [call(plan, c) for c in cs]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in cs]

    def calls(i, stream):
        with torch.cuda.stream(stream):
            for _ in range(10):
                got[i].append(call(plan, cs[i]))

    for both in (streams, [streams[0]] * 2):
        threads = [threading.Thread(target=calls, args=(i, both[i])) for i in (0, 1)]
        [t.start() for t in threads]
        [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in (0, 1):
        assert len(got[i]) == 20
        assert all(torch.equal(a, b) for x in got[i] for a, b in zip(x, alone[i]))
    assert plan.status() == binding.DR_OK


def test_results_do_not_depend_on_the_workspace():
    """A workspace full of NaN gives the same bits."""
    for make, call, case in ((Prompt, prompt_call, ([300, 90], True, 4, 2, 128, 0, False)),
                             (Linear, linear_call, ([2400, 90], True, 2, 128, 128, True, False))):
        for io in ("f32", "bf16"):
            c = make(case, io, seed=43, rest=0)
            want = call(c.plan, c)
            for ws in c.plan._spaces.values():
                ws[:ws.numel() // 4 * 4].view(torch.float32).fill_(float("nan"))
            assert all(torch.equal(a, b) for a, b in zip(call(c.plan, c), want))
