"""One plan on two streams without an event between them, and by two threads: every result is that of a call alone."""
import threading

import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding

from test_cache_attn import Case, up
from test_norm_rope import args, make, plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 70])
def test_attention(T):
    cases = [Case([9000, 5000], T, 8, 2, 128, 64, "i8", "bf16", "bf16", seed=s) for s in (71, 72)]
    # the second case's queries over the first one's cache
    c, qs = cases[0], [x.q for x in cases]
    p = binding.CacheAttention(c.cache, 2, T, 8, scale=c.softmax_scale)
    table, lens = up(c.table), up(c.lens)
    alone = [[t.clone() for t in p.forward(q, table, lens, want_lse=True)] for q in qs]
    torch.cuda.synchronize()
    got = [[], []]

    def calls(i, stream):
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[i].append(p.forward(qs[i], table, lens, want_lse=True))

    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(p.forward(qs[i], table, lens, want_lse=True))
    for both in (streams, [streams[0]] * 2):
        threads = [threading.Thread(target=calls, args=(i, both[i])) for i in (0, 1)]
        [t.start() for t in threads]
        [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in (0, 1):
        assert len(got[i]) == 50
        assert all(torch.equal(a, b) for pair in got[i] for a, b in zip(pair, alone[i]))


def test_gradient():
    case = (2, 1500, 8, 2, 128, 128, "halves", "bf16", "bf16", True)
    xs, p = [make(*case, seed=s) for s in (73, 74)], plan(case)
    alone = [p.backward(*args(x), x["dyq"], x["dyk"]) for x in xs]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, x in enumerate(xs):
            with torch.cuda.stream(streams[i]):
                got[i].append(p.backward(*args(x), x["dyq"], x["dyk"]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g[n], alone[i][n]) for g in got[i] for n in g)
