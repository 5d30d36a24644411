"""GPU parity of causal attention over whole prompts and its gradient against the fp64 restatement; the bounds are
those of mixers.py."""
import numpy as np
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from mixers import OPERAND, TYPES, ULP, Layout, check, np64, tensors
from oracle import mixers as M

pytestmark = pytest.mark.gpu

CASES = [  # lengths, packed, Hq, H, d, window, inside a projection
    ([1], False, 1, 1, 64, 0, False),
    ([2, 2], False, 4, 2, 128, 0, True),
    ([63], False, 2, 2, 64, 0, False),
    ([64, 64, 64], False, 3, 1, 128, 0, False),
    ([65], False, 2, 1, 128, 1, True),
    ([129, 129], False, 4, 4, 64, 64, True),
    ([257], False, 5, 1, 128, 100, False),
    ([513], False, 2, 1, 64, 0, False),
    ([700], False, 1, 1, 128, 300, True),
    ([5, 0, 130, 1, 257, 64, 0], True, 4, 2, 128, 0, True),
    ([0, 0, 3], True, 2, 1, 64, 0, False),
    ([127, 128, 129, 255, 256, 1], True, 4, 1, 64, 0, False),
    ([300, 31, 511], True, 2, 2, 128, 129, False),
    ([300, 200], True, 2, 1, 64, 2 ** 31 - 1, False),
    ([1] * 70, True, 8, 2, 64, 0, False),
    ([17, 40, 3] * 14, True, 2, 1, 128, 9, True),
    ([1, 0, 3, 2] * 90, True, 1, 1, 64, 0, False),  # many sequences
]


def scale_of(d):
    return 1.3 * d ** -0.5


class Case:
    def __init__(self, case, io, seed=0, rest=11, spread=1.0):
        lens, packed, Hq, H, d, window, inside = case
        self.lay = lay = Layout(lens, packed, rest)
        self.io, self.window, self.scale = io, window, scale_of(d)
        self.q, self.k, self.v = tensors(lay, (Hq, H, H), (d, d, d), io, seed, inside, spread)
        self.dO = tensors(lay, (Hq,), (d,), io, seed + 1000)[0]
        self.plan = binding.PromptAttention(lay.B, lay.T, Hq, H, d, seqs=lay.seqs, io=io, scale=self.scale, window=window)

    def forward(self, **kw):
        return self.plan.forward(self.q, self.k, self.v, cu=self.lay.cu, want_lse=True, **kw)

    def backward(self, o, lse, **kw):
        return self.plan.backward(self.q, self.k, self.v, o, lse, self.dO, cu=self.lay.cu, **kw)

    def oracle(self):
        r = self.lay.rows
        return M.attention(r(self.q), r(self.k), r(self.v), self.lay.spans, self.scale, self.window, r(self.dO))

    def check(self, got):
        ref, size = self.oracle()
        top = size["lse"].max(initial=0.0)
        fine = 2.0 ** -16 * (1 + top) + max(self.lay.lens) * 2.0 ** -24
        op, u = OPERAND[self.io], ULP[self.io]
        times = dict(o=(1, 1), dv=(1, 2), dq=(3, 6), dk=(3, 6))
        for n, x in got.items():
            x = self.lay.rows(x)
            if n == "lse":
                check(x, ref[n], 2.0 ** -16 * (1 + top) + 2.0 ** -22 * np.abs(ref[n]), n)
            else:
                a, b = times[n]
                check(x, ref[n], (a * op + b * fine) * size[n] + u * np.abs(ref[n]), n)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case, io):
    c = Case(case, io)
    o, lse = c.forward()
    g = c.backward(o, lse)
    c.check(dict(o=o, lse=lse, **g))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_longer_sequences(d, io):
    c = Case(([1100, 1500], True, 4, 2, d, 0, False), io, seed=2)
    o, lse = c.forward()
    c.check(dict(o=o, lse=lse, **c.backward(o, lse)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_large_scores(io):
    """Scores up to a few hundred: a running maximum that keeps rising, weights of one key only."""
    c = Case(([600, 70], True, 2, 1, 128, 0, False), io, seed=4, spread=4.0)
    # keys grow along the sequence, so that later ones replace the maximum of earlier ones
    c.k *= torch.linspace(0.1, 2.0, c.lay.T).cuda()[None, :, None, None].to(c.k.dtype)
    o, lse = c.forward()
    c.check(dict(o=o, lse=lse, **c.backward(o, lse)))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_what_is_not_a_sequence_s_is_left_alone(io):
    """Rows behind the last sequence keep what they held, and what inputs hold there (or in another sequence) that is
    not finite does not get out; gradients go into ranges of one packed tensor and nothing beside them changes."""
    case = ([70, 0, 133, 5], True, 4, 2, 64, 0, False)
    c, clean = Case(case, io, seed=6), Case(case, io, seed=6)
    o0, lse0 = clean.forward()
    g0 = clean.backward(o0, lse0)
    lay, used = c.lay, c.lay.used
    for t in (c.q, c.k, c.v, c.dO):
        t[:, used:] = float("nan")
    for t in (c.k, c.v):
        t[:, 70:203] = float("inf")  # the second sequence with tokens
    dt = TYPES[io]
    o = torch.full_like(c.q, 7.0)
    lse = torch.full(c.q.shape[:3], 7.0).cuda()
    wide = torch.full((1, lay.T, 4 + 2 + 2 + 1, 64), 5.0, dtype=dt).cuda()
    out = dict(dq=wide[:, :, :4], dk=wide[:, :, 4:6], dv=wide[:, :, 6:8])
    c.forward(o=o, lse=lse)
    g = c.backward(o, lse, out=out)
    assert all(g[n].data_ptr() == out[n].data_ptr() for n in out)
    for lo, hi in ((0, 70), (203, 208)):
        assert torch.equal(o[:, lo:hi], o0[:, lo:hi]) and torch.equal(lse[:, lo:hi], lse0[:, lo:hi])
        assert all(torch.equal(g[n][:, lo:hi], g0[n][:, lo:hi]) for n in g)
    assert (o[:, used:] == 7).all() and (lse[:, used:] == 7).all()
    assert (wide[:, used:] == 5).all() and (wide[:, :, 8] == 5).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_offsets_out_of_range_touch_nothing_else(io):
    c = Case(([40, 60, 30], True, 2, 1, 64, 0, False), io, seed=8, rest=0)
    o, lse = c.forward()
    cu = torch.tensor([-9, 40, 20, 1 << 30], dtype=torch.int32).cuda()  # 0 .. 40, empty, 20 .. 130
    o2, lse2 = c.plan.forward(c.q, c.k, c.v, cu=cu, want_lse=True)
    g = c.plan.backward(c.q, c.k, c.v, o2, lse2, c.dO, cu=cu)
    torch.cuda.synchronize()
    assert torch.equal(o2[:, :20], o[:, :20]) and torch.isfinite(o2).all() and torch.isfinite(g["dq"]).all()


def test_scores_of_minus_infinity():
    """A row whose only key has the score -inf is NaN with lse -inf; rows that see another key too are not."""
    c = Case(([3], False, 1, 1, 64, 0, False), "f32", seed=9)
    c.q[:] = 1.0
    c.k[:, 0] = -float("inf")
    o, lse = c.forward()
    assert torch.isnan(o[0, 0]).all() and lse[0, 0, 0] == -float("inf")
    assert torch.isfinite(lse[0, 1:]).all() and torch.equal(o[0, 1], c.v[0, 1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_same_bits_every_time_and_on_two_streams(io):
    cs = [Case(([513, 200, 31], True, 8, 2, 128, 0, True), io, seed=s) for s in (10, 11)]
    plan = cs[0].plan
    call = lambda c: (lambda o, lse: (o, lse, *plan.backward(c.q, c.k, c.v, o, lse, c.dO, cu=c.lay.cu).values()))(  # noqa: E731
        *plan.forward(c.q, c.k, c.v, cu=c.lay.cu, want_lse=True))
    used = cs[0].lay.used
    alone = [call(c) for c in cs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], [[], []]
    for _ in range(10):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                got[i].append(call(c))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(a[:, :used], b[:, :used]) for x in got[i] for a, b in zip(x, alone[i]))


def test_captured_call_takes_new_lengths():
    c = Case(([200, 100, 36], True, 4, 2, 128, 0, False), "bf16", seed=12, rest=0)
    cu = c.lay.cu.clone()
    o, lse, out = torch.zeros_like(c.q), torch.zeros(c.q.shape[:3]).cuda(), [torch.zeros_like(t) for t in (c.q, c.k, c.v)]
    out = dict(zip(("dq", "dk", "dv"), out))

    def call():
        c.plan.forward(c.q, c.k, c.v, cu=cu, o=o, lse=lse)
        c.plan.backward(c.q, c.k, c.v, o, lse, c.dO, cu=cu, out=out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    for lens in ([200, 100, 36], [1, 335, 0], [0, 0, 336]):
        d = Case((lens, True, 4, 2, 128, 0, False), "bf16", seed=12, rest=0)
        cu.copy_(d.lay.cu)
        graph.replay()
        torch.cuda.synchronize()
        want, wlse = d.forward()
        assert torch.equal(o, want) and torch.equal(lse, wlse)
        assert all(torch.equal(out[n], x) for n, x in d.backward(want, wlse).items())


def test_gradient_against_differences():
    """fp32: <gradient, u> against (L(x + h u) - L(x - h u)) / 2h, h = 2^-6.  The difference is off by its third order,
    (change of a score)^2 ~ (h |u.k|)^2 < 2^-9 of the terms' sizes, and rounding, 2^-14 of L's terms over h."""
    c = Case(([90, 41], True, 4, 2, 64, 50, False), "f32", seed=14, rest=0)
    o, lse = c.forward()
    g = c.backward(o, lse)
    _, size = c.oracle()
    gen = torch.Generator().manual_seed(15)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv")):
        x = getattr(c, n)
        u = torch.randn(x.shape, generator=gen).cuda()
        L = []
        for h in (2.0 ** -6, -2.0 ** -6):
            setattr(c, n, x + h * u)
            L.append((c.forward()[0].double() * c.dO.double()).sum().item())
        setattr(c, n, x)
        want = (L[0] - L[1]) / 2 ** -5
        have = (g[d].double() * u.double()).sum().item()
        spread = (size[d] * np.abs(np64(u)[0])).sum()
        noise = 2.0 ** -14 * 2.0 ** 5 * np.sqrt((size["o"] * np.abs(np64(c.dO)[0])).size) * (size["o"] * np.abs(np64(c.dO)[0])).max()
        assert abs(have - want) <= 2.0 ** -9 * spread + noise, (n, have, want)


def test_empty_calls():
    p = binding.PromptAttention(0, 5, 2, 1, 64)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o, lse = p.forward(z(0, 5, 2, 64), z(0, 5, 1, 64), z(0, 5, 1, 64), want_lse=True)
    assert o.shape == (0, 5, 2, 64)
    p = binding.PromptAttention(1, 9, 2, 1, 64, seqs=0)
    o = torch.full((1, 9, 2, 64), 3.0).cuda().bfloat16()
    p.forward(z(1, 9, 2, 64), z(1, 9, 1, 64), z(1, 9, 1, 64), cu=torch.zeros(1, dtype=torch.int32).cuda(), o=o)
    assert (o == 3).all()
