"""GPU parity of linear attention with a decay for each head (chunks, gradient, step) against the fp64 restatement;
the bounds are those of mixers.py."""
import numpy as np
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from mixers import OPERAND, SPLIT, TYPES, ULP, Layout, check, np64, tensors
from oracle import mixers as M

pytestmark = pytest.mark.gpu

CASES = [  # lengths, packed, H, dk, dv, states, inside a projection
    ([1], False, 1, 64, 64, False, False),
    ([2, 2], False, 2, 128, 64, True, True),
    ([63], False, 2, 64, 128, True, False),
    ([64, 64, 64], False, 1, 128, 128, False, False),
    ([65], False, 3, 64, 64, True, True),
    ([128], False, 1, 128, 128, True, False),
    ([129, 129], False, 2, 128, 64, False, True),
    ([300], False, 1, 128, 128, True, False),
    ([700], False, 2, 64, 64, True, False),
    ([5, 0, 130, 1, 257, 64, 0], True, 2, 128, 128, True, True),
    ([0, 0, 3], True, 2, 64, 64, True, False),
    ([127, 128, 129, 255, 256, 1], True, 1, 64, 128, True, False),
    ([1] * 70, True, 2, 64, 64, True, False),
    ([17, 40, 3] * 14, True, 1, 128, 64, False, True),
    ([1, 0, 3, 2] * 90, True, 1, 64, 64, True, False),  # many sequences
    ([1, 0, 2] * 100 + [2500], True, 1, 64, 64, True, False),  # and a long one, in segments
]
SMALL = [([70, 3, 0, 129], True, 2, 16, 32, True, True), ([33, 33], False, 3, 32, 16, False, False),
         ([65], False, 2, 16, 16, True, False), ([100], False, 1, 32, 128, True, True), ([90, 1], True, 2, 128, 16, True, False)]


def rates(H):
    """From memories of a few tokens to long ones."""
    return torch.log1p(-torch.exp2(-torch.linspace(1.0, 9.0, H))) if H > 1 else torch.tensor([-0.02])


class Case:
    def __init__(self, case, io, seed=0, rest=11, g=None):
        lens, packed, H, dk, dv, states, inside = case
        self.lay = lay = Layout(lens, packed, rest)
        self.io, self.scale = io, 1.3 * dk ** -0.5
        self.q, self.k, self.v = tensors(lay, (H, H, H), (dk, dk, dv), io, seed, inside)
        self.dO = tensors(lay, (H,), (dv,), io, seed + 1000)[0]
        gen = torch.Generator().manual_seed(seed + 2000)
        self.h0, self.dhT = (3 * torch.randn(len(lens), H, dk, dv, generator=gen).cuda() if states else None for _ in range(2))
        self.g = (rates(H) if g is None else g).float().cuda()
        self.plan = binding.LinearAttention(lay.B, lay.T, H, dk, dv, seqs=lay.seqs, io=io, scale=self.scale)

    def forward(self, **kw):
        return self.plan.forward(self.q, self.k, self.v, self.g, h0=self.h0, cu=self.lay.cu, **kw)

    def backward(self, **kw):
        return self.plan.backward(self.q, self.k, self.v, self.g, self.dO, h0=self.h0, dhT=self.dhT, cu=self.lay.cu, **kw)

    def run(self):
        o, hT = self.forward()
        return dict(o=o, hT=hT, **self.backward(want_dh0=True))

    def oracle(self):
        r = self.lay.rows
        return M.linear(r(self.q), r(self.k), r(self.v), np64(self.g), self.lay.spans, self.scale, np64(self.h0),
                        r(self.dO), np64(self.dhT))

    def check(self, got):
        ref, size = self.oracle()
        fine = 2.0 ** -16 + (max(self.lay.lens) + 128) * 2.0 ** -24
        for n, x in got.items():
            if n in ("hT", "dh0"):
                check(np64(x), ref[n], (SPLIT[self.io] + fine) * size[n], n)
            else:
                check(self.lay.rows(x), ref[n], (OPERAND[self.io] + fine) * size[n] + ULP[self.io] * np.abs(ref[n]), n)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES)
def test_forward_and_backward(case, io):
    c = Case(case, io)
    c.check(c.run())


@pytest.mark.parametrize("case", SMALL)
def test_small_heads(case):
    c = Case(case, "f32", seed=3)
    c.check(c.run())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128), (128, 64)])
def test_longer_sequences(dk, dv, io):
    """Few heads and a long axis: the axis is split."""
    c = Case(([1500, 2600], True, 2, dk, dv, True, False), io, seed=5)
    c.check(c.run())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decays_from_none_to_all(io):
    """g = 0 (plain sums), memories of less than a token, and -inf (nothing of the state is kept)."""
    g = torch.tensor([0.0, -1.0, -60.0, -float("inf")])
    c = Case(([150, 64, 1], True, 4, 64, 64, True, False), io, seed=7, g=g)
    got = c.run()
    assert all(torch.isfinite(x[:, :c.lay.used] if n not in ("hT", "dh0") else x).all() for n, x in got.items())
    c.check(got)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_what_is_not_a_sequence_s_is_left_alone(io):
    case = ([70, 0, 133, 5], True, 2, 64, 128, True, False)
    c, clean = Case(case, io, seed=8), Case(case, io, seed=8)
    want = clean.run()
    lay, used = c.lay, c.lay.used
    for t in (c.q, c.k, c.v, c.dO):
        t[:, used:] = float("nan")
        t[:, 70:203] = float("inf")  # the second sequence with tokens
    o = torch.full_like(c.v, 7.0)
    wide = torch.full((1, lay.T, 2 * 64 + 2 * 64 + 2 * 128 + 8), 5.0, dtype=TYPES[io]).cuda()
    out = dict(dq=wide[:, :, :128].unflatten(2, (2, 64)), dk=wide[:, :, 128:256].unflatten(2, (2, 64)),
               dv=wide[:, :, 256:512].unflatten(2, (2, 128)))
    got = dict(zip(("o", "hT"), c.forward(o=o)))
    got |= c.backward(out=out)
    assert all(got[n].data_ptr() == out[n].data_ptr() for n in out)
    for n, x in got.items():
        if n in ("hT", "dh0"):
            assert all(torch.equal(x[i], want[n][i]) for i in (0, 1, 3)), n
        else:
            assert all(torch.equal(x[:, a:b], want[n][:, a:b]) for a, b in ((0, 70), (203, 208))), n
    assert (o[:, used:] == 7).all() and (wide[:, used:] == 5).all() and (wide[:, :, 512:] == 5).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_offsets_out_of_range_touch_nothing_else(io):
    c = Case(([40, 60, 30], True, 2, 64, 64, True, False), io, seed=9, rest=0)
    o, _ = c.forward()
    cu = torch.tensor([-9, 40, 20, 1 << 30], dtype=torch.int32).cuda()  # 0 .. 40, empty, 20 .. 130
    c.lay.cu = cu
    o2, hT = c.forward()
    g = c.backward()
    torch.cuda.synchronize()
    assert torch.equal(o2[:, :20], o[:, :20]) and torch.equal(hT[1], c.h0[1]) and torch.equal(g["dh0"][1], c.dhT[1])
    assert torch.isfinite(o2).all() and torch.isfinite(g["dk"]).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_in_parts(io):
    """A prompt at once and in parts with the state handed on; gradients of the parts with dh0 handed back."""
    c = Case(([400], False, 2, 128, 64, True, False), io, seed=10)
    ref, size = c.oracle()
    parts, h, cut = [], c.h0, [0, 130, 131, 400]
    for a, b in zip(cut, cut[1:]):
        x = [t[:, a:b].contiguous() for t in (c.q, c.k, c.v)]
        p = binding.LinearAttention(1, b - a, 2, 128, 64, io=io, scale=c.scale)
        parts.append((p, x, h, a, b))
        _, h = p.forward(*x, c.g, h0=h)
    dh = c.dhT
    got = {n: torch.zeros_like(t) for n, t in (("dq", c.q), ("dk", c.k), ("dv", c.v))}
    for p, x, h0, a, b in reversed(parts):
        g = p.backward(*x, c.g, c.dO[:, a:b].contiguous(), h0=h0, dhT=dh)
        dh = g["dh0"]
        for n in got:
            got[n][:, a:b] = g[n]
    c.check(dict(hT=h, dh0=dh, **got))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_same_bits_every_time_and_on_two_streams(io):
    cs = [Case(([513, 200, 31], True, 4, 128, 128, True, True), io, seed=s) for s in (11, 12)]
    plan, used = cs[0].plan, cs[0].lay.used
    for c in cs:
        c.plan = plan
    alone = [c.run() for c in cs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cs], [[], []]
    for _ in range(10):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run())
    torch.cuda.synchronize()
    cut = lambda n, x: x if n in ("hT", "dh0") else x[:, :used]  # noqa: E731
    for i in (0, 1):
        assert all(torch.equal(cut(n, x[n]), cut(n, alone[i][n])) for x in got[i] for n in x)


def test_captured_call_takes_new_lengths():
    c = Case(([200, 100, 36], True, 2, 128, 128, True, False), "bf16", seed=13, rest=0)
    cu = c.lay.cu = c.lay.cu.clone()
    o, hT = torch.zeros_like(c.v), torch.zeros_like(c.h0)
    out = dict(dq=torch.zeros_like(c.q), dk=torch.zeros_like(c.k), dv=torch.zeros_like(c.v), dh0=torch.zeros_like(c.h0))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.forward(o=o, hT=hT), c.backward(out=out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.forward(o=o, hT=hT), c.backward(out=out)
    torch.cuda.synchronize()
    for lens in ([200, 100, 36], [1, 335, 0], [0, 0, 336]):
        d = Case((lens, True, 2, 128, 128, True, False), "bf16", seed=13, rest=0)
        cu.copy_(d.lay.cu)
        graph.replay()
        torch.cuda.synchronize()
        want = d.run()
        assert torch.equal(o, want["o"]) and torch.equal(hT, want["hT"])
        assert all(torch.equal(out[n], want[n]) for n in out)


def test_gradient_against_differences():
    """fp32.  L is linear in each of q, k, v and h0, so differences with h = 2^-2 are exact but for rounding: 2^-16 of
    the sums of the terms' sizes (2^-18 of L's terms for each side, over h)."""
    c = Case(([90, 41], True, 2, 32, 64, True, False), "f32", seed=14, rest=0)
    got = c.run()
    _, size = c.oracle()
    noise = 2.0 ** -14 * ((size["o"] * np.abs(c.lay.rows(c.dO))).sum() + (size["hT"] * np.abs(np64(c.dhT))).sum())
    gen = torch.Generator().manual_seed(15)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h0", "dh0")):
        x = getattr(c, n)
        u = torch.randn(x.shape, generator=gen).cuda()
        L = []
        for h in (0.25, -0.25):
            setattr(c, n, x + h * u)
            o, hT = c.forward()
            L.append(((o.double() * c.dO.double()).sum() + (hT.double() * c.dhT.double()).sum()).item())
        setattr(c, n, x)
        assert abs((L[0] - L[1]) * 2 - (got[d].double() * u.double()).sum().item()) <= noise, n


# ------------------------------------------------------------------------------- the step
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv,inside", [(1, 1, 1, 64, 64, False), (3, 1, 2, 128, 128, True), (2, 5, 3, 128, 64, True),
                                                (2, 8, 2, 16, 16, False), (1, 9, 2, 16, 128, False), (2, 17, 1, 32, 64, True),
                                                (5, 2, 4, 64, 32, False), (1, 1, 2, 128, 16, False)])
def test_step(B, T, H, dk, dv, inside, io):
    lay = Layout([T] * B, False)
    q, k, v = tensors(lay, (H, H, H), (dk, dk, dv), io, 20, inside)
    gen = torch.Generator().manual_seed(21)
    state = 2 * torch.randn(B, H, dk, dv, generator=gen).cuda()
    g = rates(H).cuda()
    ref, size = M.linear(lay.rows(q), lay.rows(k), lay.rows(v), np64(g), lay.spans, 0.7, np64(state))
    plan = binding.LinearAttention(B, T, H, dk, dv, io=io, scale=0.7)
    o = plan.step(q, k, v, g, state)
    fine = 2.0 ** -17 + (T + 128) * 2.0 ** -24
    check(np64(state), ref["hT"], fine * size["hT"], "state")
    check(lay.rows(o), ref["o"], fine * size["o"] + ULP[io] * np.abs(ref["o"]), "o")


def test_prompt_then_steps():
    """A prompt in chunks, then token by token, against the whole at once."""
    c = Case(([140, 140], False, 2, 128, 128, True, False), "bf16", seed=22)
    p = binding.LinearAttention(2, 100, 2, 128, 128, scale=c.scale)
    o, h = p.forward(*(t[:, :100].contiguous() for t in (c.q, c.k, c.v)), c.g, h0=c.h0)
    one, outs = binding.LinearAttention(2, 1, 2, 128, 128, scale=c.scale), [o]
    for t in range(100, 140):
        outs.append(one.step(*(x[:, t:t + 1].contiguous() for x in (c.q, c.k, c.v)), c.g, h))
    c.check(dict(o=torch.cat(outs, 1), hT=h))


def test_empty_calls():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    g = torch.zeros(2).cuda()
    h0 = torch.randn(3, 2, 64, 64).cuda()
    p = binding.LinearAttention(3, 0, 2, 64, 64)
    o, hT = p.forward(z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64), g, h0=h0)
    assert o.shape == (3, 0, 2, 64) and torch.equal(hT, h0)
    gr = p.backward(z(3, 0, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64), g, z(3, 0, 2, 64), dhT=h0)
    assert torch.equal(gr["dh0"], h0)
    p = binding.LinearAttention(0, 4, 2, 64, 64)
    o, hT = p.forward(z(0, 4, 2, 64), z(0, 4, 2, 64), z(0, 4, 2, 64), g)
    assert hT.shape == (0, 2, 64, 64)
