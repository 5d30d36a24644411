"""Gradients of both token mixers (fp32) against differences of the forward pass, along directions in which the terms do
not cancel: the gradient itself by the fp64 restatement, and random halves of its entries.

<gradient, u> is compared with D, the central difference of L along u.  Attention: D = (4 D(1/2) - D(1)) / 3 of the steps
1 and 1/2, whose error of second order cancels; linear attention: L is linear along u, one step is exact.
The bound is arithmetic on the inputs, nothing in it comes from the results that are tested:
  what D of the restatement, of the same rounded inputs, is off from <gradient, u> by; and
  the errors that mixers.py and the two test files allow o, hT and the gradient, each summed with all signs against it:
  a value e of L's error becomes (4 (e + e) + (e + e) / 2) / 3 in D, or (e + e) / 2 for one step.
It has to stay below a twentieth of <gradient, u>, or the comparison would say nothing."""
import numpy as np
import pytest
import torch

from mixers import ULP, np64
from oracle import mixers as M
from test_linear_attn import Case as Linear
from test_prompt_attn import Case as Prompt

pytestmark = pytest.mark.gpu


def halves(ref, seed):
    """The gradient, and three times a random half of it."""
    rng = np.random.RandomState(seed)
    return [ref] + [ref * rng.randint(0, 2, ref.shape) for _ in range(3)]


def moved(x, u, h):
    """x + h u as the fp32 tensor that the call gets."""
    return (x.double() + h * torch.tensor(u, device=x.device).reshape(x.shape)).float()


def compare(have, want, bound, exact, what):
    assert bound <= abs(exact) / 20, f"{what}: the bound {bound:.3g} is too wide for {exact:.3g}"
    assert abs(have - want) <= bound, f"{what}: {have:.6g}, by differences {want:.6g}, bound {bound:.2g}"


@pytest.mark.parametrize("case", [([90, 41], True, 4, 2, 64, 50, False), ([60, 0, 33], True, 3, 1, 128, 0, False)])
def test_attention(case):
    c = Prompt(case, "f32", seed=14, rest=0, spread=0.35)
    o, lse = c.forward()
    got = c.backward(o, lse)
    ref, size = c.oracle()
    dO, r = c.lay.rows(c.dO), c.lay.rows
    fine = lambda s: 2.0 ** -16 * (1 + s["lse"].max()) + max(c.lay.lens) * 2.0 ** -24  # noqa: E731

    def loss():
        """L of the kernel, L of the restatement, and how far the first may be off."""
        want, s = M.attention(r(c.q), r(c.k), r(c.v), c.lay.spans, c.scale, c.window)
        off = fine(s) * s["o"] + ULP["f32"] * np.abs(want["o"])
        return np.array([(r(c.forward()[0]) * dO).sum(), (want["o"] * dO).sum(), (off * np.abs(dO)).sum()])

    for n, d, times in (("q", "dq", 6), ("k", "dk", 6), ("v", "dv", 2)):
        x = getattr(c, n)
        allowed = times * fine(size) * size[d] + ULP["f32"] * np.abs(ref[d])
        for i, u in enumerate(halves(ref[d], 15)):
            # a step moves a row by its norm at most: scores of below two change by about as much
            u = u * (np.linalg.norm(r(x), axis=-1) / np.maximum(np.linalg.norm(u, axis=-1), 1e-30)).min()
            at = {}
            for h in (1.0, -1.0, 0.5, -0.5):
                setattr(c, n, moved(x, u, h))
                at[h] = loss()
            setattr(c, n, x)
            D, want = ((4 * (at[0.5][j] - at[-0.5][j]) - (at[1.0][j] - at[-1.0][j]) / 2) / 3 for j in (0, 1))
            exact = (ref[d] * u).sum()
            noise = (4 * (at[0.5][2] + at[-0.5][2]) + (at[1.0][2] + at[-1.0][2]) / 2) / 3
            compare((r(got[d]) * u).sum(), D, abs(want - exact) + noise + (allowed * np.abs(u)).sum(), exact, f"{d} {i}")


@pytest.mark.parametrize("case", [([90, 41], True, 2, 32, 64, True, False), ([130, 130], False, 1, 128, 16, True, False)])
def test_linear_attention(case):
    c = Linear(case, "f32", seed=14, rest=0)
    got = c.run()
    ref, size = c.oracle()
    dO, dhT, r = c.lay.rows(c.dO), np64(c.dhT), c.lay.rows
    fine = 2.0 ** -16 + (max(c.lay.lens) + 128) * 2.0 ** -24

    def loss():
        want, s = M.linear(r(c.q), r(c.k), r(c.v), np64(c.g), c.lay.spans, c.scale, np64(c.h0))
        o, hT = c.forward()
        off = (fine * s["o"] + ULP["f32"] * np.abs(want["o"])) * np.abs(dO)
        return np.array([(r(o) * dO).sum() + (np64(hT) * dhT).sum(), (want["o"] * dO).sum() + (want["hT"] * dhT).sum(),
                         off.sum() + (fine * s["hT"] * np.abs(dhT)).sum()])

    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h0", "dh0")):
        x = getattr(c, n)
        value = np64 if n == "h0" else r
        allowed = fine * size[d] + (0 if n == "h0" else ULP["f32"] * np.abs(ref[d]))
        for i, u in enumerate(halves(ref[d], 15)):
            u = u * (np.linalg.norm(value(x)) / np.linalg.norm(u))
            setattr(c, n, moved(x, u, 1.0))
            up = loss()
            setattr(c, n, moved(x, u, -1.0))
            down = loss()
            setattr(c, n, x)
            D, want = ((up[j] - down[j]) / 2 for j in (0, 1))
            exact = (ref[d] * u).sum()
            bound = abs(want - exact) + (up[2] + down[2]) / 2 + (allowed * np.abs(u)).sum()
            compare((value(got[d]) * u).sum(), D, bound, exact, f"{d} {i}")
