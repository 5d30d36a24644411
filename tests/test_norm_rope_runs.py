"""GPU parity of the norm with rotation where a group of threads takes runs of 2, 4 or 16 heads of a token: head
counts that fill no run, several runs of queries, ragged token counts.  Bounds: those of tests/test_norm_rope.py,
where dw is a chain of at most 100 terms in a thread, 16 groups, 19 parts and 32 sums: below 2^-16 of the terms'
sizes.  The reference is the definition in 64 bits."""
import pytest
import torch

from test_norm_rope import ULP, args, make, plan

pytestmark = pytest.mark.gpu

BLOCKS = 152 * 4  # of the gradient
CASES = [  # heads of a run; B, T, Hq, Hk, d, rot, style, io, out, packed
    (2, (3, 701, 18, 3, 128, 128, "halves", "bf16", "bf16", True)),
    (2, (1, 3907, 18, 3, 64, 32, "pairs", "f32", "f32", False)),
    (4, (5, 1009, 18, 3, 128, 64, "pairs", "bf16", "bf16", True)),
    (4, (1, 1201, 33, 3, 256, 144, "halves", "f32", "f32", False)),
    (4, (1, 6007, 18, 3, 96, 96, "halves", "f32", "bf16", True)),
    (16, (7, 2203, 18, 3, 128, 128, "halves", "bf16", "bf16", True)),
    (16, (3, 1501, 33, 3, 256, 256, "pairs", "f32", "f32", False)),
    (16, (3, 9901, 18, 3, 64, 32, "halves", "bf16", "f32", False)),
    (16, (1, 18013, 18, 0, 128, 128, "pairs", "bf16", "bf16", False)),
    (16, (1, 21001, 0, 21, 128, 96, "pairs", "f32", "f32", False)),
]


def lanes(d):
    return 4 if d <= 32 else 8 if d <= 64 else 16 if d <= 128 else 32


def blocks(Hq, Hk, run, tokens, d):
    """Blocks of the gradient's kernel for runs of that many heads, by the rule that shares them out."""
    tiles = -(-tokens // (128 // lanes(d)))
    share = lambda heads: min(max(1, BLOCKS * heads // (Hq + Hk)), tiles)  # noqa: E731
    n = 0
    for H in (Hq, Hk):
        runs = -(-H // run)
        n += (runs - 1) * share(run) + share(H - (runs - 1) * run) if runs else 0
    return n


@pytest.mark.parametrize("run,case", CASES)
def test_the_cases_take_the_runs_they_are_meant_for(run, case):
    B, T, Hq, Hk, d = case[:5]
    rows, groups = B * T * (Hq + Hk), 152 * 2048 // lanes(d)
    assert run == (1 if rows < 2 * groups else 2 if rows < 4 * groups else 4 if rows < 16 * groups else 16)
    p = plan(case)  # a part of dw for each block
    assert int(p._lib.dr_norm_rope_workspace_bytes(p._ref)) == 4 * d * blocks(Hq, Hk, run, B * T, d)


def rotate(n, cos, sin, rot, style, back=False):
    y = n.clone()
    if rot:
        c, s = cos[:, :, None], -sin[:, :, None] if back else sin[:, :, None]
        i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if style == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
        y[..., i] = n[..., i] * c - n[..., j] * s
        y[..., j] = n[..., j] * c + n[..., i] * s
    return y


def angles(x, T):
    pos = x["start"].long()[:, None] + torch.arange(T, device="cuda")
    return x["cos"].double()[pos], x["sin"].double()[pos]


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert err.isfinite().all(), what
    assert (err <= bound).all(), f"{what}: worst {float((err - bound).max())} over its bound, error {float(err.max())}"


@pytest.mark.parametrize("run,case", CASES)
def test_forward(run, case):
    x = make(*case, seed=51)
    T, rot, style, out = case[1], case[5], case[6], case[8]
    cos, sin = angles(x, T)
    yq, yk = plan(case).forward(*args(x), start=x["start"])
    for n, y in (("q", yq), ("k", yk)):
        if y.shape[2] == 0:
            continue
        a = x[n].double()
        nw = a / (a.square().mean(-1, keepdim=True) + 1e-6).sqrt() * x["w" + n].double()
        ref = rotate(nw, cos, sin, rot, style)
        within(y, ref, 2.0 ** -18 * nw.abs().amax(-1, keepdim=True) + ULP[out] * ref.abs(), n)


@pytest.mark.parametrize("run,case", CASES)
def test_backward(run, case):
    x = make(*case, seed=52)
    T, d, rot, style, out = case[1], case[4], case[5], case[6], case[8]
    cos, sin = angles(x, T)
    p = plan(case)
    g = p.backward(*args(x), x["dyq"], x["dyk"], start=x["start"])
    again = p.backward(*args(x), x["dyq"], x["dyk"], start=x["start"])
    assert all(torch.equal(g[n], again[n]) for n in g)
    for n in ("q", "k"):
        if x[n].shape[2] == 0:
            continue
        a, w, dy = x[n].double(), x["w" + n].double(), x["dy" + n].double()
        r = 1 / (a.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        m = rotate(dy, cos, sin, rot, style, back=True)
        dx = r * m * w - a * r ** 3 * (m * w * a).sum(-1, keepdim=True) / d
        hat, top = (a * r).abs(), dy.abs().amax(-1, keepdim=True) * 1.5
        size = r * w.abs().max() * top * (1 + hat.amax(-1, keepdim=True) * hat.mean(-1, keepdim=True))
        within(g["d" + n], dx, 2.0 ** -17 * size + ULP[out] * dx.abs(), "d" + n)
        within(g["dw" + n], (m * a * r).sum((0, 1, 2)), 2.0 ** -16 * (hat * top).sum((0, 1, 2)), "dw" + n)
