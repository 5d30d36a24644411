"""GPU parity of the norm of queries and keys with the position rotation against the fp64
restatement (oracle/attention.py).

Bounds, fixed before the first run.  Forward: an output is r (x_i A + x_p B) with fp32 products and
an fp32 sum of d <= 256 squares, at most 64 roundings of the pair's size: 2^-18 (largest |n| of the
row), plus half a unit of the output type (2^-8 of a bf16 value).  dx likewise, from
r (|g| + |x| r mean |g x r|).  dw is a sum over tokens and heads: 2^-16 of the sum of the terms'
sizes."""
import numpy as np
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding
from oracle import attention as A

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ULP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}

CASES = [  # B, T, Hq, Hk, d, rot, style, io, out, packed
    (1, 1, 1, 1, 128, 128, "halves", "bf16", "bf16", False),
    (3, 1, 16, 4, 128, 128, "halves", "bf16", "bf16", True),
    (2, 37, 16, 4, 128, 64, "pairs", "bf16", "f32", True),
    (2, 129, 5, 3, 96, 32, "halves", "f32", "f32", False),
    (1, 61, 3, 3, 96, 96, "pairs", "f32", "bf16", True),
    (2, 19, 8, 2, 64, 32, "halves", "f32", "f32", True),
    (1, 45, 2, 1, 40, 16, "halves", "bf16", "bf16", False),
    (1, 7, 3, 2, 8, 0, "halves", "f32", "f32", False),
    (2, 33, 7, 1, 256, 256, "halves", "bf16", "bf16", False),
    (1, 50, 4, 4, 256, 144, "pairs", "f32", "f32", True),
    (1, 40, 6, 0, 128, 128, "halves", "bf16", "bf16", False),
    (1, 40, 0, 6, 64, 64, "pairs", "f32", "f32", False),
    (2, 1500, 8, 2, 128, 128, "halves", "bf16", "bf16", True),  # more rows than threads: runs of heads
]


def make(B, T, Hq, Hk, d, rot, style, io, out, packed, seed=0, weights=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = TYPES[io]
    if packed:
        base = (r(B, T, Hq + 2 * Hk, d) * (1 + 3 * torch.rand(B, T, 1, 1, generator=g))).to(dt).cuda()
        q, k = base[:, :, :Hq], base[:, :, Hq:Hq + Hk]
    else:
        q, k = (r(B, T, Hq, d) * 2).to(dt).cuda(), r(B, T, Hk, d).to(dt).cuda()
    wq, wk = (1 + 0.2 * r(d), 1 + 0.2 * r(d)) if weights else (None, None)
    rows = T + 50
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    start = torch.randint(0, 50, (B,), generator=g, dtype=torch.int32)
    pos = torch.randint(0, max(T, 1), (B, T), generator=g, dtype=torch.int32)
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    return dict(q=q, k=k, wq=up(wq), wk=up(wk), cos=ang.cos().float().cuda(), sin=ang.sin().float().cuda(),
                positions=pos.cuda(), start=start.cuda(), dyq=r(B, T, Hq, d).to(dt).cuda(),
                dyk=r(B, T, Hk, d).to(dt).cuda())


def plan(case, grad=None):
    B, T, Hq, Hk, d, rot, style, io, out, packed = case
    return binding.HeadNormRope(B, T, Hq, Hk, d, rot=rot, style=style, io=io, out=out, grad=grad or out,
                                eps=1e-6)


def args(x):
    return [x[n] for n in ("q", "k", "wq", "wk", "cos", "sin")]


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def where(x, use_pos, use_start):
    B, T = x["positions"].shape
    p = x["positions"].cpu().numpy().astype(int) if use_pos else np.arange(T)[None].repeat(B, 0)
    return p + (x["start"].cpu().numpy().astype(int)[:, None] if use_start else 0)


def check(got, ref, bound, what):
    err = np.abs(np64(got) - ref)
    assert np.isfinite(err).all(), what
    assert (err <= bound).all(), f"{what}: worst {np.max(err - bound)} over its bound, error {err.max()}"


def norm_of(x, w):
    x = np64(x)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    return n if w is None else n * np64(w)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("use_pos,use_start", [(False, False), (True, True), (False, True)])
def test_forward(case, use_pos, use_start):
    x = make(*case)
    rot, style, out = case[5], case[6], case[8]
    pos = where(x, use_pos, use_start)
    yq, yk = plan(case).forward(*args(x), positions=x["positions"] if use_pos else None,
                                start=x["start"] if use_start else None)
    for name, w, y in (("q", "wq", yq), ("k", "wk", yk)):
        if y.shape[2] == 0:
            continue
        ref = A.norm_rope(np64(x[name]), np64(x[w]), np64(x["cos"]), np64(x["sin"]), pos, rot, style, 1e-6)
        size = np.abs(norm_of(x[name], x[w])).max(-1, keepdims=True)
        check(y, ref, 2.0 ** -18 * size + ULP[out] * np.abs(ref), name)


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    x = make(*case, seed=3)
    B, T, Hq, Hk, d, rot, style, io, out, packed = case
    pos = where(x, False, True)
    g = plan(case).backward(*args(x), x["dyq"], x["dyk"], start=x["start"])
    for n in ("q", "k"):
        if x[n].shape[2] == 0:
            continue
        w = np64(x["w" + n])
        dx, dw = A.norm_rope_grad(np64(x[n]), w, np64(x["cos"]), np64(x["sin"]), pos, rot, style, 1e-6,
                                  np64(x["dy" + n]))
        xx = np64(x[n])
        r = 1 / np.sqrt((xx * xx).mean(-1, keepdims=True) + 1e-6)
        m = np.abs(np64(x["dy" + n])).max(-1, keepdims=True) * 1.5
        hat = np.abs(xx * r)
        size = r * np.abs(w).max() * m * (1 + hat.max(-1, keepdims=True) * hat.mean(-1, keepdims=True))
        check(g["d" + n], dx, 2.0 ** -17 * size + ULP[out] * np.abs(dx), "d" + n)
        terms = np.abs(A.norm_rope_grad(xx, w, np64(x["cos"]), np64(x["sin"]), pos, rot, style, 1e-6,
                                        np64(x["dy" + n]))[1]) * 0
        # the terms' sizes: |m x r| <= |hat| times the pair's |dy|
        terms = (hat * m).sum((0, 1, 2))
        check(g["dw" + n], dw, 2.0 ** -16 * terms, "dw" + n)


@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_gradient_against_differences(style):
    case = (2, 9, 3, 2, 64, 32, style, "f32", "f32", False)
    x = make(*case, seed=4)
    g = plan(case).backward(*args(x), x["dyq"], x["dyk"], start=x["start"])
    pos = where(x, False, True)
    rng = np.random.default_rng(0)
    for n in ("q", "k"):
        f = lambda a, w: (np64(x["dy" + n]) * A.norm_rope(a, w, np64(x["cos"]), np64(x["sin"]), pos,  # noqa: E731
                                                          32, style, 1e-6)).sum()
        a, w, h = np64(x[n]), np64(x["w" + n]), 1e-5
        for _ in range(4):
            u, v = rng.standard_normal(a.shape), rng.standard_normal(w.shape)
            num = (f(a + h * u, w + h * v) - f(a - h * u, w - h * v)) / (2 * h)
            mine = (np64(g["d" + n]) * u).sum() + (np64(g["dw" + n]) * v).sum()
            size = np.abs(np64(g["d" + n]) * u).sum() + np.abs(np64(g["dw" + n]) * v).sum()
            assert abs(num - mine) <= 2.0 ** -15 * size


def test_without_weights_and_with_one_gradient_left_out():
    case = (2, 21, 4, 2, 128, 128, "halves", "bf16", "bf16", False)
    x = make(*case, weights=False)
    yq, _ = plan(case).forward(*args(x))
    ones = torch.ones(128, device="cuda")
    y1, _ = plan(case).forward(x["q"], x["k"], ones, ones, x["cos"], x["sin"])
    assert torch.equal(yq, y1)
    g = plan(case).backward(*args(x), x["dyq"], x["dyk"])
    assert g["dwq"] is None and g["dwk"] is None
    full = plan(case).backward(x["q"], x["k"], ones, ones, x["cos"], x["sin"], x["dyq"], x["dyk"])
    assert torch.equal(g["dq"], full["dq"]) and torch.equal(g["dk"], full["dk"])


def test_in_place_into_a_packed_tensor_and_on_another_stream():
    case = (2, 70, 16, 4, 128, 128, "halves", "bf16", "bf16", True)
    x = make(*case)
    yq, yk = plan(case).forward(*args(x), start=x["start"])
    y = make(*case)
    rest = y["q"]._base[:, :, 20:].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a, b = plan(case).forward(*args(y), start=y["start"], yq=y["q"], yk=y["k"])
    side.synchronize()
    assert torch.equal(a, yq) and torch.equal(b, yk)
    assert torch.equal(y["q"]._base[:, :, 20:], rest)  # the values beside them are untouched
    # gradients into a packed gradient tensor
    big = torch.full((2, 70, 24, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    z = make(*case)
    p = plan(case)
    ref = p.backward(*args(z), z["dyq"], z["dyk"], start=z["start"])
    out = dict(dq=big[:, :, :16], dk=big[:, :, 16:20], dwq=torch.empty(128, device="cuda"),
               dwk=torch.empty(128, device="cuda"))
    p.backward(*args(z), z["dyq"], z["dyk"], start=z["start"], out=out)
    assert all(torch.equal(out[n], ref[n]) for n in ref) and (big[:, :, 20:] == 7).all()


def test_a_position_outside_the_table_marks_its_token_only():
    case = (1, 30, 4, 2, 128, 64, "halves", "f32", "f32", False)
    x = make(*case)
    pos = torch.arange(30, dtype=torch.int32)[None].cuda()
    pos[0, 7], pos[0, 9] = -1, x["cos"].shape[0]
    good = torch.arange(30, dtype=torch.int32)[None].cuda()
    a, _ = plan(case).forward(*args(x), positions=pos)
    b, _ = plan(case).forward(*args(x), positions=good)
    bad = torch.zeros(30, dtype=torch.bool, device="cuda")
    bad[7] = bad[9] = True
    assert a[0, bad].isnan().all() and torch.equal(a[0, ~bad], b[0, ~bad])
    g = plan(case).backward(*args(x), x["dyq"], x["dyk"], positions=pos)
    assert g["dq"][0, bad].isnan().all() and g["dq"][0, ~bad].isfinite().all() and g["dwq"].isnan().all()


def test_a_nan_stays_in_its_row_and_zeros_are_finite():
    case = (1, 20, 4, 2, 128, 128, "halves", "bf16", "bf16", False)
    x = make(*case)
    x["q"][0, 3, 1, 5] = float("nan")
    x["k"][0, 4, 0] = 0
    yq, yk = plan(case).forward(*args(x))
    assert yq[0, 3, 1].isnan().all() and yq.isnan().sum() == 128
    assert (yk[0, 4, 0] == 0).all()
    g = plan(case).backward(*args(x), x["dyq"], x["dyk"])
    assert g["dk"].isfinite().all() and g["dq"].isnan().sum() == 128


def test_no_tokens_and_repeated_calls():
    x = make(2, 0, 4, 2, 64, 64, "halves", "f32", "f32", False)
    p = plan((2, 0, 4, 2, 64, 64, "halves", "f32", "f32", False))
    assert p.forward(*args(x))[0].shape == (2, 0, 4, 64)
    g = p.backward(*args(x), x["dyq"], x["dyk"])
    assert (g["dwq"] == 0).all() and (g["dwk"] == 0).all()
    case = (3, 301, 8, 2, 64, 64, "pairs", "bf16", "bf16", True)
    x = make(*case)
    p = plan(case)
    a, b = (p.backward(*args(x), x["dyq"], x["dyk"]) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_arguments_are_refused_before_a_launch():
    case = (2, 5, 4, 2, 64, 64, "halves", "bf16", "bf16", False)
    x = make(*case)
    p = plan(case)
    with pytest.raises(ValueError):
        p.forward(x["q"].float(), *args(x)[1:])
    with pytest.raises(ValueError):
        p.forward(x["q"][:, :, :3], *args(x)[1:])
    with pytest.raises(ValueError):
        p.forward(x["q"].transpose(2, 3).contiguous().transpose(2, 3), *args(x)[1:])
    with pytest.raises(ValueError):
        p.forward(*args(x), start=x["start"].long())
    with pytest.raises(binding.DrError):
        binding.HeadNormRope(2, 5, 4, 2, 60)
