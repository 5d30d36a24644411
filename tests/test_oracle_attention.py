"""Pins of the attention layer's fp64 restatement (oracle/attention.py), on the CPU."""
import numpy as np
import pytest
import torch

from oracle import attention as A


def tables(rows, rot):
    ang = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.cos(ang), np.sin(ang)


def test_rotation_keeps_lengths_and_depends_on_distance_only():
    rng = np.random.default_rng(0)
    for style in ("halves", "pairs"):
        cos, sin = tables(64, 32)
        x, y = rng.standard_normal((2, 1, 1, 1, 32))
        at = lambda z, p: A.norm_rope(z, None, cos, sin, np.array([[p]]), 32, style, 0.0)  # noqa: E731
        assert np.allclose((at(x, 9) ** 2).sum(), 32)
        assert np.allclose((at(x, 40) * at(y, 33)).sum(), (at(x, 7) * at(y, 0)).sum())


def test_rotation_of_a_worked_pair():
    # one pair (3, 4) of equal mean square 12.5: n = x / sqrt(12.5); a quarter turn gives (-n2, n1)
    x = np.zeros((1, 1, 1, 2)) + [3.0, 4.0]
    y = A.norm_rope(x, None, np.array([[0.0]]), np.array([[1.0]]), np.zeros((1, 1), int), 2, "halves", 0.0)
    assert np.allclose(y[0, 0, 0], np.array([-4.0, 3.0]) / np.sqrt(12.5))


@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("rot", [0, 16, 32])
def test_gradient_against_differences(style, rot):
    rng = np.random.default_rng(1)
    cos, sin = tables(20, rot)
    x, dy = rng.standard_normal((2, 2, 3, 2, 32))
    w, pos = rng.standard_normal(32), rng.integers(0, 20, (2, 3))
    f = lambda x, w: (dy * A.norm_rope(x, w, cos, sin, pos, rot, style, 1e-3)).sum()  # noqa: E731
    dx, dw = A.norm_rope_grad(x, w, cos, sin, pos, rot, style, 1e-3, dy)
    h = 1e-5
    for _ in range(40):
        at = tuple(rng.integers(0, s) for s in x.shape)
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for c in range(32):
        e = np.zeros(32)
        e[c] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[c]) < 1e-7


def test_codes_match_torch_and_round_trip():
    x = np.concatenate([np.linspace(-460, 460, 20001), np.linspace(-0.03, 0.03, 4001)]).astype(np.float32)
    mine = A.to_code(x, "e4m3")
    ref = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    same = (mine == ref) | (((mine & 0x7f) == 0) & ((ref & 0x7f) == 0))
    assert same.all()
    codes = np.array([c for c in range(256) if c & 0x7f != 0x7f], np.uint8)
    assert (A.to_code(A.e4m3_value(codes), "e4m3") == codes).all()
    assert list(A.to_code([0.5, 1.5, -2.5, 300, -300], "i8").view(np.int8)) == [0, 2, -2, 127, -127]


@pytest.mark.parametrize("code", ["i8", "e4m3"])
def test_append_in_one_call_or_in_two(code):
    """Values stay within a step of what was written however the tokens are split; pages that a
    sequence does not own are untouched."""
    rng = np.random.default_rng(2)
    page, H, d, T = 16, 2, 8, 41
    x = (rng.standard_normal((1, T, H, d)) * np.linspace(0.1, 4, T)[:, None, None]).astype(np.float32)
    table = np.array([[5, 1, 3]])
    for cut in (0, 7, 16, 33):
        codes = np.full((6, H, page, d), 77, np.uint8)
        scale = np.full((6, H), 9.0, np.float32)
        A.cache_write(codes, scale, x[:, :cut], table, [0], [cut], code)
        A.cache_write(codes, scale, x[:, cut:], table, [cut], [T - cut], code)
        assert (codes[[0, 2, 4]] == 77).all() and (scale[[0, 2, 4]] == 9).all()
        back = A.cache_values(codes, scale, table[0], T, code)
        s = scale[table[0]].repeat(page, 0)[:T, :, None]
        # one rounding, a second one where the scale grew: half a step each
        bound = s * 1.0 if code == "i8" else np.maximum(np.abs(x[0]) * 2.0 ** -3, s * 2.0 ** -9)
        assert (np.abs(back - x[0]) <= bound * 1.001).all()
        if cut in (0, 16):
            assert (np.abs(back - x[0]) <= 0.5 * bound * 1.001).all()


def test_a_value_that_is_not_finite_marks_its_page():
    x = np.ones((1, 20, 1, 8), np.float32)
    x[0, 3, 0, 2] = np.inf
    codes, scale = np.zeros((2, 1, 16, 8), np.uint8), np.zeros((2, 1), np.float32)
    A.cache_write(codes, scale, x, np.array([[1, 0]]), [0], [20], "i8")
    back = A.cache_values(codes, scale, [1, 0], 20, "i8")
    assert np.isnan(back[:16]).all() and np.allclose(back[16:], 1)


def test_attention_of_one_position_is_its_value_and_windows_nest():
    rng = np.random.default_rng(3)
    H, d, page, n = 2, 8, 16, 40
    codes = rng.integers(0, 120, (2, 3, H, page, d)).astype(np.uint8)
    scale = rng.uniform(0.01, 0.02, (2, 3, H)).astype(np.float32)
    table = np.array([[2, 0, 1]])
    q = rng.standard_normal((1, 3, 4, d))
    run = lambda lens, T, w: A.attention(q[:, :T], codes[0], scale[0], codes[1], scale[1], table,  # noqa: E731
                                         [lens], [T], "i8", 0.3, w)
    v = A.cache_values(codes[1], scale[1], table[0], n, "i8")
    o, lse, *_ = run(0, 1, 0)
    assert np.allclose(o[0, 0], v[0].repeat(2, 0))
    o, lse, *_ = run(n - 3, 3, 1)
    assert np.allclose(o[0], v[n - 3:].repeat(2, 1))
    a, b = run(n - 3, 3, 0), run(n - 3, 3, n)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
