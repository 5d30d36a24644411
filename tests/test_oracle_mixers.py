"""Pins of the fp64 restatement of the token mixers beside the delta rule (oracle/mixers.py), on the CPU."""
import numpy as np
import pytest

from oracle import mixers as M

SPANS = [(0, 4), (4, 4), (4, 11), (11, 12)]


def differences(f, x, h=1e-5):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        was = x[i]
        x[i] = was + h
        up = f()
        x[i] = was - h
        g[i] = (up - f()) / (2 * h)
        x[i] = was
    return g


@pytest.mark.parametrize("window", [0, 3])
def test_attention_gradient_against_differences(window):
    rng = np.random.default_rng(0)
    q, k, v, dO = (rng.standard_normal((12, h, 3)) for h in (4, 2, 2, 4))
    f = lambda: (dO * M.attention(q, k, v, SPANS, 0.7, window)[0]["o"]).sum()  # noqa: E731
    got, _ = M.attention(q, k, v, SPANS, 0.7, window, dO)
    for x, n in ((q, "dq"), (k, "dk"), (v, "dv")):
        assert np.allclose(differences(f, x), got[n], atol=1e-8), n


def test_attention_of_worked_rows():
    # equal keys: the mean of the values seen; a window of one: the value itself
    q, k = np.ones((3, 1, 2)), np.ones((3, 1, 2))
    v = np.array([[1.0, 0.0], [3.0, 2.0], [8.0, 4.0]])[:, None]
    o = M.attention(q, k, v, [(0, 3)], 1.0, 0)[0]
    assert np.allclose(o["o"][:, 0], [[1, 0], [2, 1], [4, 2]]) and np.allclose(o["lse"][:, 0], 2 + np.log([1, 2, 3]))
    assert np.allclose(M.attention(q, k, v, [(0, 3)], 1.0, 1)[0]["o"], v)


def test_linear_gradient_against_differences():
    rng = np.random.default_rng(1)
    q, k, v, dO = (rng.standard_normal((12, 2, d)) for d in (3, 3, 2, 2))
    h0, dhT = rng.standard_normal((2, 4, 2, 3, 2))
    g = np.array([-0.1, -1.3])

    def f():
        o = M.linear(q, k, v, g, SPANS, 0.7, h0)[0]
        return (dO * o["o"]).sum() + (dhT * o["hT"]).sum()

    got, _ = M.linear(q, k, v, g, SPANS, 0.7, h0, dO, dhT)
    for x, n in ((q, "dq"), (k, "dk"), (v, "dv"), (h0, "dh0")):
        assert np.allclose(differences(f, x), got[n], atol=1e-8), n
    assert np.array_equal(got["hT"][1], h0[1]) and np.array_equal(got["dh0"][1], dhT[1])


def test_linear_of_worked_tokens():
    # one channel, decay 1/2: S = 1, 0.5 + 2 = 2.5, 1.25 + 4 = 5.25
    one = np.ones((3, 1, 1))
    v = np.array([1.0, 2.0, 4.0])[:, None, None]
    got, _ = M.linear(2 * one, one, v, np.log([0.5]), [(0, 3)], 3.0)
    assert np.allclose(got["o"][:, 0, 0], [6, 15, 31.5]) and np.allclose(got["hT"], 5.25)
