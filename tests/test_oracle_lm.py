"""The oracle's norms and log probabilities: worked values, and gradients against differences."""
import numpy as np
import pytest

from oracle import lm


def differences(f, x, eps=1e-6):
    g = np.zeros(x.shape)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


def test_norm_worked():
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(lm.norm_rope(x, np.array([1.0, 2.0]), 0.0), x / np.sqrt(12.5) * [1, 2])
    # a quarter turn: (a, b) -> (-b, a)
    y = lm.norm_rope(x, np.ones(2), 0.0, np.zeros((1, 1)), np.ones((1, 1)))
    assert np.allclose(y, np.array([[[-4.0, 3.0]]]) / np.sqrt(12.5))


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_gradient(per_head, inter):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 2, 6)), rng.standard_normal((3, 2, 6))
    w = rng.standard_normal((2, 6) if per_head else 6)
    ang = rng.standard_normal((3, 2))
    cos, sin = np.cos(ang), np.sin(ang)
    f = lambda x, w: (lm.norm_rope(x, w, 1e-2, cos, sin, inter) * dy).sum()
    dx, dw = lm.norm_rope_backward(dy, x, w, 1e-2, cos, sin, inter)
    # central differences: the third derivative's term 1e-12, rounding 1e-16 / 1e-6
    assert np.abs(dx - differences(lambda a: f(a, w), x)).max() < 1e-8
    assert np.abs(dw - differences(lambda a: f(x, a), w)).max() < 1e-8


def test_logprobs_worked():
    x = np.log(np.array([[0.5, 0.25, 0.125, 0.125]]))
    r = lm.logprobs(x + 3, np.array([1]), top=4)
    assert np.allclose(r["lse"], 3) and np.allclose(r["logprob"], np.log(0.25))
    assert np.allclose(r["entropy"], 1.75 * np.log(2))
    assert r["top_id"].tolist() == [[0, 1, 2, 3]]


def test_logprobs_edges():
    x = np.array([[-np.inf, 1.0, 1.0], [-np.inf] * 3, [0.0, np.nan, 2.0]])
    r = lm.logprobs(x, np.array([0, 1, -1]), top=2)
    assert r["logprob"][0] == -np.inf and np.isclose(r["entropy"][0], np.log(2))
    assert r["top_id"].tolist() == [[1, 2], [0, 1], [2, 0]]
    assert r["lse"][1] == r["logprob"][1] == -np.inf and r["entropy"][1] == 0
    assert np.isnan(r["lse"][2]) and r["logprob"][2] == 0


@pytest.mark.parametrize("scale", [1.0, 0.6])
def test_logprobs_gradient(scale):
    rng = np.random.default_rng(2)
    x, g, h = rng.standard_normal((4, 9)), rng.standard_normal(4), rng.standard_normal(4)
    t = np.array([3, 0, -1, 8])

    def f(x):
        r = lm.logprobs(x, t, scale)
        return (g * r["logprob"] + h * r["entropy"]).sum()
    assert np.abs(lm.logprobs_backward(x, t, g, h, scale) - differences(f, x)).max() < 1e-8
    x[:, 5] = -np.inf
    d = lm.logprobs_backward(x, t, g, h, scale)
    assert np.isfinite(d).all() and (d[:, 5] == 0).all()


def test_sinks_by_hand():
    """Position 5 under a window of 2 with 3 sinks sees 0, 1, 2, 4 and 5; equal scores: the mean of their values."""
    from oracle import kv as K
    v = np.arange(6.0)[:, None, None] ** 2
    out, lse = K.attention(np.zeros((1, 1, 1)), np.ones((6, 1, 1)), v, 1.0, True, 2, 3)
    assert np.isclose(out[0, 0, 0], (0 + 1 + 4 + 16 + 25) / 5) and np.isclose(lse[0, 0], np.log(5))
    assert [j for j in range(6) if K.sees(6, 4, 0, j, True, 1, 2)] == [0, 1, 2]
    assert [j for j in range(6) if K.sees(6, 4, 0, j, False, 1, 1)] == [0, 2, 3, 4, 5]
