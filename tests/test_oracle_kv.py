"""Pins of oracle/kv.py: hand-worked rotations and attentions, closed forms, and mistakes that must show."""
import math

import numpy as np

from oracle import hadamard as H, kv as K


def test_rotation_by_hand():
    c, s = np.array([0.6, 0.0]), np.array([0.8, 1.0])
    x = np.array([1.0, 2.0, 3.0, 4.0, 9.0])
    assert np.allclose(K.rotate(x, c, s), [0.6 - 2.4, -4.0, 1.8 + 0.8, 2.0, 9.0])
    assert np.allclose(K.rotate(x, c, s, True), [0.6 - 1.6, 1.2 + 0.8, -4.0, 3.0, 9.0])


def test_rotation_keeps_products_of_relative_positions():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 8))
    w = 0.3 ** np.arange(4)
    def at(x, p, inter):
        return K.rotate(x, np.cos(p * w), np.sin(p * w), inter)
    for inter in (False, True):
        assert math.isclose(at(q, 9, inter) @ at(k, 4, inter), at(q, 25, inter) @ at(k, 20, inter), rel_tol=1e-12)
        assert not math.isclose(at(q, 9, inter) @ at(k, 4, inter), at(q, 9, inter) @ at(k, 5, inter), rel_tol=1e-6)


def test_attention_by_hand():
    q = np.array([[[1.0, 0.0]]])
    k = np.array([[[0.0, 5.0]], [[math.log(3.0), 1.0]]])
    v = np.array([[[4.0, 0.0]], [[0.0, 8.0]]])
    out, lse = K.attention(q, k, v, 1.0)
    assert np.allclose(out, [[[1.0, 6.0]]]) and np.allclose(lse, [[math.log(4.0)]])
    out, lse = K.attention(q, k, v, 0.0)
    assert np.allclose(out, [[[2.0, 4.0]]]) and np.allclose(lse, [[math.log(2.0)]])


def test_masks():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal(s) for s in ((3, 4, 8), (5, 2, 8), (5, 2, 8)))
    out, _ = K.attention(q, k, v, 1.0)
    # the first query of a chunk of 3 over 5 keys sees keys 0..2, and what later keys hold does not matter
    k2, v2 = k.copy(), v.copy()
    k2[3:], v2[3:] = np.nan, np.inf
    assert np.array_equal(K.attention(q, k2, v2, 1.0)[0][0], out[0])
    # grouped heads: heads 0, 1 read key head 0
    assert np.allclose(out[:, 2:], K.attention(q[:, 2:], k[:, 1:], v[:, 1:], 1.0)[0])
    # a window of one sees the token itself
    assert np.allclose(K.attention(q, k, v, 1.0, window=1)[0][:, 0], v[2:, 0])
    # more queries than keys: the first ones see nothing
    out, lse = K.attention(q, k[:2], v[:2], 1.0)
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all() and np.allclose(out[1, 0], v[0, 0])
    assert (K.attention(q, k[:0], v[:0], 1.0, causal=False)[0] == 0).all()


def test_rotated_basis():
    """(Hn S q).(Hn S k) = q.k, and the values come back through S Hn."""
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal(s) for s in ((4, 2, 64), (9, 2, 64), (9, 2, 64)))
    s = rng.choice([-1.0, 1.0], 64)
    r = lambda x: H.rht(x.reshape(-1, 64), s).reshape(x.shape)  # noqa: E731
    a, la = K.attention(q, k, v, 0.3)
    b, lb = K.attention(r(q), r(k), r(v), 0.3)
    assert np.allclose(H.irht(b.reshape(-1, 64), s).reshape(a.shape), a) and np.allclose(la, lb)
