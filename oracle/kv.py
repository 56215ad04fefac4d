"""Paged key/value cache and its attention, in fp64, as the definitions.

Rotary positions: a pair (a, b) of a head vector at position p becomes
(a cos - b sin, b cos + a sin) with the given table rows; pairs (i, i + r / 2)
or, interleaved, (2i, 2i + 1) of the first r coordinates.

Attention: query i of a chunk of n over kv keys sits at p = kv - n + i and sees
key j < kv when (not causal or j <= p) and (window == 0 or j > p - window or
j < sinks);
out = sum_j softmax_j(scale q.k_j) v_j over the keys it sees, 0 if none, and
lse = log sum_j exp(scale q.k_j), -inf if none.  A key that is not seen takes
no part at all, whatever it holds.
"""
import numpy as np


def rotate(x, cos, sin, interleaved=False):
    """x [..., D]; cos, sin [..., r / 2], one row per leading index."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    h = cos.shape[-1]
    for i in range(h):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y[..., a] = x[..., a] * cos[..., i] - x[..., b] * sin[..., i]
        y[..., b] = x[..., b] * cos[..., i] + x[..., a] * sin[..., i]
    return y


def sees(kv, n, i, j, causal, window, sinks=0):
    p = kv - n + i
    return j < kv and (not causal or j <= p) and (window == 0 or j > p - window or j < sinks)


def attention(q, k, v, scale, causal=True, window=0, sinks=0):
    """q [n, H, D], k and v [kv, G, D]; returns out [n, H, D], lse [n, H]."""
    n, heads, d = q.shape
    kv, kvh = k.shape[:2]
    out, lse = np.zeros((n, heads, d)), np.full((n, heads), -np.inf)
    for i in range(n):
        js = [j for j in range(kv) if sees(kv, n, i, j, causal, window, sinks)]
        if not js:
            continue
        for h in range(heads):
            g = h // (heads // kvh)
            s = scale * (k[js, g] @ q[i, h])
            top = s.max()
            p = np.exp(s - top)
            out[i, h] = (p @ v[js, g]) / p.sum()
            lse[i, h] = top + np.log(p.sum())
    return out, lse
