"""Norms of head vectors with their gradients, and log probabilities of
logits with theirs, in fp64, as the definitions.

Norm and rotation: y = R(position) (x r w), r = (mean x^2 + eps)^-1/2.

Log probabilities: z = scale x, p = softmax(z), logprob = log p[target] (0
without a target in the vocabulary), entropy = -sum p log p with 0 log 0 = 0,
the top tokens in the order of falling x, ties by index, a NaN like -inf.  A
row of only -inf: logprob = lse = -inf, entropy 0, no gradient.
"""
import numpy as np

from .kv import rotate


def rms(x, eps):
    return 1 / np.sqrt(np.mean(np.square(x), -1, keepdims=True) + eps)


def norm_rope(x, w, eps, cos=None, sin=None, interleaved=False):
    """x [tokens, heads, D], w [D] or [heads, D], cos and sin [tokens, r / 2]."""
    y = x * rms(x, eps) * w
    return y if cos is None else rotate(y, cos[:, None], sin[:, None], interleaved)


def norm_rope_backward(dy, x, w, eps, cos=None, sin=None, interleaved=False):
    """(dx, dw) by the chain rule; dw of w's shape."""
    g = dy if cos is None else rotate(dy, cos[:, None], -sin[:, None], interleaved)
    r = rms(x, eps)
    dw = (g * x * r).sum(0 if w.ndim == 2 else (0, 1))
    u = g * w
    # d(x_i r) / dx_j = r (delta_ij - x_i x_j r^2 / D)
    dx = r * u - r ** 3 * x * np.mean(u * x, -1, keepdims=True)
    return dx, dw


def logprobs(x, targets, scale=1.0, top=0):
    """dict of lse, logprob, entropy [rows], top_id, top_logprob [rows, top]."""
    rows, vocab = x.shape
    out = dict(lse=np.zeros(rows), logprob=np.zeros(rows), entropy=np.zeros(rows),
               top_id=np.zeros((rows, top), np.int64), top_logprob=np.zeros((rows, top)))
    for n in range(rows):
        z = x[n] * scale
        order = np.argsort(-np.where(np.isnan(x[n]), -np.inf, x[n]), kind="stable")[:top]
        out["top_id"][n] = order
        t = targets[n]
        if np.isnan(z).any() or (z == np.inf).any():
            out["lse"][n] = out["entropy"][n] = np.nan
            out["top_logprob"][n] = np.nan
            out["logprob"][n] = np.nan if 0 <= t < vocab else 0.0
            continue
        m = z.max()
        if m == -np.inf:
            out["lse"][n] = -np.inf
            out["top_logprob"][n] = -np.inf
            out["logprob"][n] = -np.inf if 0 <= t < vocab else 0.0
            continue
        lse = m + np.log(np.exp(z - m).sum())
        lp = z - lse
        p = np.exp(lp)
        out["lse"][n] = lse
        out["logprob"][n] = lp[t] if 0 <= t < vocab else 0.0
        out["entropy"][n] = -(p[p > 0] * lp[p > 0]).sum()
        out["top_logprob"][n] = lp[order]
    return out


def logprobs_backward(x, targets, g, h, scale=1.0):
    """The gradient of sum g logprob + h entropy with respect to x."""
    r = logprobs(x, targets, scale)
    dx = np.zeros(x.shape)
    for n in range(x.shape[0]):
        if r["lse"][n] == -np.inf:
            continue
        lp = x[n] * scale - r["lse"][n]
        p = np.exp(lp)
        lp = np.where(p > 0, lp, 0.0)
        dz = -h[n] * p * (lp + r["entropy"][n])
        if 0 <= targets[n] < x.shape[1]:
            dz -= g[n] * p
            dz[targets[n]] += g[n]
        dx[n] = dz * scale
    return dx
