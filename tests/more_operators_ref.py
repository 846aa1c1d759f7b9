"""Plain 64-bit forms of the layer norm, the gated feed-forward product and
linear attention, with the error bounds their tests use.  numpy only; inputs are
float64 arrays that hold the exact values of the tensors under test.

Bounds.  U = 2^-24 is half a float ulp, HALF_ULP half a step of a stored type.  A float
sum of n terms in any order is off by at most (n + 1) U times the sum of magnitudes.
"""
import numpy as np

U = 2.0 ** -24
HALF_ULP = {"bf16": 2.0 ** -8, "f32": U}


# ------------------------------------------------------------- layer norm ---

def layer_norm(s, gamma, beta, eps):
    """(mean, rstd, row_scale, y, bounds of a float computation of each).  A mean m is off
    by em = (n + 16) U mean|s|.  Squares of differences from such a mean, joined
    over parts by their means, are off by 2 em (sum of deviations) + 3 n em^2, and by
    their own sum's roundings; the division, sum with eps, root and reciprocal add 8 U."""
    n = max(s.shape[1], 1)
    mean = s.sum(1) / n
    dev = s - mean[:, None]
    var = (dev * dev).sum(1) / n
    rstd = 1 / np.sqrt(var + eps)
    h = dev * rstd[:, None]
    y = h * gamma + beta
    scale = np.abs(y).max(1) / 127 if s.shape[1] else np.zeros(len(s))
    em = (n + 16) * U * np.abs(s).sum(1) / n
    er = 0.5 * (2 * em * np.sqrt(var) + 3 * em * em + (n + 16) * U * var) / (var + eps) + 8 * U
    ey = np.abs(gamma) * ((em * rstd)[:, None] + np.abs(h) * er[:, None]) + 4 * U * (np.abs(h * gamma) + np.abs(beta))
    es = ey.max(1) / 127 + 4 * U * scale if s.shape[1] else np.zeros(len(s))
    return mean, rstd, scale, y, (em, er, es, ey)


def layer_norm_bwd(dy, s, mean, rstd, gamma, dsum):
    """(dx, dgamma, dbeta, magnitude of dx's terms, sums of magnitudes of the columns')."""
    h = (s - mean[:, None]) * rstd[:, None]
    n = dy * gamma
    r = rstd[:, None]
    dx = r * (n - n.mean(1, keepdims=True) - h * (n * h).mean(1, keepdims=True)) + dsum
    mag = r * (np.abs(n) + np.abs(n).mean(1, keepdims=True) + np.abs(h) * np.abs(n * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0), mag + np.abs(dsum), np.abs(dy * h).sum(0), np.abs(dy).sum(0)
