"""Rows far from zero for the layer norm's tests, and what its moments have to meet there.

Bounds.  U = 2^-24 is half a float ulp.  A sum over a row has `depth` additions on its longest path
(a thread's elements, then a tree).  A first mean m0 is off by (depth + 2) U |mean| + (depth + 2) U mean|d|, d the
deviations.  The mean of the differences s - m0, each off by U of itself, is off by (depth + 3) U mean|s - m0|, and
adding it to m0 rounds once: the mean is off by
    em = U |mean| + (depth + 4) U (mean|d| + e0),  e0 = m0's error.
Squares of differences from m0, less n (mean - m0)^2, are off by (2 depth + 8) U of their sum and twice that of the
part taken away, n e0^2, and by n em^2: the variance by
    (2 depth + 8) U (var + 2 e0^2) + em^2.
The division, the sum with eps, the root and its reciprocal add 8 U."""
import numpy as np

U = 2.0 ** -24


def rows(n, cols, mean):
    return (np.random.default_rng(cols).standard_normal((n, cols)) + mean).astype(np.float32)


def depth(cols):
    """16 elements a thread and a tree over 1024 threads; rows too long for that have cols / 1024 a thread."""
    return max(16, -(-cols // 1024)) + 12


def check(s, eps, mean, rstd, scale, q):
    """Asserts the moments, scales and codes of the layer norm of s without gain and shift."""
    s = s.astype(np.float64)
    eps = np.float64(np.float32(eps))
    n, D = s.shape[1], depth(s.shape[1])
    wm = s.sum(1) / n
    dev = s - wm[:, None]
    mad, var = np.abs(dev).sum(1) / n, (dev * dev).sum(1) / n
    wr = 1 / np.sqrt(var + eps)
    e0 = (D + 2) * U * (np.abs(wm) + mad)
    em = U * np.abs(wm) + (D + 4) * U * (mad + e0)
    er = 0.5 * ((2 * D + 8) * U * (var + 2 * e0 * e0) + em * em) / (var + eps) + 8 * U
    assert np.all(np.abs(mean - wm) <= em), "mean"
    assert np.all(np.abs(rstd - wr) <= er * wr), "rstd"
    h = dev * wr[:, None]
    ey = (em * wr)[:, None] + np.abs(h) * er[:, None] + 4 * U * np.abs(h)
    ws, es = np.abs(h).max(1) / 127, ey.max(1) / 127
    assert np.all(np.abs(scale - ws) <= es + 4 * U * ws), "scale"
    off = np.abs(q * ws[:, None] - h)
    assert np.all(off <= ws[:, None] * (0.5 + 127 * 6 * U) + ey + 127 * (es + 4 * U * ws)[:, None]), "codes"
