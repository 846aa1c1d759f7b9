"""What the layer norm's bounds on rows far from zero tell apart: the moments as the kernels take them
meet them, a deviation as the difference of two sums does not."""
import numpy as np
import pytest

import moments_ref

EPS = 1e-5
F = np.float32


def _tree(x):
    """A float sum over the last axis: 16 elements a thread in turn (more in long rows), then pairs."""
    each = max(16, -(-x.shape[1] // 1024))
    pad = -x.shape[1] % each
    x = np.pad(x, ((0, 0), (0, pad))).reshape(len(x), -1, each)
    t = x[..., 0]
    for j in range(1, each):
        t = (t + x[..., j]).astype(F)
    while t.shape[1] > 1:
        t = np.pad(t, ((0, 0), (0, t.shape[1] % 2)))
        t = (t[:, ::2] + t[:, 1::2]).astype(F)
    return t[:, 0]


def _outputs(s, mean, var):
    rstd = (1 / np.sqrt(var.astype(np.float64) + EPS)).astype(F)
    y = ((s - mean[:, None]) * rstd[:, None]).astype(F)
    top = np.abs(y).max(1)
    return mean, rstd, top / F(127), np.rint(y * (F(127) / top)[:, None])


CASES = [(c, m) for c in (64, 729, 1000, 4096, 8200, 12292, 20000, 33001) for m in (100.0, -3e4)]


@pytest.mark.parametrize("cols,mean", CASES)
def test_two_passes_with_the_mean_corrected_meet_them(cols, mean):
    s = moments_ref.rows(40, cols, mean)
    inv = F(1) / F(cols)
    m0 = (_tree(s) * inv).astype(F)
    d = (s - m0[:, None]).astype(F)
    rest = _tree(d)
    m = (m0 + rest * inv).astype(F)
    m2 = (_tree((d * d).astype(F)) - rest * rest * inv).astype(F)
    moments_ref.check(s, EPS, *_outputs(s, m, (m2 * inv).astype(F)))


@pytest.mark.parametrize("cols,mean", CASES)
def test_a_difference_of_sums_does_not(cols, mean):
    s = moments_ref.rows(40, cols, mean)
    inv = F(1) / F(cols)
    m = (_tree(s) * inv).astype(F)
    var = np.maximum((_tree((s * s).astype(F)) * inv).astype(F) - (m * m).astype(F), F(0))
    with pytest.raises(AssertionError, match="rstd"):
        exact = s.astype(np.float64).mean(1).astype(F)  # its mean is not what is told apart here
        moments_ref.check(s, EPS, *_outputs(s, exact, var))
