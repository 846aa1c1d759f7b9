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


# ------------------------------------------------- gated feed-forward ------

ACTS = ("none", "relu", "relu2", "silu", "gelu")


def _logistic_error(x):
    """Bound on sigmoid(x) from an exponential of 2 ulp whose argument, a product of at most
    three roundings, is off by 4 U of itself, one addition and a reciprocal of 1 ulp."""
    return (4 + 2 + 2 + 4 * 1.45 * np.minimum(np.abs(x), 128.0)) * 2 * U


def act(z, kind):
    """(act(z), act'(z), bounds of a float computation of each, absolute)."""
    zero = np.zeros_like(z)
    if kind == "none":
        return z, zero + 1, zero, zero
    if kind == "relu":
        return np.maximum(z, 0), (z > 0) * 1.0, zero, zero
    if kind == "relu2":
        p = np.maximum(z, 0)
        return p * p, 2 * p, 2 * U * p * p, 2 * U * p
    with np.errstate(over="ignore"):
        if kind == "silu":
            x, dx = z, zero + 1
        else:  # z sigmoid(2 u): (1 + tanh u) / 2 = sigmoid(2 u)
            c = 2 * np.sqrt(2 / np.pi)
            x, dx = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)
        e = np.exp(-np.abs(x))
        s = np.where(x >= 0, 1, e) / (1 + e)
        flat = e / (1 + e) ** 2
    rel = _logistic_error(x)
    y, slope = z * s, s + z * flat * dx
    # the exponential flushes results below 2^-126 to 0: s and flat, each at most the exponential, are
    # off by as much, y by |z| of it and the slope by (1 + |z dx|) of it
    flush = 2.0 ** -126
    return (y, slope, (rel + 4 * U) * np.abs(y) + flush * np.abs(z),
            (2 * rel + 8 * U) * (s + np.abs(z * flat * dx)) + flush * (1 + np.abs(z * dx)))


def glu_z(x, rs, cs, bias):
    """z in float32, rounding by rounding, from the exact integer product."""
    z = x.astype(np.float32)
    if rs is not None:
        z = z * rs[:, None]
    if cs is not None:
        z = z * cs
    return z + bias if bias is not None else z


def glu_bwd(dy, gate, up, kind):
    """(dgate, dup, their bounds before the rounding)."""
    y, slope, ey, es = act(gate, kind)
    dgate, dup = dy * up * slope, dy * y
    return dgate, dup, np.abs(dy * up) * es + 4 * U * np.abs(dgate), np.abs(dy) * ey + 4 * U * np.abs(dup)


# --------------------------------------------------------- linear attention ---

def linear_attend(q, k, v, log_decay, state, resets, scale, reverse=False, chunks=False):
    """The recurrence of linear attention over [batch][length][heads][d], token by token in 64 bits, and
    bounds of its float computation.  reverse: against time, a mark cutting a token off from the
    one behind it, and the first token taken undecayed.  Returns (o, last state, bound of
    o before its rounding, bound of the state).

    With A the recurrence of magnitudes, a state is off by E: the decay's relative error (its
    argument's rounding and an exponential of 2 ulp) and three roundings a step; o by q E and a float
    sum's roundings.  Parts joined along a sequence repeat at most each of these once.
    chunks: q k^T and the state are rounded to bf16 on their way to o, 2^-8 each, and what is added
    to the state to 2^-16 (two bf16 terms)."""
    batch, length, heads, dk = q.shape
    decay = np.exp(log_decay)[None, :, None, None]
    with np.errstate(invalid="ignore"):
        err = np.where(np.isinf(log_decay), 0, 6 + 3 * np.abs(np.where(np.isinf(log_decay), 0, log_decay)))[None, :, None, None] * U
    order = range(length - 1, -1, -1) if reverse else range(length)
    S = np.zeros((batch, heads, dk, v.shape[3])) if state is None else state.copy()
    A, E = np.abs(S), np.zeros_like(S)
    o = np.empty((batch, length, heads, v.shape[3]))
    eo = np.empty_like(o)
    add = (2.0 ** -16 if chunks else 0) + 4 * U
    meet = 2.0 ** -8 if chunks else 0
    for t in order:
        mark = t + 1 if reverse else t
        if resets is not None and mark < length:
            live = (resets[:, mark] == 0)[:, None, None, None]
            S, A, E = np.where(live, S, 0), np.where(live, A, 0), np.where(live, E, 0)
        c = 1.0 if reverse and t == length - 1 else decay
        kv = k[:, t, :, :, None] * v[:, t, :, None, :]
        E = c * (E + (err + 3 * U) * A) + add * np.abs(kv)
        S, A = c * S + kv, c * A + np.abs(kv)
        qt = q[:, t, :, None, :]
        o[:, t] = scale * (qt @ S)[:, :, 0]
        eo[:, t] = abs(scale) * (np.abs(qt) @ (2 * E + (meet + (dk + 16) * U) * A))[:, :, 0]
    return o, S, eo, 2 * E + 4 * U * np.abs(S)


def linear_attend_bwd(q, k, v, log_decay, do, state, resets, scale, dlast, chunks=False):
    """{name: (gradient, bound before its rounding)} of q, k, v and the state."""
    t = (0, 1, 3, 2)
    swap = lambda s: None if s is None else s.transpose(t)  # noqa: E731
    dq, _, eq, _ = linear_attend(do, v, k, log_decay, swap(state), resets, scale, chunks=chunks)
    dv, ds, ev, es = linear_attend(k, scale * q, do, log_decay, dlast, resets, 1.0, True, chunks)
    dk, _, ek, _ = linear_attend(v, do, scale * q, log_decay, swap(dlast), resets, 1.0, True, chunks)
    decay = np.exp(log_decay)[None, :, None, None]
    live = 1.0 if resets is None else (resets[:, 0] == 0)[:, None, None, None]
    ds = np.where(live, ds * decay, 0)
    es = np.where(live, es * decay + np.abs(ds) * (8 + 3 * np.abs(np.where(np.isinf(log_decay), 0, log_decay)))[None, :, None, None] * U, 0)
    return {"q": (dq, eq), "k": (dk, ek), "v": (dv, ev), "state": (ds, es)}
