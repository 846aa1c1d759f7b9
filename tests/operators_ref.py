"""Plain 64-bit forms of the norm, recurrence and epilogue operators, with the
error bounds their tests use.  numpy only; inputs are float64 arrays that hold
the exact values of the tensors under test.

Bounds.  u = 2^-24 is half a float ulp (relative, 24 bits of significand),
2^-8 half a bf16 ulp (8 bits).  A
float sum of n terms in any order is off by at most (n + 1) u times the sum of
magnitudes.  CUDA documents __expf at 2 + floor(1.173 |x|) ulp and __fdividef at
2 ulp, so sigmoid(x), as a ratio of two such results and one addition, is
within LOGISTIC(x) relative of the truth.
"""
import numpy as np

U = 2.0 ** -24
HALF_ULP = {"bf16": 2.0 ** -8, "f32": U}


def logistic_error(x):
    return (2 + 1.173 * np.minimum(np.abs(x), 128.0) + 2 + 2) * 2 * U


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1, e) / (1 + e)


# ------------------------------------------------------------------- norm ---

def norm(s, gamma, eps):
    """rstd, row_scale and the values y of rows s (already summed and rounded)."""
    cols = s.shape[1]
    rstd = 1 / np.sqrt((s * s).sum(1) / max(cols, 1) + eps)
    y = s * rstd[:, None] * gamma
    scale = np.abs(y).max(1) / 127 if cols else np.zeros(len(s))
    return rstd, scale, y


def norm_codes(s, gamma):
    """The int8 codes, step by step in float32 as the declaration gives them."""
    u = s.astype(np.float32) * gamma.astype(np.float32)
    amax = np.abs(u).max(1) if u.shape[1] else np.zeros(len(u), np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(amax > 0, np.float32(127) / amax, np.float32(0)).astype(np.float32)
    return np.clip(np.rint(u * inv[:, None]), -127, 127).astype(np.int8)


def norm_bwd(dy, s, rstd, gamma, dsum):
    """(dx, dgamma, magnitude of dx's terms, sum of magnitudes for dgamma)."""
    n = dy * gamma
    r = rstd[:, None]
    mean = (n * s).mean(1, keepdims=True)
    dx = r * (n - s * r * r * mean) + dsum
    mag = r * (np.abs(n) + np.abs(s) * r * r * np.abs(n * s).mean(1, keepdims=True)) + np.abs(dsum)
    return dx, (dy * s * r).sum(0), mag, np.abs(dy * s * r).sum(0)


# ------------------------------------------------------------- recurrence ---

def scan(gate, cand, h0, resets):
    """(h, prior, error): states, the states each step started from, and the
    bound on a float computation of h.  A step h' + k (c - h') loses the error
    of k times |c - h'| and two roundings; maps composed in a tree repeat at
    most three such evaluations of each step."""
    k = sigmoid(-gate)
    kerr = logistic_error(gate) * k
    h, prior, err = np.zeros_like(gate), np.zeros_like(gate), np.zeros_like(gate)
    state, e = h0.copy(), np.zeros_like(h0)
    for t in range(gate.shape[1]):
        keep = (resets[:, t] == 0)[:, None]
        state, e = state * keep, e * keep
        prior[:, t] = state
        c = np.where(k[:, t] == 0, 0, cand[:, t])
        e = (1 - k[:, t]) * e + 3 * (kerr[:, t] * np.abs(c - state) + 2 * U * (np.abs(c - state) * k[:, t] + np.abs(state)))
        state = state + k[:, t] * (c - state)
        h[:, t], err[:, t] = state, e
    return h, prior, err


def scan_bwd(gate, cand, prior, dh, resets, dh_last):
    """(dgate, dcand, dh0) and their bounds; prior is the state each step
    started from (0 at a reset)."""
    a, k = sigmoid(gate), sigmoid(-gate)
    kerr = logistic_error(gate)
    dgate, dcand = np.zeros_like(gate), np.zeros_like(gate)
    egate, ecand = np.zeros_like(gate), np.zeros_like(gate)
    back, e = dh_last.copy(), np.zeros_like(dh_last)
    for t in reversed(range(gate.shape[1])):
        g = back + dh[:, t]
        e = e + 3 * U * (np.abs(back) + np.abs(dh[:, t]))
        kt, diff = k[:, t], prior[:, t] - cand[:, t]
        dcand[:, t] = g * kt
        ecand[:, t] = kt * e + (kerr[:, t] + U) * np.abs(g) * kt
        dgate[:, t] = g * diff * a[:, t] * kt
        egate[:, t] = a[:, t] * kt * (np.abs(diff) * (e + (2 * kerr[:, t] + 4 * U) * np.abs(g)) +
                                      U * np.abs(g) * (np.abs(prior[:, t]) + np.abs(cand[:, t])))
        keep = (resets[:, t] == 0)[:, None]
        back = g * a[:, t] * keep
        e = (a[:, t] * e + 3 * (kerr[:, t] * kt + U) * np.abs(g)) * keep
    return (dgate, dcand, back), (egate, ecand, e)


# --------------------------------------------------------------- epilogue ---

ACTS = ("none", "relu", "relu2", "silu", "gelu")
GELU = np.sqrt(2 / np.pi)


def act(z, name):
    """(act(z), act'(z), relative error of a float evaluation)."""
    flat = np.full_like(z, 4 * U)
    if name == "none":
        return z, np.ones_like(z), flat
    if name == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64), flat
    if name == "relu2":
        return np.maximum(z, 0) ** 2, 2 * np.maximum(z, 0), flat
    if name == "silu":
        s = sigmoid(z)
        return z * s, s + z * s * (1 - s), logistic_error(z) + flat
    u = 2 * GELU * (z + 0.044715 * z ** 3)
    s = sigmoid(u)
    # the argument is itself rounded (five roundings), which the exponential
    # turns into a relative error of |u| times as much
    return (z * s, s + z * s * (1 - s) * 2 * GELU * (1 + 3 * 0.044715 * z * z),
            logistic_error(u) + flat + 6 * U * np.abs(u))
